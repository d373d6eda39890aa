// layer_scan_bf16.cu -- the selective scan's kernels for bf16 rows.
#include "layer_scan.cuh"

namespace layer {

cudaError_t launch_scan_bf16(ssu_dtype state, int N, const ScanArgs& p, const VarlenArgs& a,
                          int64_t nseqs, cudaStream_t stream) {
  return launch_scan_io<__nv_bfloat16>(state, N, p, a, nseqs, stream);
}

}  // namespace layer
