// layer_scan_f16.cu -- the selective scan's kernels for f16 rows.
#include "layer_scan.cuh"

namespace layer {

cudaError_t launch_scan_f16(ssu_dtype state, int N, const ScanArgs& p, const VarlenArgs& a,
                          int64_t nseqs, cudaStream_t stream) {
  return launch_scan_io<__half>(state, N, p, a, nseqs, stream);
}

}  // namespace layer
