// layer_scan_f32.cu -- the selective scan's kernels for f32 rows.
#include "layer_scan.cuh"

namespace layer {

cudaError_t launch_scan_f32(ssu_dtype state, int N, const ScanArgs& p, const VarlenArgs& a,
                          int64_t nseqs, cudaStream_t stream) {
  return launch_scan_io<float>(state, N, p, a, nseqs, stream);
}

}  // namespace layer
