// layer_scan_f16.cu -- the selective scan's kernels for f16 rows.
#include "layer_scan_prompt.cuh"

namespace layer {

cudaError_t launch_scan_f16(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream) {
  return launch_scan_io<__half>(N, p, a, stream);
}

cudaError_t launch_prompt_f16(int N, const ScanArgs& p, const Seqs& a,
                           cudaStream_t stream) {
  if (!p.dt_f32) return launch_scan_prompt_n<__half, __half>(N, p, a, stream);
  return launch_scan_prompt_n<__half, float>(N, p, a, stream);
}

}  // namespace layer
