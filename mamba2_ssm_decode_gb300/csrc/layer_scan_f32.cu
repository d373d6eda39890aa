// layer_scan_f32.cu -- the selective scan's kernels for f32 rows.
#include "layer_scan_prompt.cuh"

namespace layer {

cudaError_t launch_scan_f32(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream) {
  return launch_scan_io<float>(N, p, a, stream);
}

cudaError_t launch_prompt_f32(int N, const ScanArgs& p, const Seqs& a,
                           cudaStream_t stream) {
  return launch_scan_prompt_n<float, float>(N, p, a, stream);
}

}  // namespace layer
