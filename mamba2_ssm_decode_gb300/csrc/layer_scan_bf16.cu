// layer_scan_bf16.cu -- the selective scan's kernels for bf16 rows.
#include "layer_scan_prompt.cuh"

namespace layer {

cudaError_t launch_scan_bf16(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream) {
  return launch_scan_io<__nv_bfloat16>(N, p, a, stream);
}

cudaError_t launch_prompt_bf16(int N, const ScanArgs& p, const Seqs& a,
                           cudaStream_t stream) {
  if (!p.dt_f32) return launch_scan_prompt_n<__nv_bfloat16, __nv_bfloat16>(N, p, a, stream);
  return launch_scan_prompt_n<__nv_bfloat16, float>(N, p, a, stream);
}

}  // namespace layer
