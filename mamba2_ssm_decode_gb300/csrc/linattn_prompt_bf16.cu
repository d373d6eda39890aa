// linattn_prompt_bf16.cu -- linear attention over prompts of bf16 rows.
#include "linattn_prompt_launch.cuh"

namespace linattn {

cudaError_t launch_pieces_bf16(const PromptArgs& g, int ctas, cudaStream_t stream) {
  return launch_prompt_io<__nv_bfloat16, 3, false>(g, ctas, stream);
}

cudaError_t launch_chunks_bf16(const PromptArgs& g, int ctas, cudaStream_t stream) {
  return launch_prompt_io<__nv_bfloat16, 3, true>(g, ctas, stream);
}

}  // namespace linattn
