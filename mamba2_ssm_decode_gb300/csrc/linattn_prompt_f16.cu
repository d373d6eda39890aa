// linattn_prompt_f16.cu -- linear attention over prompts of fp16 rows.
#include "linattn_prompt_launch.cuh"

namespace linattn {

cudaError_t launch_pieces_f16(const PromptArgs& g, int ctas, cudaStream_t stream) {
  return launch_prompt_io<__half, 2, false>(g, ctas, stream);
}

cudaError_t launch_chunks_f16(const PromptArgs& g, int ctas, cudaStream_t stream) {
  return launch_prompt_io<__half, 2, true>(g, ctas, stream);
}

}  // namespace linattn
