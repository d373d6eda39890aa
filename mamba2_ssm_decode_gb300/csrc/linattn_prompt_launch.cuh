// linattn_prompt_launch.cuh -- launches of the prompt kernels of one type.
#pragma once

#include "linattn_prompt.cuh"

namespace linattn {

template <class IT, int DV, int DK, int PARTS, bool FULL>
cudaError_t launch_chunks(const PromptArgs& g, int ctas, cudaStream_t stream) {
  auto kernel = linattn_prompt_kernel<IT, DV, DK, PARTS, FULL>;
  constexpr int smem = (int)sizeof(PromptSmem<DV, DK, PARTS>);
  static_assert(smem <= 227 * 1024, "shared memory of an SM");
  // one CTA an SM: each takes all of the tensor memory
  constexpr int ask = smem > 116 * 1024 ? smem : 116 * 1024;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ask);
  if (e != cudaSuccess) return e;
  // what the warps' shares of the registers add up to
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != 80) return cudaErrorInvalidConfiguration;
  return launch_after(kernel, dim3((unsigned)ctas), kPromptThreads, ask, stream, g);
}

template <class IT, int PARTS, bool FULL>
cudaError_t launch_prompt_io(const PromptArgs& g, int ctas, cudaStream_t stream) {
  const int dv = g.p.dv, dk = g.p.dk;
  if (dv == 128 && dk == 128) return launch_chunks<IT, 128, 128, PARTS, FULL>(g, ctas, stream);
  if (dv == 128 && dk == 64) return launch_chunks<IT, 128, 64, PARTS, FULL>(g, ctas, stream);
  if (dv == 64 && dk == 128) return launch_chunks<IT, 64, 128, PARTS, FULL>(g, ctas, stream);
  if (dv == 64 && dk == 64) return launch_chunks<IT, 64, 64, PARTS, FULL>(g, ctas, stream);
  return cudaErrorInvalidValue;
}

}  // namespace linattn
