// linattn_walk_bf16.cu -- the recurrent form of linear attention for bf16 rows.
#include "linattn_walk.cuh"

namespace linattn {

cudaError_t launch_walk_bf16(const Args& p, const Seqs& a, cudaStream_t stream) {
  return launch_walk_io<__nv_bfloat16>(p, a, stream);
}

}  // namespace linattn
