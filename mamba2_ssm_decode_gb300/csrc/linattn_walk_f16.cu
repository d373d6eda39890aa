// linattn_walk_f16.cu -- the recurrent form of linear attention for fp16 rows.
#include "linattn_walk.cuh"

namespace linattn {

cudaError_t launch_walk_f16(const Args& p, const Seqs& a, cudaStream_t stream) {
  return launch_walk_io<__half>(p, a, stream);
}

}  // namespace linattn
