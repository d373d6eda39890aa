// linattn_walk_f32.cu -- the recurrent form of linear attention for fp32 rows.
#include "linattn_walk.cuh"

namespace linattn {

cudaError_t launch_walk_f32(const Args& p, const Seqs& a, cudaStream_t stream) {
  return launch_walk_io<float>(p, a, stream);
}

}  // namespace linattn
