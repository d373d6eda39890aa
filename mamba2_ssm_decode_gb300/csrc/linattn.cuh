// linattn.cuh -- linear attention with a decay for each head: per sequence and
// value head h, with g = h / (heads / groups), over the rows in order
//     S[p][n] <- e^ld S[p][n] + v[p] k[g][n]        (dv x dk, in fp32)
//     o[p]     = scale sum_n S[p][n] q[g][n]
// ld being 0, one value per head, or one per row and head.  A state is rounded
// only where it is stored.
#pragma once

#include "layer_common.cuh"

namespace linattn {
using namespace layer;

struct Args {
  void* state;
  int state_dtype;  // ssu_dtype
  int64_t slots;
  int H, G, hr;  // value heads, groups of queries and keys, heads per group
  int dv, dk;
  const void* q;
  int64_t q_rs, q_gs;
  const void* k;
  int64_t k_rs, k_gs;
  const void* v;
  int64_t v_rs, v_hs;
  void* out;
  int64_t o_rs, o_hs;
  const float* ld;  // nullptr: no decay
  int64_t ld_rs, ld_hs;  // ld_rs 0: one value per head
  float scale;
  int qk_vec;  // every vector of q and k starts on a 16-byte boundary
  int v_vec;   // so does every one of v
  int o_vec;   // ... and of out
  int disable;
  int64_t pad;
  int prompt;  // the state is written once, after the last row
  const uint8_t* has_init;  // prompts: per sequence, or NULL: every valid slot is read
};

// Rows [r0, r0 + len) of a sequence from the slot it reads; one launch.
cudaError_t launch_walk_f32(const Args& p, const Seqs& a, cudaStream_t stream);
cudaError_t launch_walk_bf16(const Args& p, const Seqs& a, cudaStream_t stream);
cudaError_t launch_walk_f16(const Args& p, const Seqs& a, cudaStream_t stream);

// Prompts on the tensor cores (linattn_prompt.cuh): whether they take such a call,
// and the bytes of workspace it needs.
bool takes_prompt(int64_t rows, int64_t nseqs, int64_t heads, int64_t dv, int64_t dk,
                  ssu_dtype io);
int64_t prompt_workspace(int64_t rows, int64_t nseqs, int64_t heads, int64_t dv, int64_t dk);
cudaError_t launch_prompt(const Args& p, const Seqs& a, ssu_dtype io, void* workspace,
                          cudaStream_t stream);

}  // namespace linattn
