// linattn.cu -- argument checks and entry points of linear attention.
#include "linattn.cuh"

namespace linattn {

// heads are the grid's second dimension, items of a prompt call are counted in 32 bits
constexpr int64_t kMostHeads = 4096, kMostDim = 256;

static ssu_status check(const ssu_linattn_params* c, int64_t rows, bool pool_needed, Args* p) {
  if (!c) return fail(SSU_ERR_INVALID_ARGUMENT, "params must not be NULL");
  if (!is_float(c->state_dtype))
    return fail(SSU_ERR_UNSUPPORTED, "state dtype must be f32, bf16 or f16");
  if (!is_float(c->io_dtype))
    return fail(SSU_ERR_UNSUPPORTED, "q/k/v dtype must be f32, bf16 or f16");
  if (c->slots < 0 || c->nheads < 1 || c->ngroups < 1 || c->dv < 1 || c->dk < 1)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "state must be [slots, heads, dv, dk] with positive sizes, got [%lld, %lld, %lld, "
                "%lld], ngroups %lld",
                (long long)c->slots, (long long)c->nheads, (long long)c->dv, (long long)c->dk,
                (long long)c->ngroups);
  if (c->nheads % c->ngroups != 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "heads (%lld) must be a multiple of the groups (%lld)",
                (long long)c->nheads, (long long)c->ngroups);
  if (c->nheads > kMostHeads || c->dv > kMostDim)
    return fail(SSU_ERR_UNSUPPORTED, "at most %lld heads of dv at most %lld, got %lld and %lld",
                (long long)kMostHeads, (long long)kMostDim, (long long)c->nheads, (long long)c->dv);
  const int64_t n = c->dk;
  if (n != 16 && n != 32 && n != 64 && n != 128 && n != 256)
    return fail(SSU_ERR_UNSUPPORTED, "dk %lld is not one of 16, 32, 64, 128, 256", (long long)n);
  if (rows > 0 && (!c->q || !c->k || !c->v || !c->out))
    return fail(SSU_ERR_INVALID_ARGUMENT, "q, k, v and out must not be NULL");
  if ((rows > 1 && c->out_row_stride < c->dv) || (c->nheads > 1 && c->out_head_stride < c->dv))
    return fail(SSU_ERR_INVALID_ARGUMENT, "out's rows or heads overlap");
  if (pool_needed && !c->state && c->slots > 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "state must not be NULL");
  if (!aligned(c->state, 16))
    return fail(SSU_ERR_INVALID_ARGUMENT, "state must be 16-byte aligned");
  const int es = size_of(c->io_dtype);
  if (!aligned(c->q, es) || !aligned(c->k, es) || !aligned(c->v, es) || !aligned(c->out, es) ||
      !aligned(c->log_decay, 4))
    return fail(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their element size");
  *p = Args{};
  p->state = c->state;
  p->state_dtype = c->state_dtype;
  p->slots = c->state ? c->slots : 0;
  p->H = (int)c->nheads;
  p->G = (int)c->ngroups;
  p->hr = p->H / p->G;
  p->dv = (int)c->dv;
  p->dk = (int)c->dk;
  p->q = c->q;
  p->q_rs = c->q_row_stride;
  p->q_gs = c->q_group_stride;
  p->k = c->k;
  p->k_rs = c->k_row_stride;
  p->k_gs = c->k_group_stride;
  p->v = c->v;
  p->v_rs = c->v_row_stride;
  p->v_hs = c->v_head_stride;
  p->out = c->out;
  p->o_rs = c->out_row_stride;
  p->o_hs = c->out_head_stride;
  p->ld = c->log_decay;
  p->ld_rs = c->log_decay_row_stride;
  p->ld_hs = c->log_decay_head_stride;
  p->scale = c->scale;
  auto on16 = [&](const void* ptr, int64_t rs, int64_t n, int64_t is) {
    return aligned(ptr, 16) && rs * es % 16 == 0 && (n == 1 || is * es % 16 == 0);
  };
  p->qk_vec = on16(c->q, p->q_rs, p->G, p->q_gs) && on16(c->k, p->k_rs, p->G, p->k_gs);
  p->v_vec = on16(c->v, p->v_rs, p->H, p->v_hs);
  p->o_vec = on16(c->out, p->o_rs, p->H, p->o_hs);
  p->disable = c->disable_state_update != 0;
  p->pad = c->pad_slot_id;
  return SSU_OK;
}

// out against what other threads read
static ssu_status check_out(const ssu_linattn_params* c, int64_t rows) {
  const Rows out = rows_of(c->out, c->out_row_stride, c->nheads, c->out_head_stride, c->dv,
                           c->io_dtype);
  // heads that lie behind all rows of the one before: a stride between rows alone says that
  if (c->nheads > 1 && rows > 1 && c->out_head_stride < c->out_row_stride
      && c->out_row_stride < (c->nheads - 1) * c->out_head_stride + c->dv)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out's rows and heads overlap");
  if (c->nheads > 1 && rows > 1 && c->out_head_stride >= c->out_row_stride &&
      c->out_head_stride < (rows - 1) * c->out_row_stride + c->dv)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out's rows and heads overlap");
  const struct {
    const char* name;
    Rows rows;
  } in[] = {
      {"q", rows_of(c->q, c->q_row_stride, c->ngroups, c->q_group_stride, c->dk, c->io_dtype)},
      {"k", rows_of(c->k, c->k_row_stride, c->ngroups, c->k_group_stride, c->dk, c->io_dtype)},
      {"v", rows_of(c->v, c->v_row_stride, c->nheads, c->v_head_stride, c->dv, c->io_dtype)},
      {"log_decay", rows_of(c->log_decay, c->log_decay_row_stride, c->nheads,
                            c->log_decay_head_stride, 1, SSU_F32)},
  };
  for (const auto& v : in)
    if (overlap(out, v.rows, rows))
      return fail(SSU_ERR_INVALID_ARGUMENT, "out must not overlap %s", v.name);
  // ... and against the pool, from out's first byte to its last
  const int64_t last = (rows - 1) * c->out_row_stride + (c->nheads - 1) * c->out_head_stride + c->dv;
  const int64_t pool = c->slots * c->nheads * c->dv * c->dk;
  if (rows > 0 && c->state && pool > 0 &&
      overlap(Rows{c->out, 0, last * size_of(c->io_dtype)},
              Rows{c->state, 0, pool * size_of(c->state_dtype)}, 1))
    return fail(SSU_ERR_INVALID_ARGUMENT, "out must not overlap state");
  return SSU_OK;
}

static cudaError_t launch_walk(const ssu_linattn_params* c, const Args& p, const Seqs& a,
                               cudaStream_t stream) {
  switch (c->io_dtype) {
    case SSU_F32: return launch_walk_f32(p, a, stream);
    case SSU_BF16: return launch_walk_bf16(p, a, stream);
    case SSU_F16: return launch_walk_f16(p, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace linattn

#pragma GCC visibility push(default)
extern "C" {

ssu_status ssu_linattn_update(const ssu_linattn_params* c, int64_t nseqs, int64_t rows,
                              const void* cu_seqlens, int64_t dense_steps,
                              const void* num_accepted_tokens, ssu_dtype meta_dtype,
                              const ssu_slot_table* src, const ssu_slot_table* dst,
                              ssu_dtype index_dtype, struct CUstream_st* stream) {
  using namespace linattn;
  Args p;
  Seqs a;
  ssu_status st = check(c, rows, true, &p);
  if (st == SSU_OK)
    st = check_packed(c->slots, nseqs, rows, cu_seqlens, dense_steps, num_accepted_tokens,
                      meta_dtype, src, dst, index_dtype, &a);
  if (st == SSU_OK) st = check_out(c, rows);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  return launched(launch_walk(c, p, a, (cudaStream_t)stream));
}

int64_t ssu_linattn_workspace_bytes(int64_t rows, int64_t nseqs, int64_t nheads, int64_t dv,
                                    int64_t dk, ssu_dtype io_dtype) {
  if (rows < 0 || nseqs < 0 || nheads < 0 || dv < 0 || dk < 0) return -1;
  // sizes that the call refuses
  if (rows > 0x7fffffffLL - 1024 || nseqs >= 1LL << 30 || nheads > linattn::kMostHeads) return 0;
  if (rows == 0 || nseqs == 0 || nheads == 0 ||
      !linattn::takes_prompt(rows, nseqs, nheads, dv, dk, io_dtype))
    return 0;
  return linattn::prompt_workspace(rows, nseqs, nheads, dv, dk);
}

ssu_status ssu_linattn_fwd_varlen(const ssu_linattn_params* c, int64_t nseqs, int64_t rows,
                                  const void* cu_seqlens, ssu_dtype meta_dtype,
                                  const void* state_batch_indices,
                                  const void* dst_state_batch_indices, ssu_dtype index_dtype,
                                  const uint8_t* has_initial_state, void* workspace,
                                  int64_t workspace_bytes, struct CUstream_st* stream) {
  using namespace linattn;
  Args p;
  Seqs a;
  ssu_status st = check(c, rows, false, &p);
  if (st == SSU_OK)
    st = check_prompts(c->state != nullptr, c->slots, nseqs, rows, cu_seqlens, meta_dtype,
                       state_batch_indices, dst_state_batch_indices, index_dtype, &a);
  if (st == SSU_OK) st = check_out(c, rows);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  p.prompt = 1;
  p.has_init = has_initial_state;
  // tensor maps have rows on 16-byte boundaries, at positive strides below 2^40 bytes
  auto mapped = [](int64_t n, int64_t stride) { return n == 1 || (stride > 0 && stride < 1LL << 39); };
  const bool maps = p.qk_vec && p.v_vec && mapped(rows, p.q_rs) && mapped(p.G, p.q_gs) &&
                    mapped(rows, p.k_rs) && mapped(p.G, p.k_gs) && mapped(rows, p.v_rs) &&
                    mapped(p.H, p.v_hs);
  if (maps && takes_prompt(rows, nseqs, c->nheads, c->dv, c->dk, c->io_dtype)) {
    const int64_t need = prompt_workspace(rows, nseqs, c->nheads, c->dv, c->dk);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
      return fail(SSU_ERR_INVALID_ARGUMENT,
                  "ssu_linattn_fwd_varlen needs a 16-byte aligned workspace of %lld bytes, got %lld",
                  (long long)need, (long long)workspace_bytes);
    return launched(launch_prompt(p, a, c->io_dtype, workspace, (cudaStream_t)stream));
  }
  return launched(launch_walk(c, p, a, (cudaStream_t)stream));
}

}  // extern "C"
#pragma GCC visibility pop
