// layer_scan.cu -- argument checks and entry points of the selective scan, and
// the checks of sequence metadata that it shares with the convolution.
#include "layer_scan.cuh"

namespace layer {

static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// A run of a bytes at 0 and runs of b bytes at `at` + k stride, first <= k <= last: do any meet?
static bool run_meets(int64_t a, int64_t at, int64_t stride, int64_t b, int64_t first, int64_t last) {
  // at + k stride in (-b, a)
  if (stride == 0) return at > -b && at < a;
  if (stride < 0) return run_meets(a, at, -stride, b, -last, -first);
  int64_t lo = floor_div(-b - at, stride) + 1, hi = floor_div(a - 1 - at, stride);
  lo = lo > first ? lo : first;
  hi = hi < last ? hi : last;
  return lo <= hi;
}

// One run a row on both sides, b's first at `at` of a's.
static bool runs_overlap(const Rows& a, const Rows& b, int64_t at, int64_t rows) {
  const int64_t ea = a.stride * (rows - 1), eb = b.stride * (rows - 1);
  const int64_t a0 = ea < 0 ? ea : 0, a1 = (ea < 0 ? 0 : ea) + a.bytes;
  const int64_t b0 = at + (eb < 0 ? eb : 0), b1 = at + (eb < 0 ? 0 : eb) + b.bytes;
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.stride == b.stride) return run_meets(a.bytes, at, b.stride, b.bytes, 1 - rows, rows - 1);
  for (int64_t r = 0; r < rows; ++r)   // interleaved, at other strides
    if (run_meets(a.bytes, at - r * a.stride, b.stride, b.bytes, 0, rows - 1)) return true;
  return false;
}

bool overlap(const Rows& a, const Rows& b, int64_t rows) {
  if (!a.p || !b.p || rows < 1) return false;
  const int64_t at = (int64_t)((intptr_t)b.p - (intptr_t)a.p);
  auto from = [&](const Rows& v) {
    return (v.stride < 0 ? v.stride * (rows - 1) : 0) +
           (v.piece_stride < 0 ? v.piece_stride * (v.pieces - 1) : 0);
  };
  auto to = [&](const Rows& v) {
    return (v.stride < 0 ? 0 : v.stride * (rows - 1)) +
           (v.piece_stride < 0 ? 0 : v.piece_stride * (v.pieces - 1)) + v.bytes;
  };
  if (to(a) <= at + from(b) || at + to(b) <= from(a)) return false;
  for (int64_t i = 0; i < a.pieces; ++i)
    for (int64_t j = 0; j < b.pieces; ++j)
      if (runs_overlap(a, b, at + j * b.piece_stride - i * a.piece_stride, rows)) return true;
  return false;
}

// out against the operands that other threads read.  In place: out may be x, dt or z itself,
// whose elements are read by the thread's warp alone, before it writes them.
static ssu_status check_scan_out(const ssu_scan_params* c, int64_t rows, bool in_place) {
  const Rows out = rows_of(c->out, c->out_row_stride, c->channels, c->out_dtype);
  const struct {
    const char* name;
    Rows rows;
    bool elementwise;
  } in[] = {
      {"x", rows_of(c->x, c->x_row_stride, c->channels, c->io_dtype), true},
      {"dt", rows_of(c->dt, c->dt_row_stride, c->channels, c->dt_dtype), true},
      {"z", rows_of(c->z, c->z_row_stride, c->channels, c->io_dtype), true},
      {"B", rows_of(c->B, c->B_row_stride, c->ngroups, c->B_group_stride, c->dstate, c->io_dtype), false},
      {"C", rows_of(c->C, c->C_row_stride, c->ngroups, c->C_group_stride, c->dstate, c->io_dtype), false},
  };
  for (const auto& v : in) {
    const bool same = v.rows.p == out.p && v.rows.bytes == out.bytes &&
                      (rows == 1 || v.rows.stride == out.stride);
    if (in_place && v.elementwise && same) continue;
    if (overlap(out, v.rows, rows))
      return fail(SSU_ERR_INVALID_ARGUMENT, "out must not overlap %s%s", v.name,
                  in_place && v.elementwise ? " (it may be the very same rows)" : "");
  }
  return SSU_OK;
}

static ssu_status table_args(const ssu_slot_table* t, const char* name, Table* out) {
  *out = Table{};
  if (!t || !t->indices) return SSU_OK;
  if (t->numel < 0 || t->steps < 0 || t->seq_stride < 0 || t->step_stride < 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "%s: numel, steps and strides must be >= 0", name);
  const int64_t most = 0x7fffffff;
  if (t->seq_stride > most || t->step_stride > most)
    return fail(SSU_ERR_UNSUPPORTED, "%s: strides must be below 2^31", name);
  *out = Table{t->indices, t->numel, (int)t->seq_stride, (int)t->step_stride,
               (int)(t->steps < most ? t->steps : most)};
  return SSU_OK;
}

static ssu_status check_counts(int64_t nseqs, int64_t rows) {
  if (nseqs < 0 || rows < 0) return fail(SSU_ERR_INVALID_ARGUMENT, "nseqs and rows must be >= 0");
  // the kernels count sequences and rows in 32 bits, a tile or a stride beyond the last
  if (nseqs >= 1LL << 30 || rows > 0x7fffffffLL - 1024)
    return fail(SSU_ERR_UNSUPPORTED, "nseqs must be below 2^30 and rows below 2^31 - 1024");
  return SSU_OK;
}

ssu_status check_packed(int64_t slots, int64_t nseqs, int64_t rows, const void* cu,
                        int64_t dense_steps, const void* na, ssu_dtype meta_dtype,
                        const ssu_slot_table* src, const ssu_slot_table* dst,
                        ssu_dtype index_dtype, Seqs* out) {
  ssu_status st = check_counts(nseqs, rows);
  Seqs a{};
  if (st == SSU_OK) st = table_args(src, "state_batch_indices", &a.src);
  if (st == SSU_OK) st = table_args(dst, "dst_state_batch_indices", &a.dst);
  if (st != SSU_OK) return st;
  if ((a.src.idx || a.dst.idx) && !is_index(index_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "slot tables must be int32 or int64");
  if ((cu || na) && !is_index(meta_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "cu_seqlens / num_accepted_tokens must be int32 or int64");
  if (na && !a.src.idx)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "num_accepted_tokens selects the read slot, so it needs state_batch_indices to "
                "read it from");
  if (!cu && (dense_steps < 1 || dense_steps > 0x7fffffff || nseqs * dense_steps != rows))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "without cu_seqlens %lld rows cannot be split into %lld sequences of %lld steps",
                (long long)rows, (long long)nseqs, (long long)dense_steps);
  if (!a.src.idx && nseqs > slots)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "without state_batch_indices sequence s uses slot s: %lld sequences exceed %lld "
                "slots",
                (long long)nseqs, (long long)slots);
  if (!a.dst.idx) a.dst = a.src;
  a.rows = (int)rows;
  a.n = (int)nseqs;
  a.cu = cu;
  a.steps = cu ? 0 : (int)dense_steps;
  a.na = na;
  a.meta64 = meta_dtype == SSU_I64;
  a.idx64 = index_dtype == SSU_I64;
  *out = a;
  return SSU_OK;
}

ssu_status check_prompts(bool pool, int64_t slots, int64_t nseqs, int64_t rows, const void* cu,
                         ssu_dtype meta_dtype, const void* src, const void* dst,
                         ssu_dtype index_dtype, Seqs* out) {
  ssu_status st = check_counts(nseqs, rows);
  if (st != SSU_OK) return st;
  if (!cu) return fail(SSU_ERR_INVALID_ARGUMENT, "cu_seqlens must not be NULL");
  if (!is_index(meta_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "cu_seqlens must be int32 or int64");
  if ((src || dst) && !is_index(index_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "state_batch_indices must be int32 or int64");
  if ((src || dst) && !pool)
    return fail(SSU_ERR_INVALID_ARGUMENT, "slots need the state pool that they index");
  if (pool && !src && nseqs > slots)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "without state_batch_indices sequence s uses slot s: %lld sequences exceed %lld "
                "slots",
                (long long)nseqs, (long long)slots);
  Seqs a{};
  a.rows = (int)rows;
  a.n = (int)nseqs;
  a.cu = cu;
  a.meta64 = meta_dtype == SSU_I64;
  if (src) a.src = Table{src, nseqs, 1, 1, 1};
  a.dst = dst ? Table{dst, nseqs, 1, 1, 1} : a.src;
  a.idx64 = index_dtype == SSU_I64;
  *out = a;
  return SSU_OK;
}

static ssu_status check_scan(const ssu_scan_params* c, int64_t rows, bool pool_needed,
                             ScanArgs* p) {
  if (!c) return fail(SSU_ERR_INVALID_ARGUMENT, "params must not be NULL");
  if (!is_float(c->state_dtype))
    return fail(SSU_ERR_UNSUPPORTED, "state dtype must be f32, bf16 or f16");
  if (!is_float(c->io_dtype))
    return fail(SSU_ERR_UNSUPPORTED, "x/z/B/C dtype must be f32, bf16 or f16");
  if (c->dt_dtype != c->io_dtype && c->dt_dtype != SSU_F32)
    return fail(SSU_ERR_INVALID_ARGUMENT, "dt must have the x dtype or be f32");
  if (c->out_dtype != c->io_dtype && c->out_dtype != SSU_F32)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out must have the x dtype or be f32");
  if (c->slots < 0 || c->channels < 1 || c->dstate < 1 || c->ngroups < 1)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "state must be [slots, channels, dstate] with positive sizes, got [%lld, %lld, "
                "%lld], ngroups %lld",
                (long long)c->slots, (long long)c->channels, (long long)c->dstate,
                (long long)c->ngroups);
  if (c->channels > (1 << 24)) return fail(SSU_ERR_UNSUPPORTED, "channels must not exceed 2^24");
  if (c->channels % c->ngroups != 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "channels (%lld) must be a multiple of ngroups (%lld)",
                (long long)c->channels, (long long)c->ngroups);
  const int64_t n = c->dstate;
  if (n != 16 && n != 32 && n != 64 && n != 128 && n != 256)
    return fail(SSU_ERR_UNSUPPORTED, "dstate %lld is not one of 16, 32, 64, 128, 256",
                (long long)n);
  if (rows > 0 && (!c->x || !c->out || !c->dt || !c->B || !c->C || !c->A))
    return fail(SSU_ERR_INVALID_ARGUMENT, "x, out, dt, B, C and A must not be NULL");
  if (rows > 1 && c->out_row_stride < c->channels)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out rows overlap: a stride of %lld for %lld channels",
                (long long)c->out_row_stride, (long long)c->channels);
  if (pool_needed && !c->state && c->slots > 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "state must not be NULL");
  if (!aligned(c->state, 16))
    return fail(SSU_ERR_INVALID_ARGUMENT, "state must be 16-byte aligned");
  const int es = size_of(c->io_dtype);
  if (!aligned(c->x, es) || !aligned(c->z, es) || !aligned(c->B, es) || !aligned(c->C, es) ||
      !aligned(c->dt, size_of(c->dt_dtype)) || !aligned(c->out, size_of(c->out_dtype)) ||
      !aligned(c->A, 4) || !aligned(c->D, 4) || !aligned(c->dt_bias, 4))
    return fail(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their element size");
  *p = ScanArgs{};
  p->state = c->state;
  p->state_dtype = c->state_dtype;
  p->slots = c->state ? c->slots : 0;
  p->C = (int)c->channels;
  p->G = (int)c->ngroups;
  p->x = c->x;
  p->x_rs = c->x_row_stride;
  p->z = c->z;
  p->z_rs = c->z_row_stride;
  p->out = c->out;
  p->o_rs = c->out_row_stride;
  p->out_f32 = c->out_dtype == SSU_F32;
  p->dt = c->dt;
  p->dt_rs = c->dt_row_stride;
  p->dt_f32 = c->dt_dtype == SSU_F32;
  p->B = c->B;
  p->B_rs = c->B_row_stride;
  p->B_gs = c->B_group_stride;
  p->Cm = c->C;
  p->C_rs = c->C_row_stride;
  p->C_gs = c->C_group_stride;
  p->bc_vec = aligned(c->B, 16) && aligned(c->C, 16) && c->B_row_stride * es % 16 == 0 &&
              c->C_row_stride * es % 16 == 0 &&
              (c->ngroups == 1 ||
               (c->B_group_stride * es % 16 == 0 && c->C_group_stride * es % 16 == 0));
  // ... and so do a group's channels, at which a CTA may begin
  const int64_t per = c->ngroups > 1 ? c->channels / c->ngroups : 0;
  auto rows_on_16 = [&](const void* ptr, int64_t stride, ssu_dtype d) {
    return aligned(ptr, 16) && stride * size_of(d) % 16 == 0 && per * size_of(d) % 16 == 0;
  };
  p->rows_vec = rows_on_16(c->x, c->x_row_stride, c->io_dtype) &&
                rows_on_16(c->dt, c->dt_row_stride, c->dt_dtype) &&
                rows_on_16(c->out, c->out_row_stride, c->out_dtype) &&
                (!c->z || rows_on_16(c->z, c->z_row_stride, c->io_dtype)) && p->bc_vec;
  p->A = c->A;
  p->A_rs = c->A_row_stride;
  p->a_vec = aligned(c->A, 16) && c->A_row_stride % 4 == 0;
  p->D = c->D;
  p->bias = c->dt_bias;
  p->softplus = c->dt_softplus != 0;
  p->disable = c->disable_state_update != 0;
  p->pad = c->pad_slot_id;
  return SSU_OK;
}

static cudaError_t launch_step(const ssu_scan_params* c, const ScanArgs& p, const Seqs& a, cudaStream_t stream) {
  const int N = (int)c->dstate;
  switch (c->io_dtype) {
    case SSU_F32: return launch_scan_f32(N, p, a, stream);
    case SSU_BF16: return launch_scan_bf16(N, p, a, stream);
    case SSU_F16: return launch_scan_f16(N, p, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

static cudaError_t launch_prompt(const ssu_scan_params* c, const ScanArgs& p, const Seqs& a, cudaStream_t stream) {
  const int N = (int)c->dstate;
  switch (c->io_dtype) {
    case SSU_F32: return launch_prompt_f32(N, p, a, stream);
    case SSU_BF16: return launch_prompt_bf16(N, p, a, stream);
    case SSU_F16: return launch_prompt_f16(N, p, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace layer

#pragma GCC visibility push(default)
extern "C" {

ssu_status ssu_scan_update(const ssu_scan_params* c, int64_t nseqs, int64_t rows,
                           const void* cu_seqlens, int64_t dense_steps,
                           const void* num_accepted_tokens, ssu_dtype meta_dtype,
                           const ssu_slot_table* src, const ssu_slot_table* dst,
                           ssu_dtype index_dtype, struct CUstream_st* stream) {
  using namespace layer;
  ScanArgs p;
  Seqs a;
  ssu_status st = check_scan(c, rows, true, &p);
  if (st == SSU_OK)
    st = check_packed(c->slots, nseqs, rows, cu_seqlens, dense_steps, num_accepted_tokens,
                      meta_dtype, src, dst, index_dtype, &a);
  if (st == SSU_OK) st = check_scan_out(c, rows, true);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  return launched(launch_step(c, p, a, (cudaStream_t)stream));
}

ssu_status ssu_scan_fwd_varlen(const ssu_scan_params* c, int64_t nseqs, int64_t rows,
                               const void* cu_seqlens, ssu_dtype meta_dtype,
                               const void* state_batch_indices,
                               const void* dst_state_batch_indices, ssu_dtype index_dtype,
                               const uint8_t* has_initial_state, struct CUstream_st* stream) {
  using namespace layer;
  ScanArgs p;
  Seqs a;
  ssu_status st = check_scan(c, rows, false, &p);
  if (st == SSU_OK)
    st = check_prompts(c->state != nullptr, c->slots, nseqs, rows, cu_seqlens, meta_dtype,
                       state_batch_indices, dst_state_batch_indices, index_dtype, &a);
  if (st == SSU_OK) st = check_scan_out(c, rows, false);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  p.has_init = has_initial_state;
  return launched(launch_prompt(c, p, a, (cudaStream_t)stream));
}

}  // extern "C"
#pragma GCC visibility pop
