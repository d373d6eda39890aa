// drafts.cu -- verification of drafted tokens: a sequence's drafts are taken,
// in order, while u_j q_j < p_j (p the target's probability of draft j, q the
// one that it was drawn with, u a given number in [0, 1)), and the next token is
// drawn from what is left: max(p - q, 0) where a draft was turned down, p after
// the last.  So the tokens are distributed as the target's own.
//
// Decisions are exact: the product of two fp32 numbers is a 64-bit one.  The
// draw inverts the cumulative sum of the weights round(r 2^44), r what is left
// of a token's probability, and integers add up to the same sum in any order: the
// same inputs give the same token however the row is split.
#include <cooperative_groups.h>

#include "layer_common.cuh"

namespace drafts {
using namespace layer;
namespace cg = cooperative_groups;

struct Args {
  const void* p;
  int64_t p_rs;
  int rows, V;
  const void* q;  // nullptr: each draft was certain
  int64_t q_ss, q_ts;
  const void* drafts;
  int64_t d_ss;
  int tok64;
  int n, K;
  const float* u;
  int64_t u_ss;
  const void* cu;
  int meta64;
  const uint8_t* greedy;
  void* out;
  int64_t o_ss;
  void* count;
  int count64;
  int p_vec, q_vec;  // every row of p (q) starts on a boundary of four elements
};

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kVec = 4;

// (value, index) of the largest value; the lowest index of equal ones; NaN never
struct Best {
  float v;
  int i;
  __device__ __forceinline__ void take(float w, int j) {
    if (w > v || (w == v && j < i)) v = w, i = j;
  }
};

struct Shared {
  unsigned long long sum[kWarps];  // weights of each warp's share
  Best best[kWarps];
  // of the CTA, read by the others of its cluster
  unsigned long long total;
  Best top[2];
};

// What is left of four consecutive probabilities.
template <class T>
struct Row {
  const T* p;
  const T* q;  // nullptr: nothing is taken off, but for token `drop`
  int drop;
  bool p_vec, q_vec;

  __device__ __forceinline__ void load(int i, int end, float* r) const {
    if (i + kVec <= end) {
      load_floats<T, kVec>(p + i, p_vec, r);
      if (q) {
        float s[kVec];
        load_floats<T, kVec>(q + i, q_vec, s);
#pragma unroll
        for (int e = 0; e < kVec; ++e) r[e] -= s[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        r[e] = i + e < end ? to_f(p[i + e]) : 0.0f;
        if (q && i + e < end) r[e] -= to_f(q[i + e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (i + e == drop) r[e] = 0.0f;
  }
};

// in units of 2^-44; NaN and what is below zero weigh nothing
__device__ __forceinline__ unsigned long long weight(float r) {
  return (unsigned long long)__float2ll_rn(fminf(fmaxf(r, 0.0f), 1.0f) * 0x1p44f);
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void store_int(void* p, int64_t i, int is64, int64_t v) {
  if (is64) static_cast<int64_t*>(p)[i] = v;
  else static_cast<int32_t*>(p)[i] = (int32_t)v;
}

// A cluster per sequence; its CTAs, and their warps, have consecutive shares of
// the vocabulary.
template <class T>
__global__ void __launch_bounds__(kThreads) drafts_verify_kernel(const Args a) {
  __shared__ Shared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int s = blockIdx.y, rank = cluster.block_rank(), ctas = cluster.num_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool writer = rank == 0 && threadIdx.x == 0;
  const int r0 = a.cu ? clamped(load_int(a.cu, s, a.meta64), a.rows) : s * (a.K + 1);
  const int r1 = a.cu ? clamped(load_int(a.cu, s + 1, a.meta64), a.rows) : r0 + a.K + 1;
  const int n = min(r1 - r0 - 1, a.K);  // drafts; the same in the whole cluster

  int count = 0;
  int64_t token = -1;
  if (n >= 0) {
    const bool greedy = a.greedy && a.greedy[s];
    // the warp's share [i0, i1) of the vocabulary
    const int share = ((a.V + ctas * kWarps - 1) / (ctas * kWarps) + kVec - 1) / kVec * kVec;
    const int64_t at = (int64_t)share * (rank * kWarps + warp);
    const int i0 = (int)min(at, (int64_t)a.V), i1 = (int)min(at + share, (int64_t)a.V);
    auto row_of = [&](int j) { return static_cast<const T*>(a.p) + (int64_t)(r0 + j) * a.p_rs; };
    auto draft = [&](int j) { return load_int(a.drafts, s * a.d_ss + j, a.tok64); };

    if (greedy) {
      for (int j = 0;; ++j) {
        const T* row = row_of(j);
        Best b{-INFINITY, 0x7fffffff};
        for (int i = i0 + lane * kVec; i < i1; i += 32 * kVec) {
          float r[kVec];
          if (i + kVec <= i1) load_floats<T, kVec>(row + i, a.p_vec, r);
          else
            for (int e = 0; e < kVec; ++e) r[e] = i + e < i1 ? to_f(row[i + e]) : NAN;
#pragma unroll
          for (int e = 0; e < kVec; ++e) b.take(r[e], i + e);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          b.take(__shfl_xor_sync(0xffffffffu, b.v, o), __shfl_xor_sync(0xffffffffu, b.i, o));
        if (lane == 0) sm.best[warp] = b;
        __syncthreads();
        if (threadIdx.x == 0) {
          for (int w = 1; w < kWarps; ++w) b.take(sm.best[w].v, sm.best[w].i);
          sm.top[j & 1] = b;
        }
        cluster.sync();
        Best top{-INFINITY, 0x7fffffff};
        for (int c = 0; c < ctas; ++c) {
          const Best o = *cluster.map_shared_rank(&sm.top[j & 1], c);
          top.take(o.v, o.i);
        }
        token = top.i < a.V ? top.i : -1;
        if (j == n || token < 0 || draft(j) != token) break;
        ++count;
      }
    } else {
      // the first draft that is turned down, by every warp for itself
      for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        bool taken = false;
        if (j < n) {
          const int64_t d = draft(j);
          if (d >= 0 && d < a.V) {
            const double p = to_f(row_of(j)[d]);
            const double q =
                a.q ? to_f(static_cast<const T*>(a.q)[s * a.q_ss + j * a.q_ts + d]) : 1.0f;
            taken = (double)a.u[s * a.u_ss + j] * q < p;
          }
        }
        const unsigned no = __ballot_sync(0xffffffffu, !taken);
        count = j0 + (no ? __ffs(no) - 1 : 32);
        if (no) break;
      }
      count = min(count, n);
      Row<T> row{row_of(count), nullptr, -1, a.p_vec != 0, a.q_vec != 0};
      if (count < n) {
        if (a.q) row.q = static_cast<const T*>(a.q) + s * a.q_ss + count * a.q_ts;
        else {
          const int64_t d = draft(count);
          row.drop = d >= 0 && d < a.V ? (int)d : -1;
        }
      }
      const float u = a.u[s * a.u_ss + a.K];
      // a second time, from the whole row, where nothing is left of it
      for (int pass = 0; pass < 2; ++pass) {
        unsigned long long sum = 0;
        for (int i = i0 + lane * kVec; i < i1; i += 32 * kVec) {
          float r[kVec];
          row.load(i, i1, r);
#pragma unroll
          for (int e = 0; e < kVec; ++e) sum += weight(r[e]);
        }
        sum = warp_sum(sum);
        if (lane == 0) sm.sum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
          unsigned long long t = 0;
          for (int w = 0; w < kWarps; ++w) t += sm.sum[w];
          sm.total = t;
        }
        cluster.sync();
        unsigned long long total = 0, before = 0;  // before: of the lower ranks
        for (int c = 0; c < ctas; ++c) {
          if (c == rank) before = total;
          total += *cluster.map_shared_rank(&sm.total, c);
        }
        for (int w = 0; w < warp; ++w) before += sm.sum[w];
        if (total > 0) {
          // floor(u total), below total
          const double m = floor(fmin(fmax((double)u, 0.0), 1.0) * (double)total);
          unsigned long long mark = m < 9.2e18 ? (unsigned long long)m : total - 1;
          mark = mark < total ? mark : total - 1;
          // the warp whose share holds it finds the token
          if (mark >= before && mark - before < sum) {
            unsigned long long run = before;
            for (int base = i0; base < i1; base += 32 * kVec) {
              const int i = base + lane * kVec;
              float r[kVec];
              unsigned long long w[kVec], mine = 0;
              if (i < i1) row.load(i, i1, r);
#pragma unroll
              for (int e = 0; e < kVec; ++e) {
                w[e] = i < i1 ? weight(r[e]) : 0;
                mine += w[e];
              }
              unsigned long long inc = mine;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
              }
              const unsigned long long all = __shfl_sync(0xffffffffu, inc, 31);
              if (mark < run + all) {
                unsigned long long c = run + inc - mine;
                if (mark >= c && mark < c + mine) {
                  int e = 0;
                  while (mark >= c + w[e]) c += w[e++];
                  store_int(a.out, s * a.o_ss + count, a.tok64, i + e);
                }
                break;
              }
              run += all;
            }
          }
          token = -2;  // another thread writes it
          break;
        }
        row.q = nullptr;
        row.drop = -1;
        cluster.sync();  // sm.total is read before it is written again
      }
    }
    ++count;
  }
  if (rank == 0) {
    for (int j = threadIdx.x; j <= a.K; j += kThreads) {
      if (j == count - 1) {
        if (token != -2) store_int(a.out, s * a.o_ss + j, a.tok64, token);
      } else {
        store_int(a.out, s * a.o_ss + j, a.tok64,
                  j < count ? load_int(a.drafts, s * a.d_ss + j, a.tok64) : -1);
      }
    }
  }
  if (writer) store_int(a.count, s, a.count64, count);
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

template <class T>
static cudaError_t launch(const Args& a, cudaStream_t stream) {
  int ctas = 1;
  while (ctas < 8 && a.V > ctas * 16384) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)a.n);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, drafts_verify_kernel<T>, a);
}

static ssu_status verify(const ssu_drafts_params* c, cudaStream_t stream) {
  if (!c) return fail(SSU_ERR_INVALID_ARGUMENT, "params must not be NULL");
  if (!is_float(c->probs_dtype))
    return fail(SSU_ERR_UNSUPPORTED, "probabilities must be f32, bf16 or f16");
  if (!is_index(c->token_dtype) || !is_index(c->count_dtype) ||
      (c->cu_seqlens && !is_index(c->meta_dtype)))
    return fail(SSU_ERR_INVALID_ARGUMENT, "tokens, counts and cu_seqlens must be int32 or int64");
  if (c->rows < 0 || c->nseqs < 0 || c->drafts < 0 || c->vocab < 1)
    return fail(SSU_ERR_INVALID_ARGUMENT, "rows, nseqs and drafts must be >= 0, vocab positive");
  // 2^19 weights of at most 2^44 each add up within 64 bits; the grid's second dimension
  if (c->vocab > (1 << 19) || c->nseqs > 65535 || c->drafts > 4096 || c->rows > 0x7fffffffLL - 1)
    return fail(SSU_ERR_UNSUPPORTED,
                "at most 2^19 tokens in the vocabulary, 65535 sequences, 4096 drafts a sequence "
                "and 2^31 - 2 rows");
  if (!c->cu_seqlens && c->nseqs * (c->drafts + 1) != c->rows)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "without cu_seqlens %lld rows cannot be split into %lld sequences of %lld",
                (long long)c->rows, (long long)c->nseqs, (long long)(c->drafts + 1));
  if (c->nseqs > 0 && (!c->out || !c->num_accepted || !c->uniform ||
                       (c->drafts > 0 && !c->draft_tokens) || (c->rows > 0 && !c->target_probs)))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "target_probs, draft_tokens, uniform, out and num_accepted must not be NULL");
  if (c->nseqs > 1 && c->out_seq_stride < c->drafts + 1)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out's rows overlap");
  const int es = size_of(c->probs_dtype), ts = size_of(c->token_dtype);
  if (!aligned(c->target_probs, es) || !aligned(c->draft_probs, es) ||
      !aligned(c->draft_tokens, ts) || !aligned(c->out, ts) || !aligned(c->uniform, 4) ||
      !aligned(c->num_accepted, size_of(c->count_dtype)) ||
      (c->cu_seqlens && !aligned(c->cu_seqlens, size_of(c->meta_dtype))))
    return fail(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their element size");
  const Rows out = rows_of(c->out, c->out_seq_stride, c->drafts + 1, c->token_dtype);
  if (overlap(out, rows_of(c->draft_tokens, c->draft_tokens_seq_stride, c->drafts, c->token_dtype),
              c->nseqs) ||
      overlap(out, rows_of(c->uniform, c->uniform_seq_stride, c->drafts + 1, SSU_F32), c->nseqs) ||
      overlap(out, rows_of(c->num_accepted, 1, 1, c->count_dtype), c->nseqs))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "out must not overlap draft_tokens, uniform or num_accepted");
  if (c->nseqs == 0) return ok();
  Args a{};
  a.p = c->target_probs;
  a.p_rs = c->target_row_stride;
  a.rows = (int)c->rows;
  a.V = (int)c->vocab;
  a.q = c->draft_probs;
  a.q_ss = c->draft_seq_stride;
  a.q_ts = c->draft_step_stride;
  a.drafts = c->draft_tokens;
  a.d_ss = c->draft_tokens_seq_stride;
  a.tok64 = c->token_dtype == SSU_I64;
  a.n = (int)c->nseqs;
  a.K = (int)c->drafts;
  a.u = c->uniform;
  a.u_ss = c->uniform_seq_stride;
  a.cu = c->cu_seqlens;
  a.meta64 = c->meta_dtype == SSU_I64;
  a.greedy = c->greedy;
  a.out = c->out;
  a.o_ss = c->out_seq_stride;
  a.count = c->num_accepted;
  a.count64 = c->count_dtype == SSU_I64;
  a.p_vec = aligned(c->target_probs, kVec * es) && c->target_row_stride % kVec == 0;
  a.q_vec = c->draft_probs && aligned(c->draft_probs, kVec * es) &&
            c->draft_seq_stride % kVec == 0 && c->draft_step_stride % kVec == 0;
  switch (c->probs_dtype) {
    case SSU_F32: return launched(launch<float>(a, stream));
    case SSU_BF16: return launched(launch<__nv_bfloat16>(a, stream));
    default: return launched(launch<__half>(a, stream));
  }
}

}  // namespace drafts

#pragma GCC visibility push(default)
extern "C" {

ssu_status ssu_drafts_verify(const ssu_drafts_params* c, struct CUstream_st* stream) {
  return drafts::verify(c, (cudaStream_t)stream);
}

}  // extern "C"
#pragma GCC visibility pop
