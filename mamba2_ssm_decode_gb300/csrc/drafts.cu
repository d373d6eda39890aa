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
//
// A chain of five loads and three meetings bounds one sequence (50288 tokens: 8.2 us),
// and in 3.4 waves of CTAs a batch of 256 as well (128257 tokens, 230 MB: 63 us).
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
};

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kEach = 16;           // elements a lane has under way at once
constexpr int kStep = 32 * kEach;   // ... a warp

constexpr int kRows = 4;            // rows of a greedy sequence that are looked at together

// (value, index) of the largest value; the lowest index of equal ones; NaN never
struct Best {
  float v;
  int i;
  __device__ __forceinline__ void take(float w, int j) {
    if (w > v || (w == v && j < i)) v = w, i = j;
  }
  // a number that is larger for what is better, above 0; 0 where nothing was taken
  __device__ __forceinline__ unsigned long long key() const {
    if (i == 0x7fffffff) return 0;
    const uint32_t b = __float_as_uint(v + 0.0f);  // one zero
    return (unsigned long long)(b >> 31 ? ~b : b | 0x80000000u) << 32 | (0x7fffffffu - (uint32_t)i);
  }
};

struct Shared {
  unsigned long long sum[kWarps];  // weights of each warp's share
  unsigned long long best[kRows][kWarps];  // ... best of each row, as Best::key
  // of the CTA, read by the others of its cluster
  unsigned long long total;
  unsigned long long top[2][kRows];
};

// What is left of kStep consecutive probabilities, kEach a lane.  VEC: every row
// starts on a boundary of four elements, and a lane takes them four at a time; else
// one at a time, which leaves a warp's accesses as long: rows of an odd vocabulary
// start anywhere.
template <class T, bool VEC>
struct Row {
  static constexpr int E = VEC ? 4 : 1, U = kEach / E;
  const T* p;
  const T* q;  // nullptr: nothing is taken off, but for token `drop`
  int drop;

  // element e of part u of the kStep from `base` on
  static __device__ __forceinline__ int place(int base, int u, int e) {
    return base + (u * 32 + (threadIdx.x & 31)) * E + e;
  }
  static __device__ __forceinline__ void read(const T* row, int base, int end, float none,
                                              float (&r)[kEach]) {
    if (base + kStep <= end) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_floats<T, E>(row + place(base, u, 0), true, r + u * E);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int i = place(base, u, e);
          r[u * E + e] = i < end ? to_f(row[i]) : none;
        }
    }
  }
  // zeros from `end` on
  __device__ __forceinline__ void load(int base, int end, float (&r)[kEach]) const {
    read(p, base, end, 0.0f, r);
    if (q) {
      float s[kEach];
      read(q, base, end, 0.0f, s);
#pragma unroll
      for (int i = 0; i < kEach; ++i) r[i] -= s[i];
    }
    if (drop >= base && drop < base + kStep) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (place(base, i / E, i % E) == drop) r[i] = 0.0f;
    }
  }
};

// Weights in units of 2^-44; NaN and what is below zero weigh nothing.  A weight is
// h 2^22 + l, h the nearest integer of r 2^22 and l the one of what that leaves times
// 2^22: sums of fp32 numbers and a power of two, whose low bits are the integers.
// Conversions to 64-bit integers took 26 of 92 us (256 sequences, 128257 tokens).
struct Weights {
  uint32_t h = 0, l = 0;
  int n = 0;
  __device__ __forceinline__ void add(float r) {  // at most 2^9 times
    const float t = fminf(fmaxf(r, 0.0f), 1.0f) * 0x1p22f;
    const float a = t + 0x1p23f;
    const float b = fmaf(t - (a - 0x1p23f), 0x1p22f, 0x1.8p23f);
    h += __float_as_uint(a);
    l += __float_as_uint(b);
    ++n;
  }
  __device__ __forceinline__ unsigned long long sum() const {
    return ((unsigned long long)(h - (uint32_t)n * 0x4b000000u) << 22) +
           (long long)(int32_t)(l - (uint32_t)n * 0x4b400000u);
  }
};

__device__ __forceinline__ unsigned long long weight(float r) {
  Weights w;
  w.add(r);
  return w.sum();
}

// floor(u W), in whole numbers (u is m 2^-s with m below 2^24): of 68 bits fp64 has 53, and may
// round up to the whole number that is the next token's.  0 for NaN and below 0, W - 1 from 1 on.
__device__ __forceinline__ unsigned long long mark_of(float u, unsigned long long W) {
  if (!(u > 0.0f)) return 0;
  if (u >= 1.0f) return W - 1;
  const uint32_t bits = __float_as_uint(u), e = bits >> 23;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int s = 150 - (int)(e ? e : 1u);  // 24 to 149
  const unsigned long long low = W * m, high = __umul64hi(W, m);
  return s < 64 ? high << (64 - s) | low >> s : s < 128 ? high >> (s - 64) : 0;
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
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) drafts_verify_kernel(const Args a) {
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
    const int share = ((a.V + ctas * kWarps - 1) / (ctas * kWarps) + kStep - 1) / kStep * kStep;
    const int64_t at = (int64_t)share * (rank * kWarps + warp);
    const int i0 = (int)min(at, (int64_t)a.V), i1 = (int)min(at + share, (int64_t)a.V);
    auto row_of = [&](int j) { return static_cast<const T*>(a.p) + (int64_t)(r0 + j) * a.p_rs; };
    auto draft = [&](int j) { return load_int(a.drafts, s * a.d_ss + j, a.tok64); };

    if (greedy) {
      // Blocks of kStep of the next kRows rows, dealt to all of the cluster's warps: row
      // after row would wait for a meeting of the CTAs each time.
      const int blocks = (a.V + kStep - 1) / kStep;
      for (int j0 = 0, odd = 0;; j0 += kRows, odd ^= 1) {
        const int rows = min(kRows, n + 1 - j0);
        int id = rank * kWarps + warp;
        for (int j = 0; j < rows; ++j) {
          using R = Row<T, VEC>;
          Best b{-INFINITY, 0x7fffffff};
          const T* row = row_of(j0 + j);
          for (; id < (j + 1) * blocks; id += ctas * kWarps) {
            float r[kEach];
            const int base = (id - j * blocks) * kStep;
            R::read(row, base, a.V, NAN, r);
#pragma unroll
            for (int i = 0; i < kEach; ++i) b.take(r[i], R::place(base, i / R::E, i % R::E));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            b.take(__shfl_xor_sync(0xffffffffu, b.v, o), __shfl_xor_sync(0xffffffffu, b.i, o));
          if (lane == 0) sm.best[j][warp] = b.key();
        }
        __syncthreads();
        static_assert(kRows <= kWarps && kWarps <= 32, "a warp a row");
        if (warp < rows) {
          unsigned long long b = lane < kWarps ? sm.best[warp][lane] : 0;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long v = __shfl_xor_sync(0xffffffffu, b, o);
            b = v > b ? v : b;
          }
          if (lane == 0) sm.top[odd][warp] = b;
        }
        cluster.sync();
        bool more = true;
        for (int j = 0; j < rows && more; ++j) {
          unsigned long long best = 0;
          for (int c = 0; c < ctas; ++c) {
            const unsigned long long b = *cluster.map_shared_rank(&sm.top[odd][j], c);
            best = b > best ? b : best;
          }
          token = best ? (int64_t)(0x7fffffffu - (uint32_t)best) : -1;
          more = j0 + j < n && token >= 0 && draft(j0 + j) == token;
          count += more;
        }
        if (!more) break;
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
      Row<T, VEC> row{row_of(count), nullptr, -1};
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
        for (int base = i0; base < i1; base += kStep) {
          float r[kEach];
          row.load(base, i1, r);
          Weights w;
#pragma unroll
          for (int i = 0; i < kEach; ++i) w.add(r[i]);
          sum += w.sum();
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
          const unsigned long long mark = mark_of(u, total);
          // the warp whose share holds it finds the token
          if (mark >= before && mark - before < sum) {
            unsigned long long run = before;
            for (int base = i0; base < i1; base += kStep) {
              constexpr int E = Row<T, VEC>::E;
              float r[kEach];
              row.load(base, i1, r);
              Weights w;
#pragma unroll
              for (int i = 0; i < kEach; ++i) w.add(r[i]);
              unsigned long long mine = w.sum();
              const unsigned long long here = warp_sum(mine);
              if (mark >= run + here) {
                run += here;
                continue;
              }
#pragma unroll
              for (int u = 0; u < kEach / E; ++u) {
                mine = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) mine += weight(r[u * E + e]);
                unsigned long long inc = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                  const unsigned long long v = __shfl_up_sync(0xffffffffu, inc, o);
                  if (lane >= o) inc += v;
                }
                unsigned long long c = run + inc - mine;
                if (mark >= c && mark < c + mine) {
#pragma unroll
                  for (int e = 0; e < E; ++e) {
                    const unsigned long long w = weight(r[u * E + e]);
                    if (mark >= c && mark < c + w)
                      store_int(a.out, s * a.o_ss + count, a.tok64, row.place(base, u, e));
                    c += w;
                  }
                }
                run += __shfl_sync(0xffffffffu, inc, 31);
              }
              break;
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

template <class T, bool VEC>
static cudaError_t launch(const Args& a, cudaStream_t stream) {
  // Twice as many CTAs while a warp has more than one step and all sequences together have
  // fewer than four CTAs an SM (so below eight in the end): for one sequence of 50288 tokens
  // 1, 2, 4 and 8 take 25, 12, 9.6 and 8.2 us, for 256 of 128257 2, 4 and 8 take 65, 66 and
  // 87 us.
  int ctas = 1;
  while (ctas < 8 && a.V > ctas * kWarps * kStep && (int64_t)a.n * ctas < 4LL * ssu::sm_count())
    ctas *= 2;
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
  return cudaLaunchKernelEx(&cfg, drafts_verify_kernel<T, VEC>, a);
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
      overlap(out, rows_of(c->uniform, c->uniform_seq_stride, c->drafts + 1, SSU_F32), c->nseqs))
    return fail(SSU_ERR_INVALID_ARGUMENT, "out must not overlap draft_tokens or uniform");
  // the results against each other and the other operands, which other sequences' CTAs still
  // read: the bytes from an operand's first to its last
  struct Span {
    const char* name;
    const void* p;
    int64_t bytes;
  };
  auto span = [](const char* name, const void* p, int64_t rows, int64_t stride, int64_t n, int64_t s) {
    return Span{name, p, rows > 0 && n > 0 && p ? ((rows - 1) * stride + n) * s : 0};
  };
  const int64_t S = c->nseqs, K = c->drafts;
  const Span all[] = {
      span("out", c->out, S, c->out_seq_stride, K + 1, ts),
      span("num_accepted", c->num_accepted, 1, 0, S, size_of(c->count_dtype)),
      span("target_probs", c->target_probs, c->rows, c->target_row_stride, c->vocab, es),
      span("draft_probs", c->draft_probs, S, c->draft_seq_stride,
           K > 0 ? (K - 1) * c->draft_step_stride + c->vocab : 0, es),
      span("cu_seqlens", c->cu_seqlens, 1, 0, S + 1, c->cu_seqlens ? size_of(c->meta_dtype) : 0),
      span("greedy", c->greedy, 1, 0, S, 1),
      span("draft_tokens", c->draft_tokens, S, c->draft_tokens_seq_stride, K, ts),
      span("uniform", c->uniform, S, c->uniform_seq_stride, K + 1, 4)};
  constexpr int kAll = (int)(sizeof(all) / sizeof(all[0]));
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < (i ? kAll : kAll - 2); ++j)  // out's rows may lie beside the last two's
      if (all[i].bytes > 0 && all[j].bytes > 0 &&
          overlap(Rows{all[i].p, 0, all[i].bytes}, Rows{all[j].p, 0, all[j].bytes}, 1))
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s must not overlap %s", all[i].name, all[j].name);
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
  auto fours = [&](const void* p, int64_t stride, int64_t more) {
    return aligned(p, 4 * es) && stride % 4 == 0 && more % 4 == 0;
  };
  const bool vec = fours(c->target_probs, c->target_row_stride, 0) &&
                   (!c->draft_probs ||
                    fours(c->draft_probs, c->draft_seq_stride, c->draft_step_stride));
  switch (c->probs_dtype) {
    case SSU_F32: return launched((vec ? launch<float, true> : launch<float, false>)(a, stream));
    case SSU_BF16:
      return launched((vec ? launch<__nv_bfloat16, true> : launch<__nv_bfloat16, false>)(a, stream));
    default: return launched((vec ? launch<__half, true> : launch<__half, false>)(a, stream));
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
