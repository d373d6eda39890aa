// linattn_prompt.cuh -- linear attention (linattn.cuh) over prompts, on the fifth-
// generation tensor cores: 16-bit q, k and v, dk and dv 64 or 128.
//
// A chunk is 64 tokens.  With a_t the running sum of the log decays over the
// chunk, a_C its last, and S the state that enters it (dv x dk):
//   P[t][s] = scale e^(a_t - a_s) q_t . k_s          for s <= t, else 0
//   o_t     = sum_s P[t][s] v_s + scale e^(a_t) S q_t
//   S      <- e^(a_C) S + sum_s (e^(a_C - a_s) v_s) k_s^T
// Four products, all with 64 tokens as one side, so that every operand in
// shared memory is a tile as it lies in global memory:
//   scores (t x s)   = Q K^T                  A, B: Q and K, rows of dk
//   o1^T   (dv x t)  = V^T P^T                A: V, dv within a row; B: P, rows of s
//   o2^T   (dv x t)  = S Q^T                  A: S, in tensor memory; B: Q
//   D      (dv x dk) = (w V)^T K              A: w V; B: K, both along the tokens
// S itself stays in fp32 registers of the threads that own its rows in tensor
// memory, so a chunk costs it one read of D and no write.
//
// P, S and w V are computed, not given, and enter the products as 16-bit parts
// that add up to them: P and S as a high part and a remainder (to 2^-17 of each
// with bf16, 2^-22 with fp16, where one part alone would be as far off as the
// output's own rounding), w V as three of bf16 where the state is kept in 32 bits
// (2^-26; two leave 2^-17, which shows in it), else two.
//
// One CTA of 20 warps works on a chunk of one head at a time, chunks of a
// sequence in order: 4 warps turn scores into P, 4 write outputs, 8 update S and
// weigh V (each owns 32 lanes of tensor memory, so the tiles' rows), one issues
// the products, three load Q, K, V and sum the decays, three chunks ahead.
// Items -- a sequence's, or a piece's, chunks of one head -- are handed out by a
// counter, longest first.  A sequence of more chunks than every SM's fair share
// is cut into pieces: a first launch computes what each piece adds to the state
// (the fourth product alone) and its decay, and a piece's item then starts by
// adding up the pieces before it.
#pragma once

#include "linattn.cuh"
#include "ssd_tc.cuh"
#include "ssu_bulk.cuh"

namespace linattn {
namespace tc = ssd::tc;
using ssu::mbar_arrive;
using ssu::mbar_init;
using ssu::mbar_test;
using ssu::smem_addr;

constexpr int kC = 64;             // tokens of a chunk
constexpr int kCol = kC * 16 + 16;  // bytes between the 16-byte columns of a tile: 16 of padding
                                    // put the pieces of a row on banks of their own
constexpr int kStages = 3;
constexpr unsigned kErrMma = SSU_DEVICE_ERR_MMA_TIMEOUT;

// A piece of a sequence, as the plan lists it.
struct Piece {
  int seq, r0, len;  // rows [r0, r0 + len)
  int j, of;         // piece j of `of`
  int base;          // of > 1: the sequence's first entry in the workspace's states
};

// What the plan leaves in the workspace.
struct Header {
  int next[2];   // items handed out: of the first launch, of the second
  int count[2];  // pieces of each
};

struct PromptArgs {
  Args p;
  Seqs a;
  Header* head;
  Piece* pieces[2];
  float* decay;  // [entries][H]: what a piece decays the state by
  float* state;  // [entries][H][dv * dk], in the threads' order
  int fair, cut;  // chunks: more than `fair` of them are cut into pieces of about `cut`
  int entries;
  unsigned* err;
};

// ---------------------------------------------------------------------------
// plan: the pieces, longest first
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kBuckets = 64;

struct Cut {
  int r0, len, chunks, pieces, each;  // each: chunks of a piece (the last may have fewer)
  __device__ __forceinline__ Cut(const PromptArgs& g, int s, bool split) {
    r0 = clamped(load_int(g.a.cu, s, g.a.meta64), g.a.rows);
    const int end = clamped(load_int(g.a.cu, s + 1, g.a.meta64), g.a.rows);
    len = end > r0 ? end - r0 : 0;
    chunks = (len + kC - 1) / kC;
    pieces = split && chunks > g.fair ? (chunks + g.cut - 1) / g.cut : chunks > 0;
    each = pieces ? (chunks + pieces - 1) / pieces : 0;
    if (pieces) pieces = (chunks + each - 1) / each;
  }
  // the longest first
  __device__ __forceinline__ int bucket(const PromptArgs& g, int j) const {
    const int n = j + 1 < pieces ? each : chunks - j * each;
    const int most = g.fair > g.cut ? g.fair : g.cut;
    const int64_t b = (int64_t)n * (kBuckets - 1) / most;
    return kBuckets - 1 - (b < kBuckets ? (int)b : kBuckets - 1);
  }
};

static __global__ void __launch_bounds__(kPlanThreads) linattn_plan_kernel(const PromptArgs g) {
  __shared__ int at[2][kBuckets];
  __shared__ int used, want;
  const int tid = threadIdx.x;
  if (tid < kBuckets) at[0][tid] = at[1][tid] = 0;
  if (tid == 0) used = want = 0;
  __syncthreads();
  for (int s = tid; s < g.a.n; s += kPlanThreads) {
    const Cut c(g, s, true);
    if (c.pieces > 1) atomicAdd(&want, c.pieces);
  }
  __syncthreads();
  // starts that do not ascend could ask for more than the workspace has room for
  const bool split = want <= g.entries;
  for (int s = tid; s < g.a.n; s += kPlanThreads) {
    const Cut c(g, s, split);
    for (int j = 0; j < c.pieces; ++j) {
      const int b = c.bucket(g, j);
      atomicAdd(&at[1][b], 1);
      if (j + 1 < c.pieces) atomicAdd(&at[0][b], 1);
    }
  }
  __syncthreads();
  if (tid < 2) {
    int sum = 0;
    for (int b = 0; b < kBuckets; ++b) {
      const int n = at[tid][b];
      at[tid][b] = sum;
      sum += n;
    }
    g.head->count[tid] = sum;
    g.head->next[tid] = 0;
  }
  __syncthreads();
  for (int s = tid; s < g.a.n; s += kPlanThreads) {
    const Cut c(g, s, split);
    int base = 0;
    if (c.pieces > 1) base = atomicAdd(&used, c.pieces);
    for (int j = 0; j < c.pieces; ++j) {
      const int first = j * c.each * kC;
      const Piece piece{s, c.r0 + first, min(c.len - first, c.each * kC), j, c.pieces, base};
      const int b = c.bucket(g, j);
      g.pieces[1][atomicAdd(&at[1][b], 1)] = piece;
      if (j + 1 < c.pieces) g.pieces[0][atomicAdd(&at[0][b], 1)] = piece;
    }
  }
}

// ---------------------------------------------------------------------------
// the chunks
// ---------------------------------------------------------------------------
// A chunk in a stage.
struct Chunk {
  int h, r0, rows;    // head, first row, rows there are
  int first, last;    // of its item
  int stop;           // no chunk: there are no more
  Piece piece;
};

struct Tables {        // of a chunk, in units of log2
  float a[kC];         // a_t
  float ea[kC];        // scale e^(a_t)
  float w[kC];         // e^(a_C - a_s); 0 behind the last row
  float keep, add;     // e^(a_C) = keep + add, keep 0 or 1
  float decay;         // e^(a_C)
};

template <int DV, int DK>
struct Sizes {
  static constexpr int kQ = DK / 8 * kCol, kV = DV / 8 * kCol, kP = kC / 8 * kCol;
  static constexpr int kStage = 2 * kQ + kV;
  static constexpr int kCols = 512;  // of tensor memory
  // columns: D, o1, o2, scores (two), S (high parts, remainders)
  static constexpr int kD = 0, kO1 = 128, kO2 = 192, kSc = 256, kS = 384;
};

template <int DV, int DK, int PARTS>
struct PromptSmem {
  using Z = Sizes<DV, DK>;
  unsigned char stage[kStages][Z::kStage];
  unsigned char wv[PARTS][Z::kV];
  unsigned char p[2][Z::kP];
  Tables tab[kStages];
  Chunk chunk[kStages];
  float row_max[2][128];    // fp16: the largest value of half a row of S
  float row_scale[2][128];  // fp16: what a row of S was divided by
  int bad[2][128];          // the first token of the chunk whose v is not finite
  int any_bad[2];
  uint64_t full[kStages], empty[kStages], sc_full[2];
  uint64_t p_ready, p_free, o_full, o_free, s_ready, v_ready, d_full;
  uint64_t loaders, state_warps, out_warps, fin;  // warps of a role meet; the last product
  uint32_t tmem;
  int abort;
  int item;
};

constexpr int kPromptThreads = 640;
constexpr int kLoaders = 96;

__device__ __forceinline__ void st_tmem8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// As tc::mma, with A in tensor memory.
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Waits for a phase; gives up after two seconds, or when another thread did.
template <class SM>
__device__ __forceinline__ bool wait(SM& sm, unsigned* err, uint64_t* bar, uint32_t parity) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = ssu::global_ns();
  while (!ssu::mbar_test_sleep(bar, parity, 20000u)) {
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if (ssu::global_ns() - t0 > ssu::kWaitLimitNs) {
      *reinterpret_cast<volatile int*>(&sm.abort) = 1;
      atomicOr(err, kErrMma);
      return false;
    }
  }
  return true;
}

// ... for a whole warp, which goes on or gives up as one.
template <class SM>
__device__ __forceinline__ bool warp_wait(SM& sm, unsigned* err, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(sm, err, bar, parity));
}

// The warps of a role meet: a barrier of its own that gives up like every wait.
template <class SM>
__device__ __forceinline__ bool meet(SM& sm, unsigned* err, uint64_t* bar, uint32_t& parity) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  const bool ok = warp_wait(sm, err, bar, parity);
  parity ^= 1;
  return ok;
}

template <class IT>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <class IT>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The part of (a, b) that 16 bits hold, and what they leave of it.
template <class IT>
__device__ __forceinline__ uint32_t part(float& a, float& b) {
  const uint32_t w = pack2<IT>(a, b);
  const float2 f = unpack2<IT>(w);
  a -= f.x;
  b -= f.y;
  return w;
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Sixteen values of this thread's row of a state in global memory, columns
// [c, c + 16): loaded (or stored) by the warp in whole rows, 16 bytes a lane, and
// turned through `buf`, ROWS rows of 80 bytes.  `rows`: rows the warp has (32 or 16;
// row = lane).  ST is the state's type.
template <class ST, int DK, int ROWS>
__device__ __forceinline__ void load_rows16(const ST* tile, int c, unsigned char* buf, float* v) {
  constexpr int PER = 16 * (int)sizeof(ST) / 16;  // lanes of a row
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < ROWS * PER / 32; ++i) {
    const int row = (i * 32 + lane) / PER, piece = lane % PER;
    const uint4 w =
        *reinterpret_cast<const uint4*>(tile + (int64_t)row * DK + c + piece * (16 / sizeof(ST)));
    *reinterpret_cast<uint4*>(buf + row * 80 + piece * 16) = w;
  }
  __syncwarp();
  const unsigned char* mine = buf + (lane % ROWS) * 80;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(mine + i * 16);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(ST) == 4) v[i * 4 + k] = __uint_as_float(u[k]);
      else {
        const float2 f = unpack2<ST>(u[k]);
        v[i * 8 + 2 * k] = f.x;
        v[i * 8 + 2 * k + 1] = f.y;
      }
    }
  }
  __syncwarp();
}

template <class ST, int DK, int ROWS>
__device__ __forceinline__ void store_rows16(ST* tile, int c, unsigned char* buf, const float* v) {
  constexpr int PER = 16 * (int)sizeof(ST) / 16;
  const int lane = threadIdx.x & 31;
  if (lane < ROWS) {
    unsigned char* mine = buf + lane * 80;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(ST) == 4) u[k] = __float_as_uint(v[i * 4 + k]);
        else u[k] = pack2<ST>(v[i * 8 + 2 * k], v[i * 8 + 2 * k + 1]);
      }
      *reinterpret_cast<uint4*>(mine + i * 16) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < ROWS * PER / 32; ++i) {
    const int row = (i * 32 + lane) / PER, piece = lane % PER;
    const uint4 w = *reinterpret_cast<const uint4*>(buf + row * 80 + piece * 16);
    *reinterpret_cast<uint4*>(tile + (int64_t)row * DK + c + piece * (16 / sizeof(ST))) = w;
  }
  __syncwarp();
}

// FULL: the outputs and final states.  Else: what the pieces add to the state.
template <class IT, int DV, int DK, int PARTS, bool FULL>
__global__ void __launch_bounds__(kPromptThreads, 1)
    linattn_prompt_kernel(const __grid_constant__ PromptArgs g) {
  using Z = Sizes<DV, DK>;
  using SM = PromptSmem<DV, DK, PARTS>;
  constexpr bool kBF16 = std::is_same<IT, __nv_bfloat16>::value;
  constexpr int LIST = FULL ? 1 : 0;
  constexpr int ROWS = DV / 4;  // lanes of each 32 that hold a row where dv is one side (M = DV)
  constexpr int HALF = DK / 2;  // columns of S a thread owns
  extern __shared__ __align__(128) unsigned char smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const Args& p = g.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], kLoaders);
      mbar_init(&sm.empty[i], FULL ? 5 : 1);  // the products' end; the output warps' look at a_t
    }
    mbar_init(&sm.sc_full[0], 1);
    mbar_init(&sm.sc_full[1], 1);
    mbar_init(&sm.p_ready, 4);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, 4);
    mbar_init(&sm.s_ready, 8);
    mbar_init(&sm.v_ready, 8);
    mbar_init(&sm.d_full, 1);
    mbar_init(&sm.loaders, kLoaders / 32);
    mbar_init(&sm.state_warps, 8);
    mbar_init(&sm.out_warps, 4);
    mbar_init(&sm.fin, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sm.abort = 0;
    sm.any_bad[0] = sm.any_bad[1] = 0;
  }
  if (tid < 128) sm.bad[0][tid] = sm.bad[1][tid] = kC;
  if (warp == 16) tc::alloc(smem_addr(&sm.tmem), Z::kCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;  // this warp's lanes

  if (wg == 4) {
    regs_dec<80>();
    if (warp == 16) {
      // ---- the products --------------------------------------------------
      if (lane == 0) {
        constexpr uint32_t kIdSc = tc::idesc_f16(kBF16, 64, 64, false, false);
        constexpr uint32_t kIdO1 = tc::idesc_f16(kBF16, DV, 64, true, false);
        constexpr uint32_t kIdO2 = tc::idesc_f16(kBF16, DV, 64, false, false);
        constexpr uint32_t kIdD = tc::idesc_f16(kBF16, DV, DK, true, true);
        const uint32_t sp = smem_addr(sm.p[0]), swv = smem_addr(sm.wv[0]);
        auto scores = [&](int n) {
          const uint32_t q = smem_addr(sm.stage[n % kStages]), k = q + Z::kQ;
          tc::fence_after_sync();
          tc::fence_proxy_async();
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            tc::mma(tmem + Z::kSc + (n & 1) * 64, tc::sdesc(q + kk * 2 * kCol, kCol, 128),
                    tc::sdesc(k + kk * 2 * kCol, kCol, 128), kIdSc, kk != 0);
          tc::commit(smem_addr(&sm.sc_full[n & 1]));
        };
        bool ahead = false;  // the scores of chunk n are under way
        for (int n = 0;; ++n) {
          const int st = n % kStages;
          if (!wait(sm, g.err, &sm.full[st], (n / kStages) & 1)) break;
          if (sm.chunk[st].stop) break;
          const uint32_t q = smem_addr(sm.stage[st]), k = q + Z::kQ, v = k + Z::kQ;
          if constexpr (FULL) {
            if (!ahead) scores(n);
            const int nx = (n + 1) % kStages;
            ahead = mbar_test(&sm.full[nx], ((n + 1) / kStages) & 1) && !sm.chunk[nx].stop;
            if (ahead) scores(n + 1);
            if (!wait(sm, g.err, &sm.p_ready, n & 1)) break;
          }
          if (!wait(sm, g.err, &sm.v_ready, n & 1)) break;
          if constexpr (FULL) {
            if (n > 0 && !wait(sm, g.err, &sm.o_free, (n - 1) & 1)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < kC / 16; ++kk)
                tc::mma(tmem + Z::kO1, tc::sdesc(v + kk * 256, 128, kCol),
                        tc::sdesc(sp + part * Z::kP + kk * 2 * kCol, kCol, 128), kIdO1,
                        (part | kk) != 0);
            tc::commit(smem_addr(&sm.p_free));
            if (!wait(sm, g.err, &sm.s_ready, n & 1)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < DK / 16; ++kk)
                mma_ta(tmem + Z::kO2, tmem + Z::kS + part * HALF + kk * 8,
                       tc::sdesc(q + kk * 2 * kCol, kCol, 128), kIdO2, (part | kk) != 0);
            tc::commit(smem_addr(&sm.o_full));
          }
          tc::fence_after_sync();
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int kk = 0; kk < kC / 16; ++kk)
              tc::mma(tmem + Z::kD, tc::sdesc(swv + part * Z::kV + kk * 256, 128, kCol),
                      tc::sdesc(k + kk * 256, 128, kCol), kIdD, (part | kk) != 0);
          tc::commit(smem_addr(&sm.d_full));
          tc::commit(smem_addr(&sm.empty[st]));
        }
        // nothing is in flight any more when the tensor memory is given back
        tc::commit(smem_addr(&sm.fin));
        const uint64_t t0 = ssu::global_ns();
        while (!mbar_test(&sm.fin, 0) && ssu::global_ns() - t0 < ssu::kWaitLimitNs) {
        }
      }
      __syncwarp();
    } else {
      // ---- loads, three warps --------------------------------------------
      const int lt = tid - 17 * 32;  // 0 .. 95
      const int items = g.head->count[LIST] * p.H;
      int n = 0;
      bool live = true;
      uint32_t met = 0;
      auto landed = [&](int m) {  // this thread's copies of chunk m are in shared memory
        tc::fence_proxy_async();
        mbar_arrive(&sm.full[m % kStages]);
      };
      int next = 0;
      if (lt == 0) next = atomicAdd(&g.head->next[LIST], 1);
      while (live) {
        if (lt == 0) {
          sm.item = next;
          next = atomicAdd(&g.head->next[LIST], 1);  // on its way during this item
        }
        if (!meet(sm, g.err, &sm.loaders, met)) live = false;
        const int item = sm.item;
        if (!meet(sm, g.err, &sm.loaders, met)) live = false;
        if (!live || item >= items) break;
        const Piece piece = g.pieces[LIST][item / p.H];
        const int h = item % p.H, grp = h / p.hr;
        const IT* qg = static_cast<const IT*>(p.q) + (int64_t)piece.r0 * p.q_rs + grp * p.q_gs;
        const IT* kg = static_cast<const IT*>(p.k) + (int64_t)piece.r0 * p.k_rs + grp * p.k_gs;
        const IT* vg = static_cast<const IT*>(p.v) + (int64_t)piece.r0 * p.v_rs + h * p.v_hs;
        const int chunks = (piece.len + kC - 1) / kC;
        auto decay_at = [&](int t) {
          return p.ld && t < piece.len ? p.ld[(int64_t)(piece.r0 + t) * p.ld_rs + h * p.ld_hs]
                                       : 0.0f;
        };
        float l0 = 0.0f, l1 = 0.0f;
        if (warp == 17) l0 = decay_at(2 * lane), l1 = decay_at(2 * lane + 1);
        for (int c = 0; c < chunks; ++c, ++n) {
          const int st = n % kStages;
          if (n >= kStages && !warp_wait(sm, g.err, &sm.empty[st], (n / kStages - 1) & 1)) {
            live = false;
            break;
          }
          const int t0 = c * kC, rows = min(kC, piece.len - t0);
          const uint32_t q = smem_addr(sm.stage[st]), k = q + Z::kQ, v = k + Z::kQ;
          auto tile = [&](uint32_t to, const IT* from, int64_t rs, int pieces) {
            for (int i = lt; i < kC * pieces; i += kLoaders) {
              const int row = i / pieces, col = i % pieces;
              tc::cp16(to + col * kCol + row * 16, from + (t0 + (row < rows ? row : 0)) * rs + col * 8,
                       row < rows ? 16u : 0u);
            }
          };
          if constexpr (FULL) tile(q, qg, p.q_rs, DK / 8);
          tile(k, kg, p.k_rs, DK / 8);
          tile(v, vg, p.v_rs, DV / 8);
          tc::cp_commit();
          if (warp == 17) {
            // a_t in 64 bits: differences of large sums keep their digits.  A log decay below
            // -160 (in units of log2) is a decay of zero in fp32 and is held there.
            auto held = [](float l) {
              l *= kLog2e;
              asm("max.NaN.f32 %0, %0, %1;" : "+f"(l) : "f"(-160.0f));
              return (double)l;
            };
            const double d0 = held(l0), d1 = held(l1);
            double inc = d0 + d1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const double u = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += u;
            }
            const double end = __shfl_sync(0xffffffffu, inc, 31);
            const double a1 = inc, a0 = inc - d1;
            Tables& tab = sm.tab[st];
            const int t = 2 * lane;
            tab.a[t] = (float)a0;
            tab.a[t + 1] = (float)a1;
            tab.ea[t] = p.scale * exp2f((float)a0);
            tab.ea[t + 1] = p.scale * exp2f((float)a1);
            tab.w[t] = t < rows ? exp2f((float)(end - a0)) : 0.0f;
            tab.w[t + 1] = t + 1 < rows ? exp2f((float)(end - a1)) : 0.0f;
            if (lane == 0) {
              // near 1 the decay is 1 + add: rounded by itself it would be off by the same
              // 2^-25 chunk after chunk
              const float e = exp2f((float)end);
              tab.decay = e;
              tab.keep = e > 0.5f ? 1.0f : 0.0f;
              tab.add = e > 0.5f ? expm1f((float)(end * 0.69314718055994531)) : e;
            }
            l0 = decay_at(t0 + kC + 2 * lane);
            l1 = decay_at(t0 + kC + 2 * lane + 1);
          }
          if (lt == 0)
            sm.chunk[st] = Chunk{h, piece.r0 + t0, rows, c == 0, c == chunks - 1, 0, piece};
          if (n > 0) {
            tc::cp_wait<1>();
            landed(n - 1);
          }
        }
      }
      tc::cp_wait<0>();
      if (live) {
        if (n > 0) landed(n - 1);
        const int st = n % kStages;
        if (n < kStages || warp_wait(sm, g.err, &sm.empty[st], (n / kStages - 1) & 1)) {
          if (lt == 0) sm.chunk[st].stop = 1;
          landed(n);
        }
      }
    }
  } else if (wg == 0) {
    regs_dec<80>();
    if constexpr (FULL) {
      // ---- P --------------------------------------------------------------
      const int t = 16 * warp + (lane & 15);
      for (int n = 0;; ++n) {
        const int st = n % kStages;
        if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
        if (!warp_wait(sm, g.err, &sm.sc_full[n & 1], (n >> 1) & 1)) break;
        if (n > 0 && !warp_wait(sm, g.err, &sm.p_free, (n - 1) & 1)) break;
        __syncwarp();
        tc::fence_after_sync();
        const Tables& tab = sm.tab[st];
        const float at = tab.a[t];
#pragma unroll
        for (int c = 0; c < kC; c += 16) {
          float s[16];
          tc::ld16(tmem + quad + Z::kSc + (n & 1) * 64 + c, s);
          tc::wait_ld();
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float x = c + i <= t ? s[i] * (p.scale * ex2(at - tab.a[c + i])) : 0.0f;
            float y = c + i + 1 <= t ? s[i + 1] * (p.scale * ex2(at - tab.a[c + i + 1])) : 0.0f;
            hi[i / 2] = part<IT>(x, y);
            lo[i / 2] = pack2<IT>(x, y);
          }
          if (lane < 16) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              unsigned char* to = sm.p[0] + (c / 8 + j) * kCol + t * 16;
              *reinterpret_cast<uint4*>(to) =
                  make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
              *reinterpret_cast<uint4*>(to + Z::kP) =
                  make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
            }
          }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready);
      }
    }
  } else if (wg == 1) {
    regs_dec<80>();
    if constexpr (FULL) {
      // ---- outputs -----------------------------------------------------------
      const int pv = ROWS * (warp & 3) + lane % ROWS;
      uint32_t met = 0;
      bool any_dead = false;
      for (int n = 0; !any_dead; ++n) {
        const int st = n % kStages;
        if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
        const int rows = sm.chunk[st].rows;
        IT* out = static_cast<IT*>(p.out) + (int64_t)sm.chunk[st].r0 * p.o_rs +
                  sm.chunk[st].h * p.o_hs + pv;
        if (!warp_wait(sm, g.err, &sm.o_full, n & 1)) break;
        __syncwarp();
        tc::fence_after_sync();
        const float back = kBF16 ? 1.0f : sm.row_scale[n & 1][pv];
        const int any = sm.any_bad[n & 1];
        const int bad = any ? sm.bad[n & 1][pv] : kC;
#pragma unroll
        for (int c = 0; c < kC; c += 16) {
          float o1[16], o2[16];
          tc::ld16(tmem + quad + Z::kO1 + c, o1);
          tc::ld16(tmem + quad + Z::kO2 + c, o2);
          tc::wait_ld();
          if (c == kC - 16) {  // all of it read
            if (any) {
              if (!meet(sm, g.err, &sm.out_warps, met)) any_dead = true;
              if (lane < ROWS) sm.bad[n & 1][pv] = kC;
              if (tid == 128) sm.any_bad[n & 1] = 0;
            }
            tc::fence_before_sync();
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y = fmaf(o2[i] * back, sm.tab[st].ea[c + i], o1[i]);
            if (c + i >= bad) y = NAN;
            if (lane < ROWS && c + i < rows) out[(c + i) * p.o_rs] = from_f<IT>(y);
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.o_free);
          mbar_arrive(&sm.empty[st]);
        }
      }
    }
  } else {
    regs_inc<120>();
    // ---- S and w V -------------------------------------------------------
    const int half = wg - 2, st_tid = tid - 256;  // 0 .. 255
    const int row = ROWS * (warp & 3) + lane % ROWS;
    unsigned char* buf = sm.wv[0] + (warp - 8) * ROWS * 80;  // this warp's, while w V is not in use
    static_assert(8 * ROWS * 80 <= PARTS * Z::kV, "the buffers fit w V's place");
    float S[HALF];
    float total = 1.0f;
    uint32_t met = 0;
    bool dead = false;
    auto state_warps_meet = [&] {
      if (!meet(sm, g.err, &sm.state_warps, met)) dead = true;
    };
    // S as the next chunk's operand
    auto give = [&](int n) {
      float by = 1.0f;
      if constexpr (!kBF16) {
        // fp16 has no room for a large S: each row is brought to about 2^10 by a power of two
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < HALF; ++i) m = fmaxf(m, fabsf(S[i]));
        if (lane < ROWS) sm.row_max[half][row] = m;
        state_warps_meet();
        m = fmaxf(sm.row_max[0][row], sm.row_max[1][row]);
        int e = (int)((__float_as_uint(m) >> 23) & 255) - 127 - 10;
        e = m > 0.0f ? (e < -100 ? -100 : e > 110 ? 110 : e) : 0;
        by = __uint_as_float((uint32_t)(127 - e) << 23);
        if (half == 0 && lane < ROWS)
          sm.row_scale[n & 1][row] = __uint_as_float((uint32_t)(127 + e) << 23);
        state_warps_meet();  // row_max is written again in the next chunk
      }
#pragma unroll
      for (int c = 0; c < HALF; c += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x = S[c + 2 * i] * by, y = S[c + 2 * i + 1] * by;
          hi[i] = part<IT>(x, y);
          lo[i] = pack2<IT>(x, y);
        }
        const uint32_t at = tmem + quad + Z::kS + (half * HALF + c) / 2;
        st_tmem8(at, hi);
        st_tmem8(at + HALF, lo);
      }
      wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_ready);
    };
    auto rows_of_state = [&](auto* pool, int64_t slot, int h) {
      return pool + ((slot * p.H + h) * DV + ROWS * (warp & 3)) * DK + half * HALF;
    };
    auto entry = [&](int e, int h) {  // of the workspace's states; this thread's first four values
      return reinterpret_cast<float4*>(g.state) + ((int64_t)e * p.H + h) * (DV * DK / 4) +
             (half * 4 + (warp & 3)) * (HALF / 4 * ROWS) + lane % ROWS;
    };
    for (int n = 0; !dead; ++n) {
      const int st = n % kStages;
      if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
      const Tables& tab = sm.tab[st];
      // what is looked at after w V is given over, when the stage may be filled again
      const float keep = tab.keep, add = tab.add;
      const bool last = sm.chunk[st].last;
      const Piece pc = sm.chunk[st].piece;
      const int h = sm.chunk[st].h;
      if (sm.chunk[st].first) {
#pragma unroll
        for (int i = 0; i < HALF; ++i) S[i] = 0.0f;
        total = 1.0f;
        if (FULL && pc.of > 1) {
          // the entry behind the last piece before this one, from the first on
          const int e0 = pc.j > 0 ? 1 : 0;
          for (int e = e0; e <= pc.j; ++e) {
            const float by = e > e0 ? g.decay[(int64_t)(pc.base + e - 1) * p.H + h] : 0.0f;
            const float4* from = entry(pc.base + e, h);
#pragma unroll
            for (int i = 0; i < HALF / 4; ++i) {
              const float4 v = from[i * ROWS];
              S[4 * i] = fmaf(S[4 * i], by, v.x);
              S[4 * i + 1] = fmaf(S[4 * i + 1], by, v.y);
              S[4 * i + 2] = fmaf(S[4 * i + 2], by, v.z);
              S[4 * i + 3] = fmaf(S[4 * i + 3], by, v.w);
            }
          }
        } else if (pc.j == 0) {
          const Slot from = load_slot(g.a.src, pc.seq, 0, g.a.idx64);
          const int64_t slot = from.id(pc.seq, g.a.idx64);
          if (from.found && slot_ok(slot, p.pad, p.slots) && (!p.has_init || p.has_init[pc.seq])) {
#pragma unroll
            for (int c = 0; c < HALF; c += 16) {
              if (p.state_dtype == SSU_F32)
                load_rows16<float, DK, ROWS>(rows_of_state(static_cast<const float*>(p.state), slot, h),
                                             c, buf, S + c);
              else if (p.state_dtype == SSU_BF16)
                load_rows16<__nv_bfloat16, DK, ROWS>(
                    rows_of_state(static_cast<const __nv_bfloat16*>(p.state), slot, h), c, buf, S + c);
              else
                load_rows16<__half, DK, ROWS>(
                    rows_of_state(static_cast<const __half*>(p.state), slot, h), c, buf, S + c);
            }
          }
          if (!FULL && lane < ROWS) {  // the second launch finds it here, whatever is in the slot then
            float4* to = entry(pc.base, h);
#pragma unroll
            for (int i = 0; i < HALF / 4; ++i)
              to[i * ROWS] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
          }
        }
        state_warps_meet();  // the buffers are w V's again
        if (FULL) give(n);
      }
      total *= tab.decay;
      // w V
      const unsigned char* v = sm.stage[st] + 2 * Z::kQ;
#pragma unroll 1
      for (int i = st_tid; i < kC * (DV / 8); i += 256) {
        const int s = i % kC, at = i / kC * kCol + s * 16;
        const uint4 raw = *reinterpret_cast<const uint4*>(v + at);
        uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
        const float w = tab.w[s];
        uint32_t o[PARTS][4];
        bool odd = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t e = kBF16 ? 0x7f807f80u : 0x7c007c00u;
          const uint32_t x = u[k] & e;
          odd |= (x & 0xffffu) == (e & 0xffffu) || (x >> 16) == (e >> 16);
          const float2 f = unpack2<IT>(u[k]);
          float a = f.x * w, b = f.y * w;
#pragma unroll
          for (int r = 0; r < PARTS - 1; ++r) o[r][k] = part<IT>(a, b);
          o[PARTS - 1][k] = pack2<IT>(a, b);
        }
#pragma unroll
        for (int r = 0; r < PARTS; ++r)
          *reinterpret_cast<uint4*>(sm.wv[r] + at) = make_uint4(o[r][0], o[r][1], o[r][2], o[r][3]);
        if (odd) {
          // A value that is not finite must not reach the tokens before its own, as 0 x
          // infinity would in P V: it is taken out of V, and the outputs of its channel are
          // NaN from its token on, as the state is.
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const uint32_t e = kBF16 ? 0x7f80u : 0x7c00u;
            uint16_t* x = reinterpret_cast<uint16_t*>(const_cast<unsigned char*>(v + at)) + k;
            if ((*x & e) == e) {
              *x = 0;
              atomicMin(&sm.bad[n & 1][i / kC * 8 + k], s);
              sm.any_bad[n & 1] = 1;
            }
          }
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_ready);
      if (!warp_wait(sm, g.err, &sm.d_full, n & 1)) break;
      __syncwarp();
      tc::fence_after_sync();
#pragma unroll
      for (int c = 0; c < HALF; c += 16) {
        float d[16];
        tc::ld16(tmem + quad + Z::kD + half * HALF + c, d);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) S[c + i] = fmaf(S[c + i], add, fmaf(keep, S[c + i], d[i]));
      }
      tc::fence_before_sync();
      if (!last) {
        if (FULL) give(n + 1);
        continue;
      }
      if constexpr (!FULL) {
        if (lane < ROWS) {
          float4* to = entry(pc.base + pc.j + 1, h);
#pragma unroll
          for (int i = 0; i < HALF / 4; ++i)
            to[i * ROWS] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
        if (st_tid == 0) g.decay[(int64_t)(pc.base + pc.j) * p.H + h] = total;
      } else if (pc.j == pc.of - 1) {
        const Slot from = load_slot(g.a.src, pc.seq, 0, g.a.idx64);
        int64_t to;
        if (from.found && slot_ok(from.id(pc.seq, g.a.idx64), p.pad, p.slots) &&
            write_slot(g.a, pc.seq, 0, p.pad, p.slots, &to)) {
#pragma unroll
          for (int c = 0; c < HALF; c += 16) {
            if (p.state_dtype == SSU_F32)
              store_rows16<float, DK, ROWS>(rows_of_state(static_cast<float*>(p.state), to, h), c,
                                            buf, S + c);
            else if (p.state_dtype == SSU_BF16)
              store_rows16<__nv_bfloat16, DK, ROWS>(
                  rows_of_state(static_cast<__nv_bfloat16*>(p.state), to, h), c, buf, S + c);
            else
              store_rows16<__half, DK, ROWS>(rows_of_state(static_cast<__half*>(p.state), to, h), c,
                                             buf, S + c);
          }
        }
        state_warps_meet();
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 16) tc::dealloc(tmem, Z::kCols);
}

}  // namespace linattn
