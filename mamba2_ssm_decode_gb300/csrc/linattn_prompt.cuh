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
// output's own rounding), w V as three of bf16 (all of an fp32 number; two leave
// 2^-17, which shows in an fp32 state) or two of fp16.  fp16 has no room for what
// is large or small: there the rows of P and S and all of a chunk's w V are brought
// to the middle of its range by powers of two, which are taken out of the products.
// (One power for all of w V: a channel whose largest value is below 2^-17 of the
// chunk's keeps fewer than 22 bits in the state, 16 at 2^-23, down to fp16's last
// subnormal.  A power for each channel would have every warp look at all tokens.)
// Exponents are differences of 64-bit sums, or are taken so that 2^-17 is left of them
// at most; e^ a sum counts as zero below 2^-126.
//
// One CTA of 24 warps works on a chunk of one head at a time, chunks of a
// sequence in order: 4 warps turn scores into P, 4 write outputs, 8 update S (each
// owns 32 lanes of tensor memory, so the tiles' rows), 4 weigh V, half a chunk
// ahead of its product, three issue the products, one has Q, K and V copied (TMA,
// three chunks ahead, 128-byte swizzle) and sums the decays.
// Items -- a sequence's, or a piece's, chunks of one head -- are handed out by a
// counter, longest first.  A sequence of more chunks than every SM's fair share
// is cut into pieces: a first launch computes what each piece adds to the state
// (the fourth product alone) and the exponent of its decay, a second one adds them up
// to the state that enters each piece.  Every launch but the first is set up while the one before
// runs (programmatic dependent launch).
//
// 20634 tokens of 16 prompts, 32 heads of 128 x 128 in bf16: 204 us (HBM's floor 108,
// the tensor pipe's 62).  A chunk takes some 4000 cycles, in which the roles wait for one
// another: of a warp's cycles for each instruction 4.9 go to barriers and memory, 2.0 to
// the next instruction (six roles share each scheduler's instruction cache), 1.4 to fixed
// latencies, 1.2 to shared memory; 48 % of the issue slots are used.  More stages (210 us)
// and fewer waits for them (204) took nothing off.
#pragma once

#include <cuda.h>

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
  int next[2];   // items handed out: of the pieces' launch, of the last
  int count[2];  // pieces of each
  int cuts;      // sequences in pieces
};

// A sequence in pieces: its entries in the workspace's states.
struct CutSeq {
  int base, of;
};

struct PromptArgs {
  CUtensorMap q, k, v;  // [rows][groups or heads][dk or dv], boxes of 64 rows x 1 x 64
  Args p;
  Seqs a;
  Header* head;
  Piece* pieces[2];
  CutSeq* cuts;
  float* decay;  // [entries][H]: log2 of what a piece decays the state by
  float* state;  // [entries][H][dv * dk], in the threads' order
  int fair, cut;  // chunks: more than `fair` of them are cut into pieces of about `cut`
  int entries, splits;  // room: states, sequences in pieces
  unsigned* err;
};

// ---------------------------------------------------------------------------
// plan: the pieces, longest first
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kBuckets = 64;

struct Cut {
  int r0, len, chunks, pieces, each;  // each: chunks of a piece (the last may have fewer)
  Cut() = default;
  __device__ __forceinline__ Cut(const PromptArgs& g, int s, bool split) {
    r0 = len = chunks = pieces = each = 0;
    if (s >= g.a.n) return;
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

// What follows may be set up by now; it waits for this launch's end all the same.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// The launch before has ended, and its results can be read.
__device__ __forceinline__ void launch_before_ended() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch that may be set up while the one before it on the stream still runs.
template <class... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// f(piece, base, j) for every piece of sequences s .. s + 31 (a lane's own is c): a
// whole sequence by its lane, one in pieces by all lanes.  base: of its entries.
template <class F>
__device__ __forceinline__ void each_piece(const Cut& c, int base, F f) {
  const int lane = threadIdx.x & 31;
  if (c.pieces == 1) f(c, base, lane, 0);
  for (unsigned m = __ballot_sync(0xffffffffu, c.pieces > 1); m; m &= m - 1) {
    const int from = __ffs(m) - 1;
    Cut d;
    d.r0 = __shfl_sync(0xffffffffu, c.r0, from);
    d.len = __shfl_sync(0xffffffffu, c.len, from);
    d.chunks = __shfl_sync(0xffffffffu, c.chunks, from);
    d.pieces = __shfl_sync(0xffffffffu, c.pieces, from);
    d.each = __shfl_sync(0xffffffffu, c.each, from);
    const int b = __shfl_sync(0xffffffffu, base, from);
    for (int j = lane; j < d.pieces; j += 32) f(d, b, from, j);
  }
}

static __global__ void __launch_bounds__(kPlanThreads) linattn_plan_kernel(const PromptArgs g) {
  __shared__ int at[2][kBuckets];
  __shared__ int used, want, many, cuts;
  let_next_start();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < kBuckets) at[0][tid] = at[1][tid] = 0;
  if (tid == 0) used = want = many = cuts = 0;
  __syncthreads();
  for (int s = tid; s < g.a.n; s += kPlanThreads) {
    const Cut c(g, s, true);
    if (c.pieces > 1) {
      atomicAdd(&want, c.pieces);
      atomicAdd(&many, 1);
    }
  }
  __syncthreads();
  // starts that do not ascend could ask for more than the workspace has room for
  const bool split = want <= g.entries && many <= g.splits;
  for (int s0 = tid - lane; s0 < g.a.n; s0 += kPlanThreads)
    each_piece(Cut(g, s0 + lane, split), 0, [&](const Cut& c, int, int, int j) {
      const int b = c.bucket(g, j);
      atomicAdd(&at[1][b], 1);
      if (j + 1 < c.pieces) atomicAdd(&at[0][b], 1);
    });
  __syncthreads();
  if (tid < 64) {  // where each bucket starts
    static_assert(kBuckets == 64, "two of a lane");
    int* mine = at[tid >> 5];
    const int n0 = mine[2 * lane], n1 = mine[2 * lane + 1];
    int inc = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    mine[2 * lane] = inc - n0 - n1;
    mine[2 * lane + 1] = inc - n1;
    if (lane == 31) {
      g.head->count[tid >> 5] = inc;
      g.head->next[tid >> 5] = 0;
    }
  }
  __syncthreads();
  for (int s0 = tid - lane; s0 < g.a.n; s0 += kPlanThreads) {
    const Cut c(g, s0 + lane, split);
    int base = 0;
    if (c.pieces > 1) {
      base = atomicAdd(&used, c.pieces);
      g.cuts[atomicAdd(&cuts, 1)] = CutSeq{base, c.pieces};
    }
    each_piece(c, base, [&](const Cut& d, int b, int from, int j) {
      const int first = j * d.each * kC;
      const Piece piece{s0 + from, d.r0 + first, min(d.len - first, d.each * kC), j, d.pieces, b};
      const int k = d.bucket(g, j);
      g.pieces[1][atomicAdd(&at[1][k], 1)] = piece;
      if (j + 1 < d.pieces) g.pieces[0][atomicAdd(&at[0][k], 1)] = piece;
    });
  }
  __syncthreads();
  if (tid == 0) g.head->cuts = cuts;
}

// ---------------------------------------------------------------------------
// the states that enter pieces
// ---------------------------------------------------------------------------
// Entry base is the state that enters the first piece, base + 1 the one that leaves
// it, base + j + 1 what piece j adds; from the third on they become what enters
// piece j: E_j = decay of piece j - 1 E_(j - 1) + what it adds.
constexpr int kJoinThreads = 256;

// 2^l as a factor: near 1 as 1 + add, as a chunk's decay is, and in three equal steps where
// fp32 has no room for it, though it may have for the product (nothing stays nothing).
struct Factor {
  float step, last;
  bool near;
  __device__ __forceinline__ explicit Factor(float l) {
    near = fabsf(l) < 1.0f;
    const float m = l > 360.0f && l < INFINITY ? 360.0f : l;  // beyond, all but zero is infinite
    const bool inside = fabsf(m) < 126.0f;
    step = inside ? 1.0f : ex2(m * (1.0f / 3.0f));
    last = near ? expm1f(l * 0.693147181f) : inside ? ex2(m) : step;
  }
  // v + 2^l s
  __device__ __forceinline__ float times(float s, float v) const {
    s = s * step * step;
    return fmaf(s, last, near ? s + v : v);
  }
};

static __global__ void __launch_bounds__(kJoinThreads) linattn_join_kernel(const PromptArgs g) {
  let_next_start();
  launch_before_ended();
  if ((int)blockIdx.y >= g.head->cuts) return;
  const CutSeq c = g.cuts[blockIdx.y];
  const int64_t per = (int64_t)g.p.dv * g.p.dk / 4, all = per * g.p.H;  // of an entry
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  if (i >= all || c.of < 3) return;
  const int h = (int)(i / per);
  float4* e = reinterpret_cast<float4*>(g.state) + (int64_t)(c.base + 1) * all + i;
  const float* by = g.decay + (int64_t)(c.base + 1) * g.p.H + h;
  float4 s = *e;
#pragma unroll 4
  for (int j = 2; j < c.of; ++j) {
    e += all;
    const Factor d(*by);
    by += g.p.H;
    const float4 v = *e;
    s.x = d.times(s.x, v.x);
    s.y = d.times(s.y, v.y);
    s.z = d.times(s.z, v.z);
    s.w = d.times(s.w, v.w);
    *e = s;
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

// a - b
__device__ __forceinline__ float between(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }
// A sum of log decays as two floats: in units of 2^-44 its multiples of 2^-8, whole below
// 2^16, and the rest to 2^-32; of a double what fp32 takes and what that leaves.
__device__ __forceinline__ float2 in_two(long long v) {
  return make_float2((float)(int)(v >> 36) * 0x1p-8f, (float)(uint32_t)(v >> 4) * 0x1p-40f);
}
__device__ __forceinline__ float2 in_two(double v) {
  const float high = (float)v;
  return make_float2(high, (float)(v - (double)high));
}

struct alignas(16) Tables {  // of a chunk, in units of log2; read in pairs
  float a[kC];         // a_t
  float2 two[kC];      // a_t as the sum of two, which gives a difference its own rounding
                       // however large the sums are
  float x[kC];         // e^(r - a_s), r the a of the last token of s's 16
  float ea[kC];        // scale e^(a_t)
  float w[kC];         // e^(a_C - a_s); 0 behind the last row
  float r[kC / 16];    // the four r
  float keep, add;     // e^(a_C) = keep + add, keep 0 or 1
  int mild;            // inside the 16 of an r, e^(a_t - r) stays below 2^60 and e^(r - a_s) below
                       // 2 (it can lift nothing that e^(a_t - r) loses at 2^-126), and a_t stays
                       // within 128, so that a_t - r is off by 2^-17 at most
};

// A tile: 64 rows (tokens) of 128 bytes, one after the other, the 16-byte pieces
// of row s at (piece ^ s % 8): the 128-byte swizzle, whose atoms are 8 rows.  Wider
// rows are several tiles.
constexpr int kTile = kC * 128;
__device__ __forceinline__ int tile_at(int s, int piece) {
  return (piece >> 3) * kTile + s * 128 + ((piece ^ s) & 7) * 16;
}
// Descriptors of operands in tiles.  Rows are the operand's M (or N): 32 bytes
// further per 16 of K.  Rows are its K: 16 of them are 2048 bytes, and 64 of M (N)
// a tile.
__device__ __forceinline__ uint64_t rows_mn(uint32_t addr) {
  return tc::sdesc(addr, 16, 1024) | (2ull << 61);
}
__device__ __forceinline__ uint64_t rows_k(uint32_t addr) {
  return tc::sdesc(addr, kTile, 1024) | (2ull << 61);
}

template <int DV, int DK>
struct Sizes {
  static constexpr int kQ = DK / 64 * kTile, kV = DV / 64 * kTile, kP = kTile;
  static constexpr int kStage = 2 * kQ + kV;
  static constexpr int kCols = 512;  // of tensor memory
  // columns: D, o1, o2, scores (two), S (high parts, remainders)
  static constexpr int kD = 0, kO1 = 128, kO2 = 192, kSc = 256, kS = 384;
  // outputs are turned in the place of Q, where they fit: Q is done with by then
  static constexpr int kOut = DV > DK ? kV : 0;
};

template <int DV, int DK, int PARTS>
struct PromptSmem {
  using Z = Sizes<DV, DK>;
  unsigned char stage[kStages][Z::kStage];  // Q, K, V
  unsigned char wv[PARTS][Z::kV];
  unsigned char p[2][Z::kP];
  alignas(16) unsigned char out[Z::kOut ? Z::kOut : 16];
  Tables tab[kStages];
  Chunk chunk[kStages];
  // fp16 (two parts) alone
  static constexpr int kScaled = PARTS == 2 ? 128 : 1;
  float row_max[2][2][kScaled];  // the largest value of half a row of S
  float row_scale[2][kScaled];  // what a row of S was divided by
  alignas(16) float p_scale[2][kScaled];  // ... a token's row of P, read in pairs
  float v_scale[kStages];       // ... w V
  uint32_t v_max[kStages][4];   // the largest of w V, by warp
  int bad[kStages][128];    // the first token of the chunk whose v is not finite
  int any_bad[kStages];
  uint64_t full[kStages], empty[kStages], v_ready[kStages], sc_full[2], sc_free[2];
  uint64_t p_ready, p_free, o_full, o_free, s_ready, s_free, d_full, d_free, wv_ready[2], wv_free[2];
  uint64_t state_warps, out_warps, v_warps, fin;  // warps of a role meet; the last product
  uint32_t tmem;
  int abort;
};

constexpr int kPromptThreads = 768;

__device__ __forceinline__ void st_tmem8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The products, issued by a whole warp of which one lane is elected (the same one
// every time).  What a product is given lies in uniform registers, which takes
// control flow that the compiler knows to be uniform and unrolled loops: then a
// product of 128 x 128 x 16 takes 65 cycles, 68 among 20 busy warps; from a loop
// that is not unrolled 65 and 440.
// D (tensor memory) = A B^T, or += where `accumulate` is not 0.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// ... with A in tensor memory.
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrival on `bar` once every product before has completed.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// A box of 64 rows x 64 elements from (row, group, column).
__device__ __forceinline__ void load_box(uint32_t to, const CUtensorMap* map, uint32_t bar, int col,
                                         int group, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5}], [%2];" ::"r"(to),
      "l"(map), "r"(bar), "r"(col), "r"(group), "r"(row)
      : "memory");
}

// 16 lanes x 32 (or 16) columns as 8 x 8 fragments: v[4 f + i] is row lane / 4 + (i
// < 2 ? 0 : 8), column 8 f + 2 (lane % 4) + i % 2.
__device__ __forceinline__ void ld_frag4(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void ld_frag2(uint32_t addr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Four 8 x 8 matrices of fragments to shared memory; lane l gives the address of row
// l % 8 of matrix l / 8.  TRANS: rows in memory are the fragments' columns.
template <bool TRANS>
__device__ __forceinline__ void st_frags(uint32_t addr, const uint32_t (&w)[4]) {
  if constexpr (TRANS)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// Waits for a phase; gives up after about two seconds, or when another thread did.
// Few instructions, because it stands in two dozen places: a test may sleep for a
// microsecond, and 2^21 of them are the limit.
template <class SM>
__device__ __forceinline__ bool wait(SM& sm, unsigned* err, uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int tries = 0; !ssu::mbar_test_sleep(bar, parity, 1000u); ++tries) {
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if (tries >> 21) {
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

// The 16-bit part of two fp32 numbers, which leaves the rest of them.
template <class IT>
__device__ __forceinline__ uint32_t part(float2& v) {
  const uint32_t w = pack2<IT>(v.x, v.y);
  v = __ffma2_rn(unpack2<IT>(w), make_float2(-1.0f, -1.0f), v);
  return w;
}
// ... cut off, not rounded: three such parts of 8 bits are all of an fp32 number.
__device__ __forceinline__ uint32_t part_cut(float2& v) {
  const uint32_t x = __float_as_uint(v.x), y = __float_as_uint(v.y);
  const float2 f = make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u));
  v = __ffma2_rn(f, make_float2(-1.0f, -1.0f), v);
  return __byte_perm(x, y, 0x7632);
}

// The power of two that brings m to [2^to, 2^(to + 1)), and its reciprocal; 1 where m
// is 0 or not finite.  Held so that both are normal fp32 numbers: an m below 2^(to - 126)
// stays lower.
__device__ __forceinline__ float toward(float m, int to, float* back) {
  const int field = (int)(__float_as_uint(m) >> 23) & 255;
  int e = field - 127 - to;
  e = field == 255 || !(m > 0.0f) ? 0 : e < -126 ? -126 : e;
  *back = __uint_as_float((uint32_t)(127 + e) << 23);
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// Stays 0 while the two values of every word are finite.
template <class IT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w, uint32_t acc) {
  if constexpr (std::is_same<IT, __nv_bfloat16>::value) {
    const __nv_bfloat162 r =
        __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __nv_bfloat162{},
                *reinterpret_cast<const __nv_bfloat162*>(&acc));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&w), __half2{},
                              *reinterpret_cast<const __half2*>(&acc));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 bytes of global memory, in one access where `wide` says that they start on such
// a boundary: a whole sector a lane.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&r)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
    r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&r)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    static_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// N values of this thread's row of a state; ST is the state's type.
template <class ST, int N>
__device__ __forceinline__ void load_row(const ST* row, bool wide, float* v) {
  constexpr int E = 32 / (int)sizeof(ST);
  uint32_t r[N / E][8];
#pragma unroll
  for (int i = 0; i < N / E; ++i) load32(row + i * E, wide, r[i]);
#pragma unroll
  for (int i = 0; i < N / E; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (sizeof(ST) == 4) {
        v[i * E + k] = __uint_as_float(r[i][k]);
      } else {
        const float2 f = unpack2<ST>(r[i][k]);
        v[i * E + 2 * k] = f.x;
        v[i * E + 2 * k + 1] = f.y;
      }
    }
}

template <class ST, int N>
__device__ __forceinline__ void store_row(ST* row, bool wide, const float* v) {
  constexpr int E = 32 / (int)sizeof(ST);
#pragma unroll
  for (int i = 0; i < N / E; ++i) {
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (sizeof(ST) == 4) r[k] = __float_as_uint(v[i * E + k]);
      else r[k] = pack2<ST>(v[i * E + 2 * k], v[i * E + 2 * k + 1]);
    }
    store32(row + i * E, wide, r);
  }
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
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const Args& p = g.p;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), wg = warp >> 2;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 2);              // the copies' bytes; the tables
      mbar_init(&sm.empty[i], FULL ? 15 : 9);  // the products' end; S's warps; the output warps
      mbar_init(&sm.v_ready[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.sc_full[i], 1);
      mbar_init(&sm.sc_free[i], 4);
    }
    mbar_init(&sm.p_ready, 4);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, 4);
    mbar_init(&sm.s_ready, 8);
    mbar_init(&sm.s_free, 1);
    mbar_init(&sm.d_free, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.wv_ready[i], 4);
      mbar_init(&sm.wv_free[i], 1);
    }
    mbar_init(&sm.d_full, 1);
    mbar_init(&sm.state_warps, 8);
    mbar_init(&sm.out_warps, 4);
    mbar_init(&sm.v_warps, 4);
    mbar_init(&sm.fin, FULL ? 3 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sm.abort = 0;
    for (int i = 0; i < kStages; ++i) sm.any_bad[i] = 0;
  }
  if (tid < 128)
    for (int i = 0; i < kStages; ++i) sm.bad[i][tid] = kC;
  // P above its diagonal stays zero throughout
  for (int i = tid; i < 2 * Z::kP / 16; i += kPromptThreads)
    reinterpret_cast<uint4*>(sm.p[0])[i] = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_proxy_async();
  if (warp == 20) tc::alloc(smem_addr(&sm.tmem), Z::kCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if constexpr (!FULL) let_next_start();
  launch_before_ended();
  const uint32_t tmem = sm.tmem;
  const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;  // this warp's lanes

  if (wg == 5) {
    regs_dec<48>();
    // ---- the products: scores, D and the outputs' two from a warp each, so that none
    // waits for what only another one needs
    if (warp == 20 || warp == 22 || warp == 23) {
      constexpr uint32_t kIdSc = tc::idesc_f16(kBF16, 64, 64, false, false);
      constexpr uint32_t kIdO2 = tc::idesc_f16(kBF16, DV, 64, false, false);
      constexpr uint32_t kIdD = tc::idesc_f16(kBF16, DV, DK, true, true);
      const uint32_t sp = smem_addr(sm.p[0]), swv = smem_addr(sm.wv[0]);
      auto at_k = [](int kk) { return (uint32_t)(kk / 4 * kTile + kk % 4 * 32); };
      for (int n = 0; FULL || warp == 22; ++n) {
        const int st = n % kStages;
        if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1)) break;
        if (__any_sync(0xffffffffu, sm.chunk[st].stop)) break;
        const uint32_t q = smem_addr(sm.stage[st]), k = q + Z::kQ, v = k + Z::kQ;
        if (warp == 20) {
          if (n > 1 && !warp_wait(sm, g.err, &sm.sc_free[n & 1], ((n >> 1) - 1) & 1)) break;
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma(tmem + Z::kSc + (n & 1) * 64, rows_mn(q + at_k(kk)), rows_mn(k + at_k(kk)), kIdSc,
                kk);
          commit(smem_addr(&sm.sc_full[n & 1]));
        } else if (warp == 22) {
          // D, ahead of S: all that it waits for is the reading of the D before
          bool dead = n > 0 && !warp_wait(sm, g.err, &sm.d_free, (n - 1) & 1);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {  // half of the tokens
            dead = dead || !warp_wait(sm, g.err, &sm.wv_ready[hh], n & 1);
            tc::fence_after_sync();
#pragma unroll
            for (int i = 0; i < 2 * PARTS; ++i) {
              const int part = i >> 1, kk = 2 * hh + (i & 1);
              mma(tmem + Z::kD, rows_k(swv + part * Z::kV + kk * 2048), rows_k(k + kk * 2048), kIdD,
                  part | kk);
            }
            commit(smem_addr(&sm.wv_free[hh]));
          }
          if (dead) break;
          commit(smem_addr(&sm.d_full));
        } else {
          if (!warp_wait(sm, g.err, &sm.s_ready, n & 1)) break;
          if (n > 0 && !warp_wait(sm, g.err, &sm.o_free, (n - 1) & 1)) break;
          tc::fence_after_sync();
#pragma unroll
          for (int i = 0; i < DK / 8; ++i)  // the high parts, then the remainders
            mma_ta(tmem + Z::kO2, tmem + Z::kS + i * 8, rows_mn(q + at_k(i % (DK / 16))), kIdO2, i);
          commit(smem_addr(&sm.s_free));
          // values that are not finite are out of V by then
          if (!warp_wait(sm, g.err, &sm.v_ready[st], (n / kStages) & 1)) break;
          if (!warp_wait(sm, g.err, &sm.p_ready, n & 1)) break;
          tc::fence_after_sync();
          // tokens before s take nothing from it: the first 16 kk columns are done
#pragma unroll
          for (int i = 0; i < kC / 8; ++i) {
            const int part = i >> 2, kk = i & 3;
            mma(tmem + Z::kO1 + 16 * kk, rows_k(v + kk * 2048),
                rows_mn(sp + part * Z::kP + kk * 2048 + kk * 32),
                tc::idesc_f16(kBF16, DV, kC - 16 * kk, true, false), i);
          }
          commit(smem_addr(&sm.p_free));
          commit(smem_addr(&sm.o_full));
        }
        commit(smem_addr(&sm.empty[st]));
      }
      if (FULL || warp == 22) {
        // nothing is in flight any more when the tensor memory is given back
        commit(smem_addr(&sm.fin));
        const uint64_t t0 = ssu::global_ns();
        while (!mbar_test(&sm.fin, 0) && ssu::global_ns() - t0 < ssu::kWaitLimitNs) {
        }
      }
      __syncwarp();
    } else if (warp == 21) {
      // ---- copies and tables -----------------------------------------------
      const int items = g.head->count[LIST] * p.H;
      int n = 0;
      bool live = true;
      int next = 0;
      if (lane == 0) next = atomicAdd(&g.head->next[LIST], 1);
      while (live) {
        const int item = __shfl_sync(0xffffffffu, next, 0);
        if (item >= items) break;
        if (lane == 0) next = atomicAdd(&g.head->next[LIST], 1);  // on its way during this item
        const Piece piece = g.pieces[LIST][item / p.H];
        const int h = item % p.H, grp = h / p.hr;
        const int chunks = (piece.len + kC - 1) / kC;
        auto decay_at = [&](int t) {
          return p.ld && t < piece.len ? p.ld[(int64_t)(piece.r0 + t) * p.ld_rs + h * p.ld_hs]
                                       : 0.0f;
        };
        float l0 = decay_at(2 * lane), l1 = decay_at(2 * lane + 1);
        double whole = 0.0;  // log2 of what the piece decays a state by
        for (int c = 0; c < chunks; ++c, ++n) {
          const int st = n % kStages;
          const int t0 = c * kC, rows = min(kC, piece.len - t0);
          // A log decay below -320 (in units of log2) is held there: a decay of zero in fp32,
          // also where the chunk's other rows grow by all that fp32 has room for.
          auto held = [](float l) {
            l *= kLog2e;
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(l) : "f"(-320.0f));
            return l;
          };
          const float d0 = held(l0), d1 = held(l1);
          l0 = decay_at(t0 + kC + 2 * lane);
          l1 = decay_at(t0 + kC + 2 * lane + 1);
          // a_t in 64 bits, so that differences of large sums keep their digits: in units of
          // 2^-44 (sums of doubles took this warp twice the time of a chunk's products), or
          // as doubles where the batch has something that these do not hold
          float2 two0, two1;            // a_t
          float x0, x1, w0, w1, end;    // r - a_t; a_C - a_t; a_C
          [[maybe_unused]] double exact;      // a_C
          auto sums = [&](auto e0, auto e1, float unit) {
            auto inc = e0 + e1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const auto u = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += u;
            }
            const auto all = __shfl_sync(0xffffffffu, inc, 31);
            const auto ref = __shfl_sync(0xffffffffu, inc, lane | 7);
            const auto before = inc - e1;
            two0 = in_two(before);
            two1 = in_two(inc);
            x0 = (float)(ref - before) * unit;
            x1 = (float)(ref - inc) * unit;
            w0 = (float)(all - before) * unit;
            w1 = (float)(all - inc) * unit;
            end = (float)all * unit;
            if constexpr (!FULL) exact = (double)all * (double)unit;
          };
          if (__all_sync(0xffffffffu, d0 <= 4096.0f && d1 <= 4096.0f))
            sums(__float2ll_rn(d0 * 0x1p44f), __float2ll_rn(d1 * 0x1p44f), 0x1p-44f);
          else
            sums((double)d0, (double)d1, 1.0f);
          // all of it before the stage is free
          const int t = 2 * lane;
          const float2 x = make_float2(ex2(x0), ex2(x1));
          const float a0 = two0.x + two0.y, a1 = two1.x + two1.y;
          const float2 ea = make_float2(p.scale * ex2(a0), p.scale * ex2(a1));
          const float2 w = make_float2(t < rows ? ex2(w0) : 0.0f, t + 1 < rows ? ex2(w1) : 0.0f);
          const bool mild = __all_sync(0xffffffffu, x0 >= -60.0f && x0 <= 1.0f && x1 >= -60.0f &&
                                                        x1 <= 1.0f && fabsf(a0) <= 128.0f &&
                                                        fabsf(a1) <= 128.0f);
          // near 1 the decay is 1 + add: rounded by itself it would be off by the same
          // 2^-25 chunk after chunk
          const float e = ex2(end);
          if constexpr (!FULL) {
            // summed before the exponential is taken: a product of the chunks' decays would be
            // off by each one's rounding.  What fp32 forgets here it does not remember, whatever
            // a state grows by behind it.
            whole += exact;
            if (e == 0.0f || whole < -320.0) whole = -INFINITY;
            if (c == chunks - 1 && lane == 0)
              g.decay[(int64_t)(piece.base + piece.j) * p.H + h] = (float)whole;
          }
          const float keep = e > 0.5f ? 1.0f : 0.0f;
          const float add = e > 0.5f ? expm1f(end * 0.693147181f) : e;
          if (n >= kStages && !warp_wait(sm, g.err, &sm.empty[st], (n / kStages - 1) & 1)) {
            live = false;
            break;
          }
          if (lane == 0) {
            const uint32_t q = smem_addr(sm.stage[st]), k = q + Z::kQ, v = k + Z::kQ;
            const uint32_t bar = smem_addr(&sm.full[st]);
            ssu::mbar_arrive_expect_tx(&sm.full[st], FULL ? Z::kStage : Z::kStage - Z::kQ);
#pragma unroll
            for (int i = 0; i < DK / 64; ++i) {
              if (FULL) load_box(q + i * kTile, &g.q, bar, 64 * i, grp, piece.r0 + t0);
              load_box(k + i * kTile, &g.k, bar, 64 * i, grp, piece.r0 + t0);
            }
#pragma unroll
            for (int i = 0; i < DV / 64; ++i)
              load_box(v + i * kTile, &g.v, bar, 64 * i, h, piece.r0 + t0);
            sm.chunk[st] = Chunk{h, piece.r0 + t0, rows, c == 0, c == chunks - 1, 0, piece};
          }
          Tables& tab = sm.tab[st];
          *reinterpret_cast<float2*>(tab.a + t) = make_float2(a0, a1);
          *reinterpret_cast<float4*>(tab.two + t) = make_float4(two0.x, two0.y, two1.x, two1.y);
          *reinterpret_cast<float2*>(tab.x + t) = x;
          *reinterpret_cast<float2*>(tab.ea + t) = ea;
          *reinterpret_cast<float2*>(tab.w + t) = w;
          if ((lane & 7) == 7) tab.r[lane / 8] = a1;
          if (lane == 0) {
            tab.keep = keep;
            tab.add = add;
            tab.mild = mild;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[st]);
        }
      }
      if (live && lane == 0) {
        const int st = n % kStages;
        if (n < kStages || wait(sm, g.err, &sm.empty[st], (n / kStages - 1) & 1)) {
          sm.chunk[st].stop = 1;
          mbar_arrive(&sm.full[st]);
          mbar_arrive(&sm.full[st]);
        }
      }
      __syncwarp();
    }
  } else if (wg == 0) {
    regs_dec<64>();
    if constexpr (FULL) {
      // ---- P: rows 16 warp + r and r + 8, r = lane / 4; columns 2 (lane % 4) and the next of
      // each eight -------------------------------------------------------------
      const int r = lane >> 2, cc = 2 * (lane & 3);
      const int t0 = 16 * warp + r, t1 = t0 + 8;
      // where this lane's row of the four matrices of 16 x 16 values goes
      const int mrow = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), mpiece = lane >> 4;
      for (int n = 0;; ++n) {
        const int st = n % kStages;
        if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
        const Tables& tab = sm.tab[st];
        const float a0 = tab.a[t0], a1 = tab.a[t1];
        const bool mild = tab.mild;
        if (!warp_wait(sm, g.err, &sm.sc_full[n & 1], (n >> 1) & 1)) break;
        if (kBF16 && n > 0 && !warp_wait(sm, g.err, &sm.p_free, (n - 1) & 1)) break;
        tc::fence_after_sync();
        // 16 columns: scale e^(a_t - a_s) q_t . k_s, 0 above the diagonal
        auto weighed = [&](auto mild, int b, float2 (&y)[4]) {
          float s[8];
          ld_frag2(tmem + quad + Z::kSc + (n & 1) * 64 + 16 * b, s);
          float u0, u1;
          float2 r0, r1;
          if constexpr (mild) {
            u0 = p.scale * ex2(a0 - tab.r[b]), u1 = p.scale * ex2(a1 - tab.r[b]);
          } else {
            r0 = tab.two[t0], r1 = tab.two[t1];
          }
          tc::wait_ld();
#pragma unroll
          for (int f = 0; f < 2; ++f) {  // 8 columns
            const int c = 16 * b + 8 * f + cc;
            float2 e0, e1;
            if constexpr (mild) {
              const float2 x = *reinterpret_cast<const float2*>(tab.x + c);
              e0 = __fmul2_rn(x, make_float2(u0, u0));
              e1 = __fmul2_rn(x, make_float2(u1, u1));
            } else {
              const float4 x = *reinterpret_cast<const float4*>(tab.two + c);
              const float2 c0 = make_float2(x.x, x.y), c1 = make_float2(x.z, x.w);
              e0 = make_float2(p.scale * ex2(between(r0, c0)), p.scale * ex2(between(r0, c1)));
              e1 = make_float2(p.scale * ex2(between(r1, c0)), p.scale * ex2(between(r1, c1)));
            }
            float2 &y0 = y[2 * f], &y1 = y[2 * f + 1];
            y0 = __fmul2_rn(make_float2(s[4 * f], s[4 * f + 1]), e0);
            y1 = __fmul2_rn(make_float2(s[4 * f + 2], s[4 * f + 3]), e1);
            if (b == warp) {
              if (c > t0) y0.x = 0.0f;
              if (c + 1 > t0) y0.y = 0.0f;
              if (c > t1) y1.x = 0.0f;
              if (c + 1 > t1) y1.y = 0.0f;
            }
          }
        };
        auto leave = [&](int b, float2 (&y)[4]) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hi[i] = part<IT>(y[i]);
            lo[i] = pack2<IT>(y[i].x, y[i].y);
          }
          const uint32_t to = smem_addr(sm.p[0]) + tile_at(mrow, 2 * b + mpiece);
          st_frags<false>(to, hi);
          st_frags<false>(to + Z::kP, lo);
        };
        if constexpr (kBF16) {
#pragma unroll 1
          for (int b = 0; b <= warp; ++b) {
            float2 y[4];
            if (mild) weighed(std::true_type{}, b, y);
            else weighed(std::false_type{}, b, y);
            leave(b, y);
          }
        } else {
          float2 y[4][4];
          float m0 = 0.0f, m1 = 0.0f;
          auto all = [&](auto kind) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (b > warp) continue;
              weighed(kind, b, y[b]);
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                m0 = fmaxf(m0, fmaxf(fabsf(y[b][2 * f].x), fabsf(y[b][2 * f].y)));
                m1 = fmaxf(m1, fmaxf(fabsf(y[b][2 * f + 1].x), fabsf(y[b][2 * f + 1].y)));
              }
            }
          };
          if (mild) all(std::true_type{});
          else all(std::false_type{});
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
          }
          float back0, back1;
          const float by0 = toward(m0, 10, &back0), by1 = toward(m1, 10, &back1);
          if (n > 0 && !warp_wait(sm, g.err, &sm.p_free, (n - 1) & 1)) break;
          if ((lane & 3) == 0) {
            sm.p_scale[n & 1][t0] = back0;
            sm.p_scale[n & 1][t1] = back1;
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (b > warp) continue;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              y[b][2 * f] = __fmul2_rn(y[b][2 * f], make_float2(by0, by0));
              y[b][2 * f + 1] = __fmul2_rn(y[b][2 * f + 1], make_float2(by1, by1));
            }
            leave(b, y[b]);
          }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.sc_free[n & 1]);
          mbar_arrive(&sm.p_ready);
        }
      }
    }
  } else if (wg == 1) {
    regs_dec<64>();
    if constexpr (FULL) {
      // ---- outputs: o^T's rows are channels; turned in shared memory -----------
      const int w = warp & 3, r = lane >> 2, cc = 2 * (lane & 3);
      constexpr int SEG = ROWS / 8;  // 16-byte pieces of a token's row that a warp writes
      const bool vec = p.o_vec;
      uint32_t met = 0;
      bool dead = false;
      for (int n = 0; !dead; ++n) {
        const int st = n % kStages;
        if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
        const int rows = sm.chunk[st].rows;
        IT* out = static_cast<IT*>(p.out) + (int64_t)sm.chunk[st].r0 * p.o_rs +
                  sm.chunk[st].h * p.o_hs;
        unsigned char* turn = Z::kOut ? sm.out : sm.stage[st];
        const Tables& tab = sm.tab[st];
        if (!warp_wait(sm, g.err, &sm.o_full, n & 1)) break;
        tc::fence_after_sync();
        const int any = sm.any_bad[st];
#pragma unroll 1
        for (int i = 0; i < ROWS / 16 * 2; ++i) {  // 16 channels, 32 tokens
          const int lh = i >> 1, c0 = (i & 1) * 32, ch = ROWS * w + 16 * lh;
          float back0 = 1.0f, back1 = 1.0f;
          if constexpr (!kBF16) {
            back0 = sm.row_scale[n & 1][ch + r];
            back1 = sm.row_scale[n & 1][ch + r + 8];
          }
          float o1[16], o2[16];
          ld_frag4(tmem + quad + ((uint32_t)(16 * lh) << 16) + Z::kO1 + c0, o1);
          ld_frag4(tmem + quad + ((uint32_t)(16 * lh) << 16) + Z::kO2 + c0, o2);
          tc::wait_ld();
          uint32_t y[8];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int c = c0 + 8 * f + cc;
            const float2 e = *reinterpret_cast<const float2*>(tab.ea + c);
            const float2 b0 = kBF16 ? e : make_float2(e.x * back0, e.y * back0);
            const float2 b1 = kBF16 ? e : make_float2(e.x * back1, e.y * back1);
            float2 v0 = make_float2(o1[4 * f], o1[4 * f + 1]);
            float2 v1 = make_float2(o1[4 * f + 2], o1[4 * f + 3]);
            if constexpr (!kBF16) {
              const float2 back = *reinterpret_cast<const float2*>(&sm.p_scale[n & 1][c]);
              v0 = __fmul2_rn(v0, back);
              v1 = __fmul2_rn(v1, back);
            }
            v0 = __ffma2_rn(make_float2(o2[4 * f], o2[4 * f + 1]), b0, v0);
            v1 = __ffma2_rn(make_float2(o2[4 * f + 2], o2[4 * f + 3]), b1, v1);
            y[2 * f] = pack2<IT>(v0.x, v0.y);
            y[2 * f + 1] = pack2<IT>(v1.x, v1.y);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // 16 tokens x 16 channels
            const int t = c0 + 16 * k + (lane >> 4) * 8 + (lane & 7);
            const uint32_t four[4] = {y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]};
            st_frags<true>(smem_addr(turn) + tile_at(t, ch / 8 + ((lane >> 3) & 1)), four);
          }
        }
        if (any) {
          __syncwarp();
          if (lane < ROWS) {
            const int ch = ROWS * w + lane;
#pragma unroll 1
            for (int t = sm.bad[st][ch]; t < kC; ++t)
              reinterpret_cast<IT*>(turn + tile_at(t, ch / 8))[ch % 8] = from_f<IT>(NAN);
            sm.bad[st][ch] = kC;
          }
          if (!meet(sm, g.err, &sm.out_warps, met)) dead = true;  // all have looked at any_bad
          if (w == 0 && lane == 0) sm.any_bad[st] = 0;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free);
        // the warp's channels of every token: 16 bytes a lane
#pragma unroll 4
        for (int i = 0; i < kC * SEG / 32; ++i) {
          const int t = (i * 32 + lane) / SEG, piece = w * SEG + lane % SEG;
          const uint4 y = *reinterpret_cast<const uint4*>(turn + tile_at(t, piece));
          if (t >= rows) continue;
          IT* to = out + t * p.o_rs + piece * 8;
          if (vec) {
            *reinterpret_cast<uint4*>(to) = y;
          } else {
            const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(u[e >> 1] >> (e & 1 ? 16 : 0));
          }
        }
        tc::fence_proxy_async();  // the stage is filled by copies again
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);
      }
    }
  } else if (wg == 4) {
    regs_dec<64>();
    // ---- w V ---------------------------------------------------------------
    const int w4 = warp & 3;  // pieces w4, w4 + 4, ... of a token's row
    uint32_t met = 0;
    for (int n = 0;; ++n) {
      const int st = n % kStages;
      if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
      const int rows = sm.chunk[st].rows;
      unsigned char* k = sm.stage[st] + Z::kQ;
      unsigned char* v = k + Z::kQ;
      bool dead = false;
      float by = 1.0f;
      if constexpr (!kBF16) {
        // the largest finite |w v| of the chunk comes to 2^14
        float m = 0.0f;
#pragma unroll
        for (int s = lane; s < kC; s += 32) {
          __half2 top{};
#pragma unroll
          for (int i = 0; i < DV / 32; ++i) {
            const uint4 raw = *reinterpret_cast<const uint4*>(v + tile_at(s, 4 * i + w4));
            const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&u[e])));
          }
          if (s < rows) m = fmaxf(m, sm.tab[st].w[s] * fmaxf(__low2float(top), __high2float(top)));
        }
        uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (most == 0x7f800000u) {
          // the channel of an infinite value is lost (below); the others keep their scale
          m = 0.0f;
#pragma unroll 1
          for (int j = lane; j < rows * (DV / 4); j += 32) {
            const int s = j / (DV / 4), i = j % (DV / 4);
            const float x = fabsf(__half2float(*reinterpret_cast<const __half*>(
                v + tile_at(s, 4 * (i / 8) + w4) + i % 8 * 2)));
            if (x < INFINITY) m = fmaxf(m, sm.tab[st].w[s] * x);
          }
          most = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        }
        if (lane == 0) sm.v_max[st][w4] = most;
        if (!meet(sm, g.err, &sm.v_warps, met)) dead = true;
        m = __uint_as_float(max(max(sm.v_max[st][0], sm.v_max[st][1]),
                                max(sm.v_max[st][2], sm.v_max[st][3])));
        float back;
        by = toward(m, 14, &back);
        // D of the chunk that had this stage before is read: the products two chunks on are done
        if (n > 0 && !warp_wait(sm, g.err, &sm.wv_free[0], (n - 1) & 1)) dead = true;
        if (w4 == 0 && lane == 0) sm.v_scale[st] = back;
      }
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {
        const int s = 32 * hh + lane;  // the token whose pieces this thread takes
        const float w = sm.tab[st].w[s] * by;
        if (n > 0 && !warp_wait(sm, g.err, &sm.wv_free[hh], (n - 1) & 1)) dead = true;
        if (rows < kC && s >= rows) {
          // another sequence's rows: zeros, which leave D alone whatever they held
#pragma unroll 1
          for (int i = w4; i < DK / 8; i += 4)
            *reinterpret_cast<uint4*>(k + tile_at(s, i)) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
          for (int i = w4; i < DV / 8; i += 4)
            *reinterpret_cast<uint4*>(v + tile_at(s, i)) = make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t odd = 0;
#pragma unroll 2
        for (int i = 0; i < DV / 32; ++i) {
          const int at = tile_at(s, 4 * i + w4);
          const uint4 raw = *reinterpret_cast<const uint4*>(v + at);
          const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
          uint32_t o[PARTS][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            odd = not_finite<IT>(u[e], odd);
            float2 x = __fmul2_rn(unpack2<IT>(u[e]), make_float2(w, w));
            if constexpr (PARTS == 3) {
              o[0][e] = part_cut(x);
              o[1][e] = part_cut(x);
              o[2][e] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
            } else {
              o[0][e] = part<IT>(x);
              o[1][e] = pack2<IT>(x.x, x.y);
            }
          }
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            *reinterpret_cast<uint4*>(sm.wv[q] + at) = make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
        }
        if (odd) {
          // A value that is not finite must not reach the tokens before its own, as 0 x
          // infinity would in P V: it is taken out of V, and the outputs of its channel are
          // NaN from its token on, as the state is.
#pragma unroll 1
          for (int c = 0; c < DV / 4; ++c) {
            const int piece = 4 * (c / 8) + w4;
            uint16_t* x = reinterpret_cast<uint16_t*>(v + tile_at(s, piece)) + c % 8;
            const uint32_t e = kBF16 ? 0x7f80u : 0x7c00u;
            if ((*x & e) == e) {
              *x = 0;
              atomicMin(&sm.bad[st][piece * 8 + c % 8], s);
              sm.any_bad[st] = 1;
            }
          }
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.wv_ready[hh]);
      }
      if (lane == 0) mbar_arrive(&sm.v_ready[st]);
      if (dead) break;
    }
  } else {
    regs_inc<120>();
    // ---- S ---------------------------------------------------------------
    const int half = wg - 2;
    const int row = ROWS * (warp & 3) + lane % ROWS;
    float S[HALF];
    uint32_t met = 0;
    bool dead = false;
    // fp16: the largest value of this thread's half of a row, left for the other half's
    // threads; the warps meet when it is looked at
    auto measure = [&](int n) {
      float m[4] = {};
#pragma unroll
      for (int i = 0; i < HALF; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], fabsf(S[i + k]));
      if (lane < ROWS) sm.row_max[n & 1][half][row] = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.state_warps);
    };
    // S as a chunk's operand: columns [c, c + 16), divided by a power of two
    auto operand = [&](int c, float by) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 v = make_float2(S[c + 2 * i], S[c + 2 * i + 1]);
        if (!kBF16) v = __fmul2_rn(v, make_float2(by, by));
        hi[i] = part<IT>(v);
        lo[i] = pack2<IT>(v.x, v.y);
      }
      const uint32_t at = tmem + quad + Z::kS + (half * HALF + c) / 2;
      st_tmem8(at, hi);
      st_tmem8(at + HALF, lo);
    };
    auto given = [&] {
      wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_ready);
    };
    auto give = [&](int n) {
      float by = 1.0f;
      if constexpr (!kBF16) {
        // fp16 has no room for a large S: each row is brought to about 2^10 by a power of two
        if (!warp_wait(sm, g.err, &sm.state_warps, met)) dead = true;
        met ^= 1;
        const float m = fmaxf(sm.row_max[n & 1][0][row], sm.row_max[n & 1][1][row]);
        float back;
        by = toward(m, 10, &back);
        if (half == 0 && lane < ROWS) sm.row_scale[n & 1][row] = back;
      }
#pragma unroll
      for (int c = 0; c < HALF; c += 16) operand(c, by);
      given();
    };
    auto row_of_state = [&](auto* pool, int64_t slot, int h) {
      return pool + ((slot * p.H + h) * DV + row) * DK + half * HALF;
    };
    const bool wide = ((uintptr_t)p.state & 31) == 0;
    auto entry = [&](int e, int h) {  // of the workspace's states; this thread's first four values
      return reinterpret_cast<float4*>(g.state) + ((int64_t)e * p.H + h) * (DV * DK / 4) +
             (half * 4 + (warp & 3)) * (HALF / 4 * ROWS) + lane % ROWS;
    };
    for (int n = 0; !dead; ++n) {
      const int st = n % kStages;
      if (!warp_wait(sm, g.err, &sm.full[st], (n / kStages) & 1) || sm.chunk[st].stop) break;
      const Tables& tab = sm.tab[st];
      const float keep = tab.keep, add = tab.add;
      const bool first = sm.chunk[st].first, last = sm.chunk[st].last;
      Piece pc{};
      int h = 0;
      if (first || last) {
        pc = sm.chunk[st].piece;
        h = sm.chunk[st].h;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);  // all that this warp looks at
      if (first) {
#pragma unroll
        for (int i = 0; i < HALF; ++i) S[i] = 0.0f;
        if (FULL && pc.of > 1) {
          const float4* from = entry(pc.base + pc.j, h);
#pragma unroll
          for (int i = 0; i < HALF / 4; ++i) {
            const float4 v = from[i * ROWS];
            S[4 * i] = v.x;
            S[4 * i + 1] = v.y;
            S[4 * i + 2] = v.z;
            S[4 * i + 3] = v.w;
          }
        } else if (pc.j == 0) {
          const Slot from = load_slot(g.a.src, pc.seq, 0, g.a.idx64);
          const int64_t slot = from.id(pc.seq, g.a.idx64);
          if (from.found && slot_ok(slot, p.pad, p.slots) && (!p.has_init || p.has_init[pc.seq])) {
#pragma unroll
            for (int c = 0; c < HALF; c += 32) {
              if (p.state_dtype == SSU_F32)
                load_row<float, 32>(row_of_state(static_cast<const float*>(p.state), slot, h) + c,
                                    wide, S + c);
              else if (p.state_dtype == SSU_BF16)
                load_row<__nv_bfloat16, 32>(
                    row_of_state(static_cast<const __nv_bfloat16*>(p.state), slot, h) + c, wide, S + c);
              else
                load_row<__half, 32>(row_of_state(static_cast<const __half*>(p.state), slot, h) + c,
                                     wide, S + c);
            }
          }
          if (!FULL && lane < ROWS) {  // the second launch finds it here, whatever is in the slot then
            float4* to = entry(pc.base, h);
#pragma unroll
            for (int i = 0; i < HALF / 4; ++i)
              to[i * ROWS] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
          }
        }
        if constexpr (FULL && !kBF16) measure(n);
      }
      if constexpr (FULL) {
        // o2 of the chunk before has read its S
        if (n > 0 && !warp_wait(sm, g.err, &sm.s_free, (n - 1) & 1)) break;
        tc::fence_after_sync();
        give(n);
      }
      if (!warp_wait(sm, g.err, &sm.d_full, n & 1)) break;
      tc::fence_after_sync();
      float back = 1.0f;
      if constexpr (!kBF16) back = sm.v_scale[st];
#pragma unroll
      for (int c = 0; c < HALF; c += 16) {
        float d[16];
        tc::ld16(tmem + quad + Z::kD + half * HALF + c, d);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 x = make_float2(S[c + i], S[c + i + 1]);
          float2 y = make_float2(d[i], d[i + 1]);
          if constexpr (kBF16)
            y = __ffma2_rn(x, make_float2(keep, keep), y);
          else  // keep is 0 or 1: rounded once, too
            y = __ffma2_rn(y, make_float2(back, back), __fmul2_rn(x, make_float2(keep, keep)));
          y = __ffma2_rn(x, make_float2(add, add), y);
          S[c + i] = y.x;
          S[c + i + 1] = y.y;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.d_free);
      if (!last) {
        if constexpr (FULL && !kBF16) measure(n + 1);
        continue;
      }
      if constexpr (!FULL) {
        if (lane < ROWS) {
          float4* to = entry(pc.base + pc.j + 1, h);
#pragma unroll
          for (int i = 0; i < HALF / 4; ++i)
            to[i * ROWS] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
      } else if (pc.j == pc.of - 1) {
        const Slot from = load_slot(g.a.src, pc.seq, 0, g.a.idx64);
        int64_t to;
        if (from.found && slot_ok(from.id(pc.seq, g.a.idx64), p.pad, p.slots) &&
            write_slot(g.a, pc.seq, 0, p.pad, p.slots, &to) && lane < ROWS) {
          if (p.state_dtype == SSU_F32)
            store_row<float, HALF>(row_of_state(static_cast<float*>(p.state), to, h), wide, S);
          else if (p.state_dtype == SSU_BF16)
            store_row<__nv_bfloat16, HALF>(row_of_state(static_cast<__nv_bfloat16*>(p.state), to, h),
                                           wide, S);
          else
            store_row<__half, HALF>(row_of_state(static_cast<__half*>(p.state), to, h), wide, S);
        }
        __syncwarp();
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 20) tc::dealloc(tmem, Z::kCols);
}

}  // namespace linattn
