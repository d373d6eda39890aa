// layer_scan_prompt.cuh -- the selective scan over prompts.
//
// A CTA takes CH channels of one sequence through its rows, TT at a time: LPC
// lanes share a channel and own NPT of its state columns each, in registers
// for the whole chain.  What a channel needs once per row (dt', dt' x, the D
// and z terms) costs more instructions than a state column does, so each is
// worked out once, by one thread, when a tile is staged: dt' and dt' x go to
// shared memory beside the tile's B and C in fp32; the sums over dstate come
// back through shared memory for the gate and a whole-row store.  The next
// tile's rows are in flight in registers meanwhile.
//
// Four state columns of a channel's row take 8 packed fp32 operations (about 2.3
// cycles each: 18 to 21), 4 exponentials (16 cycles of the special-function
// pipe), two shared memory reads of B and C for two channels and two of dt' and
// dt' x, and a quarter of a staged value.  So neither HBM nor one pipe alone
// bounds it: at 9001 x 4096 rows x 16 in 16 sequences, 192 us, the fp32 pipe is
// busy 52 % of the time, the special-function pipe 39 %, shared memory 58 %, the
// issue slots 66 %; 36 cycles a unit in the full waves, the rest is the tail.
#pragma once

#include "layer_scan.cuh"

namespace layer {

constexpr int kPromptThreads = 128;

// R channels of NPT state columns per thread.
template <int N, int R, int NPT>
struct PromptTile {
  static constexpr int LPC = N / NPT;                        // lanes per channel
  static constexpr int LG = kPromptThreads / LPC;            // groups of such lanes
  static constexpr int CH = R * LG;                          // channels per CTA
  static constexpr int WANT = 8 * N / (R * NPT);             // rows for 8 values a staging thread
  static constexpr int TT = WANT > 32 ? (N > 128 ? 16 : 32) : WANT;  // rows per tile
  static constexpr int TPR = kPromptThreads / TT;            // staging threads per row
  static constexpr int SV = CH >= TPR ? CH / TPR : 1;        // channels per staging thread
  static constexpr int BV = N / TPR;                         // B (and C) columns per staging thread
  static constexpr int TG = LPC < 8 ? LPC : 8;               // rows whose sums are reduced together
  static constexpr int YS = CH + 32 / TG;                    // row stride of the sums
  static constexpr int CPW = 32 / LPC;                       // lane groups per warp

  // A staging thread owns SV neighbouring channels and moves them to and from
  // shared memory four at a time.  With SV = 8 a row there holds the first
  // halves of all threads' channels, then the second: threads side by side are
  // then 16 bytes apart, on distinct banks, where 32 would collide.  The
  // channel at place i of a row, and the place of a thread's f-th four:
  __device__ static __forceinline__ int channel(int i) {
    return SV == 8 ? i % (CH / 2) / 4 * 8 + i / (CH / 2) * 4 + i % 4 : i;
  }
  __device__ static __forceinline__ int place(int thread, int f) {
    return SV == 8 ? f * (CH / 2) + thread * 4 : thread * SV + f * 4;
  }
};

template <class K, int N>
struct alignas(16) PromptSmem {
  // rows of channels in the order of K::channel
  float d[K::TT][K::CH];    // dt'
  float dx[K::TT][K::CH];   // dt' x
  float B[K::TT][N];
  float C[K::TT][N];
  float y[K::TT][K::YS];    // sums over dstate
  float D[K::CH];
  float bias[K::CH];
};

// Sums of G rows over the LPC lanes that share a channel (lanes STRIDE apart,
// the lane's index among them q): at each level a lane keeps half of its rows
// and sends the others, so that it ends up with row `base` alone; levels left
// over once it has one row are plain sums, equal in the lanes that differ in
// the bits of `plain`.
template <int G, int OFF, int STRIDE>
struct GroupSum {
  __device__ static __forceinline__ void run(float* v, int q, int& base, int& plain) {
    if constexpr (OFF > 0) {
      if constexpr (G > 1) {
        const bool upper = (q & OFF) != 0;
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
          const float send = upper ? v[i] : v[G / 2 + i];
          const float keep = upper ? v[G / 2 + i] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, OFF * STRIDE);
        }
        if (upper) base += G / 2;
        GroupSum<G / 2, OFF / 2, STRIDE>::run(v, q, base, plain);
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], OFF * STRIDE);
        plain |= OFF;
        GroupSum<1, OFF / 2, STRIDE>::run(v, q, base, plain);
      }
    }
  }
};

// Four state columns from or to a slot, in the state's type.
__device__ __forceinline__ float4 load_state4(const ScanArgs& p, int64_t at) {
  if (p.state_dtype == SSU_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p.state) + at);
  float f[4];
  if (p.state_dtype == SSU_BF16)
    load_floats<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16*>(p.state) + at, true, f);
  else load_floats<__half, 4>(static_cast<const __half*>(p.state) + at, true, f);
  return make_float4(f[0], f[1], f[2], f[3]);
}

template <class ST>
__device__ __forceinline__ void store_as4(void* state, int64_t at, float2 a, float2 b) {
  Pack<ST, 4> v;
  v.v[0] = from_f<ST>(a.x), v.v[1] = from_f<ST>(a.y);
  v.v[2] = from_f<ST>(b.x), v.v[3] = from_f<ST>(b.y);
  store_pack<ST, 4>(static_cast<ST*>(state) + at, v);
}

__device__ __forceinline__ void store_state4(const ScanArgs& p, int64_t at, float2 a, float2 b) {
  if (p.state_dtype == SSU_F32) store_as4<float>(p.state, at, a, b);
  else if (p.state_dtype == SSU_BF16) store_as4<__nv_bfloat16>(p.state, at, a, b);
  else store_as4<__half>(p.state, at, a, b);
}

// A staging thread's channels in a row of shared memory
template <class K>
__device__ __forceinline__ void from_row(const float* row, int thread, float* f) {
  if constexpr (K::SV % 4 == 0) {
#pragma unroll
    for (int i = 0; i < K::SV / 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(row + K::place(thread, i));
      f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < K::SV; ++i) f[i] = row[thread * K::SV + i];
  }
}

template <class K>
__device__ __forceinline__ void to_row(float* row, int thread, const float* f) {
  if constexpr (K::SV % 4 == 0) {
#pragma unroll
    for (int i = 0; i < K::SV / 4; ++i)
      *reinterpret_cast<float4*>(row + K::place(thread, i)) =
          make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < K::SV; ++i) row[thread * K::SV + i] = f[i];
  }
}

template <int V>
__device__ __forceinline__ void to_shared(float* p, const float* f) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = f[i];
  }
}

// FAST: every row of x, z, dt, B, C and out can be moved in whole vectors.  A
// load is then one instruction that nothing waits for until the next tile is
// staged; a choice between the two kinds of load would be waited for at once.
template <class IT, class DT, int N, int R, int NPT, bool FAST, bool OUT>
struct PromptRows {
  using K = PromptTile<N, R, NPT>;
  static constexpr int SV = K::SV, BV = K::BV;
  Words<IT, SV> x, z;
  Words<DT, SV> dt;
  Words<IT, BV> B, C;
  const IT *xp, *zp, *Bp, *Cp;
  const DT* dp;
  int sn;  // the thread's channels

  // row rt + tr, below r_end
  __device__ __forceinline__ void load(const ScanArgs& p, int rt, int tr, int r_end) {
    const bool in = tr < r_end - rt;
    const int r = in ? rt + tr : r_end - 1;  // beyond: staged as a step that changes nothing
    if constexpr (FAST) {
      x.load(xp + r * p.x_rs);
      if (OUT && p.z) z.load(zp + r * p.z_rs);
      dt.load(dp + r * p.dt_rs);
      B.load(Bp + r * p.B_rs);
      if (OUT) C.load(Cp + r * p.C_rs);
    } else {
      x.load_some(xp + r * p.x_rs, in ? sn : 0);
      if (OUT && p.z) z.load_some(zp + r * p.z_rs, in ? sn : 0);
      dt.load_some(dp + r * p.dt_rs, in ? sn : 0);
      B.load_some(Bp + r * p.B_rs, in ? BV : 0);
      if (OUT) C.load_some(Cp + r * p.C_rs, in ? BV : 0);
    }
  }
};

template <class T, int SV, bool FAST>
__device__ __forceinline__ void store_row(T* o, const float2* y, int n) {
  if constexpr (FAST) {
    Words<T, SV> v;
    v.set(y);
    v.store(o);
  } else {
#pragma unroll
    for (int i = 0; i < SV; ++i)
      if (i < n) o[i] = from_f<T>(i & 1 ? y[i >> 1].y : y[i >> 1].x);
  }
}

// The chain over rows [r0, r_end), its state in h.  OUT false: no sums and no
// outputs, only the state and dsum, the sum of dt' over the rows.
template <class IT, class DT, int N, int R, int NPT, bool FAST, bool OUT>
__device__ __forceinline__ void scan_rows(const ScanArgs& p,
                                          PromptSmem<PromptTile<N, R, NPT>, N>& sm, int g, int c0,
                                          int cn, int r0, int r_end,
                                          const float2 (&A2)[R][NPT / 2],
                                          float2 (&h)[R][NPT / 2], float (&dsum)[R]) {
  using K = PromptTile<N, R, NPT>;
  constexpr int LPC = K::LPC, TT = K::TT, SV = K::SV, BV = K::BV, TG = K::TG;
  constexpr int UG = TG < 8 ? 16 / TG < TT / TG ? 16 / TG : TT / TG : 1;  // groups of TG per pass
  // neighbouring lanes take neighbouring channels and the same columns: a load
  // of B or C then asks for the same 16 bytes in runs of lanes, which shared
  // memory serves in 1.7 cycles (runs of 8) where it takes 4 when every lane's
  // neighbour asks for other ones
  const int tid = threadIdx.x;
  const int q = (tid & 31) / K::CPW, ch = tid / 32 * K::CPW + (tid & 31) % K::CPW;

  // staging: row tr of the tile, channels s0 .. s0 + SV, columns b0 .. b0 + BV
  const int tr = tid / K::TPR, tp = tid % K::TPR;
  const int s0 = tp * SV, b0 = tp * BV;
  PromptRows<IT, DT, N, R, NPT, FAST, OUT> rows;
  rows.sn = s0 < K::CH ? (cn - s0 < SV ? cn - s0 : SV) : 0;
  const int cs = c0 + (rows.sn > 0 ? s0 : 0);  // threads without channels read the CTA's first
  rows.xp = static_cast<const IT*>(p.x) + cs;
  rows.zp = static_cast<const IT*>(p.z) + cs;
  rows.dp = static_cast<const DT*>(p.dt) + cs;
  rows.Bp = static_cast<const IT*>(p.B) + g * p.B_gs + b0;
  rows.Cp = static_cast<const IT*>(p.Cm) + g * p.C_gs + b0;
  rows.load(p, r0, tr, r_end);

  for (int rt = r0; rt < r_end; rt += TT) {
    const int n = r_end - rt < TT ? r_end - rt : TT;
    const bool in = tr < n;
    const Words<IT, SV> xk = rows.x, zk = rows.z;
    // rows beyond the sequence get dt' = 0 and zeros: a step that changes nothing,
    // since no A2 is infinite
    if (s0 < K::CH) {
      float bias[SV], d[SV], dx[SV];
      from_row<K>(sm.bias, tp, bias);
#pragma unroll
      for (int i = 0; i < SV; ++i) d[i] = rows.dt.at(i);
      if (p.softplus) {
        softplus_sums<SV>(d, bias);
      } else {
#pragma unroll
        for (int i = 0; i < SV; ++i) d[i] += bias[i];
      }
#pragma unroll
      for (int i = 0; i < SV; ++i) dx[i] = d[i] * xk.at(i);
      if (!in) {
#pragma unroll
        for (int i = 0; i < SV; ++i) d[i] = dx[i] = 0.0f;
      }
      to_row<K>(sm.d[tr], tp, d);
      to_row<K>(sm.dx[tr], tp, dx);
    }
    {
      float f[BV];
#pragma unroll
      for (int i = 0; i < BV; ++i) f[i] = in ? rows.B.at(i) : 0.0f;
      to_shared<BV>(&sm.B[tr][b0], f);
      if constexpr (OUT) {
#pragma unroll
        for (int i = 0; i < BV; ++i) f[i] = in ? rows.C.at(i) : 0.0f;
        to_shared<BV>(&sm.C[tr][b0], f);
      }
    }
    __syncthreads();
    if (r_end - rt > TT) rows.load(p, rt + TT, tr, r_end);

    for (int t = 0; t < n; t += TG * UG) {
#pragma unroll
      for (int u = 0; u < UG; ++u) {
        float acc[R][TG];
#pragma unroll
        for (int k = 0; k < TG; ++k) {
          const int row = t + u * TG + k;
          float2 sum[R];
          float d[R], dx[R];
#pragma unroll
          for (int m = 0; m < R; ++m) {
            d[m] = sm.d[row][ch + m * K::LG];
            dx[m] = sm.dx[row][ch + m * K::LG];
          }
#pragma unroll
          for (int j = 0; j < NPT / 4; ++j) {
            const float4 b = *reinterpret_cast<const float4*>(&sm.B[row][(j * LPC + q) * 4]);
            float4 c;
            if constexpr (OUT) c = *reinterpret_cast<const float4*>(&sm.C[row][(j * LPC + q) * 4]);
#pragma unroll
            for (int m = 0; m < R; ++m) {
              const float2 d2 = make_float2(d[m], d[m]), dx2 = make_float2(dx[m], dx[m]);
              const float2 e0 = __fmul2_rn(A2[m][2 * j], d2), e1 = __fmul2_rn(A2[m][2 * j + 1], d2);
              h[m][2 * j] = __ffma2_rn(h[m][2 * j], make_float2(ex2(e0.x), ex2(e0.y)),
                                       __fmul2_rn(dx2, make_float2(b.x, b.y)));
              h[m][2 * j + 1] = __ffma2_rn(h[m][2 * j + 1], make_float2(ex2(e1.x), ex2(e1.y)),
                                           __fmul2_rn(dx2, make_float2(b.z, b.w)));
              if constexpr (!OUT) continue;
              sum[m] = j == 0 ? __fmul2_rn(h[m][0], make_float2(c.x, c.y))
                              : __ffma2_rn(h[m][2 * j], make_float2(c.x, c.y), sum[m]);
              sum[m] = __ffma2_rn(h[m][2 * j + 1], make_float2(c.z, c.w), sum[m]);
            }
          }
#pragma unroll
          for (int m = 0; m < R; ++m) {
            if constexpr (OUT) acc[m][k] = sum[m].x + sum[m].y;
            else dsum[m] += d[m];
          }
        }
#pragma unroll
        for (int m = 0; m < R && OUT; ++m) {
          int base = 0, plain = 0;
          GroupSum<TG, LPC / 2, K::CPW>::run(acc[m], q, base, plain);
          if ((q & plain) == 0) sm.y[t + u * TG + base][ch + m * K::LG] = acc[m][0];
        }
      }
    }
    __syncthreads();

    if (OUT && in && rows.sn > 0) {
      constexpr int P = (SV + 1) / 2;
      float f[2 * P], D[2 * P];
      from_row<K>(sm.y[tr], tp, f);
      from_row<K>(sm.D, tp, D);
      if (SV & 1) f[SV] = D[SV] = 0.0f;
      float2 y[P];
#pragma unroll
      for (int i = 0; i < P; ++i)
        y[i] = __ffma2_rn(make_float2(D[2 * i], D[2 * i + 1]), xk.pair(i),
                          make_float2(f[2 * i], f[2 * i + 1]));
      if (p.z) {
#pragma unroll
        for (int i = 0; i < P; ++i) y[i] = __fmul2_rn(y[i], silu2(zk.pair(i)));
      }
      const int64_t o = (int64_t)(rt + tr) * p.o_rs + c0 + s0;
      if (p.out_f32) store_row<float, SV, FAST>(static_cast<float*>(p.out) + o, y, rows.sn);
      else store_row<IT, SV, FAST>(static_cast<IT*>(p.out) + o, y, rows.sn);
    }
  }
}

// A long sequence of few channels leaves most of the GPU idle, so its rows are
// split over the K CTAs of a cluster.  Every CTA but the first carries zeros
// through its piece (no outputs), which with the sum of its dt' says what the
// piece does to any state that enters:
//     h_leave = exp(A sum dt') h_enter + h_from_zero;
// the first meanwhile finishes its piece from the true state.  Then each CTA
// folds the pieces in front of its own, read from its neighbours' shared
// memory, and runs its piece for the outputs.  All pieces but the first and the
// last pay for their exponentials twice: 1.7 passes over the rows with 7 pieces.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// float at the address `p` of this CTA's shared memory, in the CTA of rank `rank`
__device__ __forceinline__ float peer_float(const float* p, int rank) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  uint32_t there;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
  return v;
}

// The factor 2^(3 e) that a piece puts on the state that enters it may leave
// fp32's range though the product does not: a state of 0 stays 0 through a piece
// that grows, a large one survives a piece that decays below 2^-126.  So it goes
// on as three factors 2^e, held to [2^-126, 2^127]: they reach from the smallest
// fp32 to the largest, and each product lies between the state and the result.
__device__ __forceinline__ float third_of_decay(float e) {
  float f = ex2(e);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(f) : "f"(0x1p-126f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(f) : "f"(0x1p127f));
  return f;
}

// What a CTA's piece does, for the CTAs behind it.
template <int R, int NPT>
struct PromptPiece {
  float h[R * NPT][kPromptThreads];
  float dsum[R][kPromptThreads];
};

constexpr int kMostPieces = 16, kLeastPieces = 4;
constexpr int kPieceTiles = 3;  // tiles of rows that a piece has at least

// First row of piece k of K, in tiles: the first piece is shorter by the work
// that the others do twice (a pass without outputs costs about 0.7 of one with).
__device__ __forceinline__ int piece_start(int tiles, int k, int K) {
  if (k == 0) return 0;
  if (k == K) return tiles;
  return (int)(((k - 1) + 0.7f) / ((K - 1) + 0.7f) * (float)tiles);
}

// CTAs start in the order of their index: with the longest sequences first the
// short ones fill the gaps that they leave at the end (16 sequences of 300 to
// 900 rows x 4096 channels, 1.7 waves: 236 us in the
// order given, 203 us so).  The sequence of rank `rank`
// by length, where there are at most kRanked.
constexpr int kRanked = 128;

__device__ __forceinline__ int by_length(const Seqs& a, int rank, int* lens) {
  static_assert(kRanked == kPromptThreads, "a thread per sequence");
  const int i = threadIdx.x;
  if (i < a.n) {
    const RawIndex b = load_index(a.cu, i, a.meta64), e = load_index(a.cu, i + 1, a.meta64);
    lens[i] = clamped(e.value(a.meta64), a.rows) - clamped(b.value(a.meta64), a.rows);
  }
  __syncthreads();
  int before = 0;
  if (i < a.n)
    for (int j = 0; j < a.n; ++j) before += lens[j] > lens[i] || (lens[j] == lens[i] && j < i);
  __shared__ int pick;
  if (i < a.n && before == rank) pick = i;
  __syncthreads();
  return pick;
}

template <class IT, class DT, int N, int R, int NPT, bool SPLIT>
__global__ void __launch_bounds__(kPromptThreads, 4)
    scan_prompt_kernel(const ScanArgs p, const Seqs a, int K_) {
  using K = PromptTile<N, R, NPT>;
  constexpr int LPC = K::LPC, TT = K::TT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  PromptSmem<K, N>& sm = *reinterpret_cast<PromptSmem<K, N>*>(smem_raw);
  PromptPiece<R, NPT>& piece = *reinterpret_cast<PromptPiece<R, NPT>*>(smem_raw + sizeof sm);

  const int tid = threadIdx.x;
  const int pieces = SPLIT ? K_ : 1, rank = SPLIT ? (int)(blockIdx.x % pieces) : 0;
  const int tile = blockIdx.x / pieces;
  const int per = p.C / p.G, tiles = (per + K::CH - 1) / K::CH;
  const int g = tile / tiles;                             // the CTA's channels are of one group
  const int c0 = g * per + (tile - g * tiles) * K::CH;
  const int cn = (g + 1) * per - c0;                      // channels from c0 to the group's end
  const int q = (tid & 31) / K::CPW;                      // which of a channel's lanes
  const int ch = tid / 32 * K::CPW + (tid & 31) % K::CPW;  // places ch + k LG, k < R
  float2 A2[R][NPT / 2];                                  // columns (j LPC + q) 4 + i; A log2 e
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = K::channel(ch + k * K::LG);
#pragma unroll
    for (int j = 0; j < NPT / 4; ++j) {
      float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (c < cn)
        load_floats<float, 4>(p.A + (int64_t)(c0 + c) * p.A_rs + (j * LPC + q) * 4, p.a_vec, f);
      A2[k][2 * j] = make_float2(log2_rate(f[0]), log2_rate(f[1]));
      A2[k][2 * j + 1] = make_float2(log2_rate(f[2]), log2_rate(f[3]));
    }
  }
  for (int i = tid; i < K::CH; i += kPromptThreads) {
    const int c = K::channel(i);
    sm.D[i] = p.D && c < cn ? p.D[c0 + c] : 0.0f;
    sm.bias[i] = p.bias && c < cn ? p.bias[c0 + c] : 0.0f;
  }
  __syncthreads();
  const bool fast = p.rows_vec && cn % K::SV == 0;

  const bool ranked = !SPLIT && a.n > 1 && a.n <= kRanked;
  for (int y = blockIdx.y; y < a.n; y += gridDim.y) {
    const int s = ranked ? by_length(a, y, reinterpret_cast<int*>(sm.d)) : y;
    const Item it = packed_item(a, s, p.pad, p.slots);
    if (it.len == 0) continue;
    const bool from = it.read_ok && (!p.has_init || p.has_init[s]);
    // a shorter sequence has fewer pieces; one of few tiles is left whole to the
    // cluster's first CTA
    const int row_tiles = (it.len + TT - 1) / TT;
    const int use = row_tiles / kPieceTiles < pieces ? row_tiles / kPieceTiles : pieces;
    const bool split = SPLIT && use >= kLeastPieces;
    if (SPLIT && !split && rank > 0) continue;
    if (SPLIT && split && rank >= use) {  // no piece: only the cluster's two barriers
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
      continue;
    }
    int r0 = it.r0, r_end = it.r0 + it.len;
    if (split) {
      if (rank < use - 1) r_end = r0 + piece_start(row_tiles, rank + 1, use) * TT;
      r0 += piece_start(row_tiles, rank, use) * TT;
    }
    float2 h[R][NPT / 2];
    float dsum[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      dsum[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < NPT / 4; ++j) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int c = K::channel(ch + k * K::LG);
        if (from && c < cn && rank == 0)
          v = load_state4(p, (it.src * p.C + c0 + c) * N + (j * LPC + q) * 4);
        h[k][2 * j] = make_float2(v.x, v.y);
        h[k][2 * j + 1] = make_float2(v.z, v.w);
      }
    }
    auto rows = [&](auto out) {
      constexpr bool OUT = decltype(out)::value;
      if (fast) scan_rows<IT, DT, N, R, NPT, true, OUT>(p, sm, g, c0, cn, r0, r_end, A2, h, dsum);
      else scan_rows<IT, DT, N, R, NPT, false, OUT>(p, sm, g, c0, cn, r0, r_end, A2, h, dsum);
    };
    if constexpr (SPLIT) {
      if (split) {
        if (rank > 0 && rank < use - 1) rows(std::false_type{});
        if (rank == 0) rows(std::true_type{});
        if (rank < use - 1) {
#pragma unroll
          for (int k = 0; k < R; ++k) {
            piece.dsum[k][tid] = dsum[k];
#pragma unroll
            for (int j = 0; j < NPT / 2; ++j) {
              piece.h[k * NPT + 2 * j][tid] = h[k][j].x;
              piece.h[k * NPT + 2 * j + 1][tid] = h[k][j].y;
            }
          }
        }
        cluster_arrive();
        cluster_wait();
        if (rank > 0) {
#pragma unroll
          for (int k = 0; k < R; ++k)
#pragma unroll
            for (int j = 0; j < NPT / 2; ++j)
              h[k][j] = make_float2(peer_float(&piece.h[k * NPT + 2 * j][tid], 0),
                                    peer_float(&piece.h[k * NPT + 2 * j + 1][tid], 0));
          for (int b = 1; b < rank; ++b) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
              const float d = peer_float(&piece.dsum[k][tid], b) * (1.0f / 3.0f);
#pragma unroll
              for (int j = 0; j < NPT / 2; ++j) {
                const float fx = third_of_decay(A2[k][j].x * d), fy = third_of_decay(A2[k][j].y * d);
                h[k][j].x = fmaf(h[k][j].x * fx * fx, fx, peer_float(&piece.h[k * NPT + 2 * j][tid], b));
                h[k][j].y = fmaf(h[k][j].y * fy * fy, fy, peer_float(&piece.h[k * NPT + 2 * j + 1][tid], b));
              }
            }
          }
        }
        cluster_arrive();  // the neighbours' pieces have been read
        if (rank > 0) rows(std::true_type{});
        cluster_wait();    // ... by all: this CTA's may be written again, and the CTA may end
      } else {
        rows(std::true_type{});
      }
    } else {
      rows(std::true_type{});
    }
    int64_t slot;
    if ((!split || rank == use - 1) && it.read_ok && !p.disable &&
        write_slot(a, s, 0, p.pad, p.slots, &slot)) {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int j = 0; j < NPT / 4; ++j) {
          const int c = K::channel(ch + k * K::LG);
          if (c < cn)
            store_state4(p, (slot * p.C + c0 + c) * N + (j * LPC + q) * 4, h[k][2 * j],
                         h[k][2 * j + 1]);
        }
    }
  }
}

template <class IT, class DT, int N, int R, int NPT, bool SPLIT>
cudaError_t launch_prompt_as(const ScanArgs& p, const Seqs& a, int64_t tiles,
                             int pieces, cudaStream_t stream) {
  using K = PromptTile<N, R, NPT>;
  auto kern = scan_prompt_kernel<IT, DT, N, R, NPT, SPLIT>;
  const int smem = (int)(sizeof(PromptSmem<K, N>) + (SPLIT ? sizeof(PromptPiece<R, NPT>) : 0));
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  if (pieces > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * pieces), (unsigned)(a.n < 65535 ? a.n : 65535));
  cfg.blockDim = dim3(kPromptThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = pieces;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = SPLIT ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, a, pieces);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class IT, class DT, int N, int R, int NPT>
cudaError_t launch_scan_prompt(const ScanArgs& p, const Seqs& a,
                               cudaStream_t stream) {
  using K = PromptTile<N, R, NPT>;
  const int per = p.C / p.G;
  const int64_t tiles = (int64_t)p.G * ((per + K::CH - 1) / K::CH);
  if (tiles * 8 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // Pieces while they fit in one wave of four CTAs an SM (12289 rows in one
  // sequence: 5120 channels, 80 CTAs whole 1014 us, in 4 pieces 812, 7 pieces
  // 592, 8 pieces, which do not fit, 660; 1536 channels in 8 pieces 312 us, 16
  // pieces 253).  Three gain little (12000 rows x 5120 channels in two sequences
  // 722 us for 740 whole), and a piece takes a few tiles to pay for the barriers
  // (512 rows x 5120: 35 us in 16 pieces of 2 tiles, 54 us in 4 of 8).
  const int64_t fit = 4LL * ssu::sm_count() / (tiles * a.n);
  const int pieces = fit < kMostPieces ? (int)fit : kMostPieces;
  if (pieces >= kLeastPieces && a.rows / a.n >= kLeastPieces * kPieceTiles * K::TT)
    return launch_prompt_as<IT, DT, N, R, NPT, true>(p, a, tiles, pieces, stream);
  return launch_prompt_as<IT, DT, N, R, NPT, false>(p, a, tiles, 1, stream);
}

// Two channels a thread share what is read of B and C.  Four columns of each
// leave 125 registers and 16 warps an SM; eight (one wave of 512 CTAs for 1024)
// take 207 us where four take 202, four channels of four 225.  The long rows
// have eight: half the lanes to a channel, half the sums to reduce.
//
// Four CTAs an SM serve every type and dstate.  Three, with 168 registers, take as
// long within 2 % for 16-bit rows of dstate 32 to 256, more for an odd number of
// channels (336 us for 296) and for the split of 6001 x 1024 x 128 in fp32 (892 us
// for 732), less for other fp32 rows (9001 x 4096 x 16 196 us for 226, 2001 x 4096
// x 128 488 for 512, where four spill 1.5 KB, 1001 x 4096 x 256 720 for 765).
template <class IT, class DT>
cudaError_t launch_scan_prompt_n(int N, const ScanArgs& p, const Seqs& a,
                                 cudaStream_t stream) {
  switch (N) {
    case 16: return launch_scan_prompt<IT, DT, 16, 2, 4>(p, a, stream);
    case 32: return launch_scan_prompt<IT, DT, 32, 2, 4>(p, a, stream);
    case 64: return launch_scan_prompt<IT, DT, 64, 2, 4>(p, a, stream);
    case 128: return launch_scan_prompt<IT, DT, 128, 2, 8>(p, a, stream);
    case 256: return launch_scan_prompt<IT, DT, 256, 2, 8>(p, a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace layer
