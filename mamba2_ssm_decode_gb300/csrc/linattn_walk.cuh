// linattn_walk.cuh -- the recurrent form of linear attention (linattn.cuh):
// tokens, drafted tokens, and the prompts that the tensor cores do not take.
//
// A state is read and written once and bounds the call: 256 tokens of 32 heads of 128 x
// 128 fp32, 163 us (1082 MB, 98 % of a copy's rate).  128 sequences of 1 to 4 drafted
// tokens, 80 heads of 64 x 128 bf16, where the state is written after each: 128 us (595
// MB).  With the next row's operands in registers meanwhile they took 187 and 148 us:
// warps cover the loads better than registers do.
#pragma once

#include "linattn.cuh"

namespace linattn {

// A state row is dk elements; a lane owns 16 of them, as 16-byte chunks that
// alternate with those of the row's other lanes, so that a warp's load covers
// whole 128-byte lines.  A lane owns the same chunks of U rows.  ONE: a row a
// sequence; sequences of several rows wait for one's operands after the other's, and
// more warps, of fewer state rows each, cover that.
template <class ST, int DK, bool ONE>
struct WalkLayout {
  static constexpr int E = 16;                      // elements a lane owns of a row
  static constexpr int VEC = 16 / (int)sizeof(ST);  // elements of a chunk
  static constexpr int CPL = E / VEC;               // chunks a lane owns of a row
  static constexpr int LPR = DK / E;                // lanes of a row
  static constexpr int RPW = 32 / LPR;              // rows of a warp's load
  static constexpr int U = LPR >= 8 ? (ONE ? 4 : 2) : LPR == 4 && ONE ? 2 : 1;
  static constexpr int ROWS = RPW * U;              // rows of a warp
};

constexpr int kWalkWarps = 4;

// A lane's part of a state: rows p0 + u RPW of dv.  What a row does not have stays
// zero and is not stored.
template <class ST, int DK, bool ONE>
struct WalkState {
  using L = WalkLayout<ST, DK, ONE>;
  static constexpr int U = L::U, E = L::E, VEC = L::VEC, CPL = L::CPL, LPR = L::LPR;
  float2 S[U][E / 2];  // in pairs: an instruction for two

  __device__ __forceinline__ void load(const ST* src, bool from, int p0, int dv, int ql) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * L::RPW;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        Pack<ST, VEC> w = zero_pack<ST, VEC>();
        if (from && row < dv)
          w = load_pack<ST, VEC>(src + (int64_t)row * DK + (c * LPR + ql) * VEC);
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
          S[u][(c * VEC + e) / 2] = make_float2(to_f(w.v[e]), to_f(w.v[e + 1]));
      }
    }
  }
  // One row: the lane's elements of k and q, v(u) of its state rows; every lane of a
  // row gets the row's output, but for the scale.
  template <class V>
  __device__ __forceinline__ void step(const float* k, const float* q, float decay, const V& v,
                                       float* y) {
    const float2 d = make_float2(decay, decay);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float one = v(u);
      const float2 vu = make_float2(one, one);
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        S[u][e] = __ffma2_rn(vu, make_float2(k[2 * e], k[2 * e + 1]), __fmul2_rn(S[u][e], d));
        sum = __ffma2_rn(S[u][e], make_float2(q[2 * e], q[2 * e + 1]), sum);
      }
      y[u] = sum.x + sum.y;
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) y[u] += __shfl_xor_sync(0xffffffffu, y[u], o);
  }
  __device__ __forceinline__ void store(ST* dst, int p0, int dv, int ql) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * L::RPW;
      if (row >= dv) continue;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        Pack<ST, VEC> w;
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          Words<ST, 2> two;
          two.set(&S[u][(c * VEC + e) / 2]);
          two.store(&w.v[e]);
        }
        store_pack<ST, VEC>(dst + (int64_t)row * DK + (c * LPR + ql) * VEC, w);
      }
    }
  }
};

// CTAs an SM that a sequence of several rows is bounded to: warps cover what its rows wait
// for.  128 sequences of 1 to 4 rows, 32 heads of 128 x dk: fp32 and dk 32 56.9 us for 59.8
// unbounded, dk 64 53.7 for 57.5; bf16 and dk 64 76.5 at ten and 80.3 at eight.  From dk 128
// on nine fit; bounded to that, other code spilled (80 heads of 64 x 128 bf16: 133 -> 141 us).
template <class ST, int DK, bool ONE>
constexpr int walk_ctas() {
  return ONE || DK >= 128 ? 0 : DK == 64 && sizeof(ST) == 2 ? 10 : 8;
}

// Tokens.  ONE: a row a sequence, which is that of its number.
template <class ST, class IT, int DK, bool ONE>
__global__ void __launch_bounds__(kWalkWarps * 32, (walk_ctas<ST, DK, ONE>()))
    linattn_walk_kernel(const Args p, const Seqs a) {
  using L = WalkLayout<ST, DK, ONE>;
  constexpr int U = L::U, E = L::E, VEC = L::VEC, CPL = L::CPL, LPR = L::LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ql = lane % LPR;
  const int s = blockIdx.x;
  const int h = blockIdx.y, g = h / p.hr;
  const int p0 = (blockIdx.z * kWalkWarps + warp) * L::ROWS + lane / LPR;

  const Item it = packed_item<ONE>(a, s, p.pad, p.slots);
  if (it.len == 0) return;
  const int64_t head = (int64_t)p.dv * DK;
  WalkState<ST, DK, ONE> state;
  state.load(static_cast<const ST*>(p.state) + (it.src * p.H + h) * head, it.read_ok, p0, p.dv, ql);

  const IT *qp, *kp, *vp;
  IT* op;
  const float* lp;
  auto row_at = [&](int t) {
    const int64_t r = it.r0 + t;
    qp = static_cast<const IT*>(p.q) + r * p.q_rs + (int64_t)g * p.q_gs;
    kp = static_cast<const IT*>(p.k) + r * p.k_rs + (int64_t)g * p.k_gs;
    vp = static_cast<const IT*>(p.v) + r * p.v_rs + (int64_t)h * p.v_hs;
    op = static_cast<IT*>(p.out) + r * p.o_rs + (int64_t)h * p.o_hs;
    lp = p.ld ? p.ld + r * p.ld_rs + (int64_t)h * p.ld_hs : nullptr;
  };
  // Several rows of wide states: each one's addresses are worked out when it comes.  Kept along
  // they take ten registers and a CTA an SM or three: 128 sequences of 1 to 4 rows, 32 heads of
  // 128 x 128 fp32, take 223 us for 175 (narrow states: 63 for 54).
  constexpr bool AGAIN = !ONE && DK >= 128;
  row_at(0);

  for (int t = 0; t < it.len; ++t) {
    if constexpr (AGAIN) row_at(t);
    float k[E], q[E], y[U];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      load_floats<IT, VEC>(kp + (c * LPR + ql) * VEC, p.qk_vec, k + c * VEC);
      load_floats<IT, VEC>(qp + (c * LPR + ql) * VEC, p.qk_vec, q + c * VEC);
    }
    const float decay = lp ? expf(*lp) : 1.0f;
    auto v = [&](int u) {
      const int row = p0 + u * L::RPW;
      return row < p.dv ? to_f(vp[row]) : 0.0f;
    };
    state.step(k, q, decay, v, y);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * L::RPW;
      if (ql == 0 && row < p.dv) op[row] = from_f<IT>(y[u] * p.scale);
    }
    int64_t to;
    if (it.read_ok && !p.disable && write_slot(a, s, t, p.pad, p.slots, &to))
      state.store(static_cast<ST*>(p.state) + (to * p.H + h) * head, p0, p.dv, ql);
    if constexpr (!AGAIN) {
      qp += p.q_rs;
      kp += p.k_rs;
      vp += p.v_rs;
      op += p.o_rs;
      if (lp) lp += p.ld_rs;
    }
  }
}

// Prompts: the same walk, with blocks of kBlock rows brought to shared memory as fp32
// while the block before is computed.  The longest prompt's chain of rows bounds it: 16 prompts
// of 128 rows on average and up to 197, 8 heads of 128 x 128 fp32, take 86 us, and 275 with a
// row's operands asked for in its turn; 256 prompts of two rows on average 173 us against 222.
constexpr int kBlock = 8;

template <class ST, class IT, int DK>
__global__ void __launch_bounds__(kWalkWarps * 32)
    linattn_rows_kernel(const Args p, const Seqs a) {
  using L = WalkLayout<ST, DK, false>;
  constexpr int U = L::U, E = L::E, VEC = L::VEC, CPL = L::CPL, LPR = L::LPR;
  constexpr int TILE = kWalkWarps * L::ROWS, THREADS = kWalkWarps * 32;
  constexpr int N = kBlock * (2 * DK + TILE), PER = (N + THREADS - 1) / THREADS;
  __shared__ __align__(16) float rows[2][N];  // k, q and v of a block's rows
  __shared__ float decays[2][kBlock];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ql = lane % LPR;
  const int s = blockIdx.x;
  const int h = blockIdx.y, g = h / p.hr;
  const int tile0 = blockIdx.z * TILE;
  const int mine = warp * L::ROWS + lane / LPR, p0 = tile0 + mine;

  const Item it = packed_item(a, s, p.pad, p.slots);
  if (it.len == 0) return;
  const int64_t head = (int64_t)p.dv * DK;
  WalkState<ST, DK, false> state;
  state.load(static_cast<const ST*>(p.state) + (it.src * p.H + h) * head,
             it.read_ok && (!p.has_init || p.has_init[s]), p0, p.dv, ql);

  const IT* qp = static_cast<const IT*>(p.q) + (int64_t)it.r0 * p.q_rs + (int64_t)g * p.q_gs;
  const IT* kp = static_cast<const IT*>(p.k) + (int64_t)it.r0 * p.k_rs + (int64_t)g * p.k_gs;
  const IT* vp = static_cast<const IT*>(p.v) + (int64_t)it.r0 * p.v_rs + (int64_t)h * p.v_hs;
  IT* op = static_cast<IT*>(p.out) + (int64_t)it.r0 * p.o_rs + (int64_t)h * p.o_hs;
  const float* lp = p.ld ? p.ld + (int64_t)it.r0 * p.ld_rs + (int64_t)h * p.ld_hs : nullptr;

  float x[PER], decay = 1.0f;  // this thread's share of the block that comes
  auto fetch = [&](int t0) {
#pragma unroll
    for (int n = 0; n < PER; ++n) {
      const int i = tid + n * THREADS;
      x[n] = 0.0f;
      if (i < 2 * kBlock * DK) {
        const int t = t0 + i / DK % kBlock, e = i % DK;
        if (t < it.len)
          x[n] = to_f(i < kBlock * DK ? kp[(int64_t)t * p.k_rs + e] : qp[(int64_t)t * p.q_rs + e]);
      } else if (i < N) {
        const int j = i - 2 * kBlock * DK, t = t0 + j / TILE, row = tile0 + j % TILE;
        if (t < it.len && row < p.dv) x[n] = to_f(vp[(int64_t)t * p.v_rs + row]);
      }
    }
    if (lp && tid < kBlock && t0 + tid < it.len) decay = expf(lp[(int64_t)(t0 + tid) * p.ld_rs]);
  };
  auto leave = [&](int b) {
#pragma unroll
    for (int n = 0; n < PER; ++n)
      if (tid + n * THREADS < N) rows[b][tid + n * THREADS] = x[n];
    if (tid < kBlock) decays[b][tid] = decay;
  };
  fetch(0);
  leave(0);
  __syncthreads();
  for (int t0 = 0, b = 0; t0 < it.len; t0 += kBlock, b ^= 1) {
    const bool more = t0 + kBlock < it.len;
    if (more) fetch(t0 + kBlock);
    const int n = min(kBlock, it.len - t0);
    for (int r = 0; r < n; ++r) {
      float k[E], q[E], y[U];
      const float* kr = rows[b] + r * DK;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        load_floats<float, VEC>(kr + (c * LPR + ql) * VEC, true, k + c * VEC);
        load_floats<float, VEC>(kr + kBlock * DK + (c * LPR + ql) * VEC, true, q + c * VEC);
      }
      auto v = [&](int u) { return rows[b][2 * kBlock * DK + r * TILE + mine + u * L::RPW]; };
      state.step(k, q, decays[b][r], v, y);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = p0 + u * L::RPW;
        if (ql == 0 && row < p.dv) op[row] = from_f<IT>(y[u] * p.scale);
      }
      op += p.o_rs;
    }
    if (more) leave(b ^ 1);
    __syncthreads();
  }
  int64_t to;
  if (it.read_ok && write_slot(a, s, 0, p.pad, p.slots, &to))
    state.store(static_cast<ST*>(p.state) + (to * p.H + h) * head, p0, p.dv, ql);
}

template <class ST, class IT, int DK>
cudaError_t launch_walk_dk(const Args& p, const Seqs& a, cudaStream_t stream) {
  const bool one = !a.cu && !a.na && a.steps == 1 && !p.prompt;
  const int per = kWalkWarps * (one ? WalkLayout<ST, DK, true>::ROWS : WalkLayout<ST, DK, false>::ROWS);
  // sequences along x, which has room for them all
  const dim3 grid((unsigned)a.n, (unsigned)p.H, (unsigned)((p.dv + per - 1) / per));
  if (p.prompt) linattn_rows_kernel<ST, IT, DK><<<grid, kWalkWarps * 32, 0, stream>>>(p, a);
  else if (one) linattn_walk_kernel<ST, IT, DK, true><<<grid, kWalkWarps * 32, 0, stream>>>(p, a);
  else linattn_walk_kernel<ST, IT, DK, false><<<grid, kWalkWarps * 32, 0, stream>>>(p, a);
  return cudaGetLastError();
}

template <class ST, class IT>
cudaError_t launch_walk_st(const Args& p, const Seqs& a, cudaStream_t stream) {
  switch (p.dk) {
    case 16: return launch_walk_dk<ST, IT, 16>(p, a, stream);
    case 32: return launch_walk_dk<ST, IT, 32>(p, a, stream);
    case 64: return launch_walk_dk<ST, IT, 64>(p, a, stream);
    case 128: return launch_walk_dk<ST, IT, 128>(p, a, stream);
    case 256: return launch_walk_dk<ST, IT, 256>(p, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <class IT>
cudaError_t launch_walk_io(const Args& p, const Seqs& a, cudaStream_t stream) {
  switch (p.state_dtype) {
    case SSU_F32: return launch_walk_st<float, IT>(p, a, stream);
    case SSU_BF16: return launch_walk_st<__nv_bfloat16, IT>(p, a, stream);
    case SSU_F16: return launch_walk_st<__half, IT>(p, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace linattn
