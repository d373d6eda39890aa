// linattn_walk.cuh -- the recurrent form of linear attention (linattn.cuh):
// tokens, drafted tokens, and the prompts that the tensor cores do not take.
//
// A state is read and written once and bounds the call: 256 tokens of 32 heads of 128 x
// 128 fp32, 163 us (1082 MB, 98 % of a copy's rate).  128 sequences of 1 to 4 drafted
// tokens, 80 heads of 64 x 128 bf16, where the state is written after each: 123 us (595
// MB; 71 % of issue slots).  With the next row's operands in registers meanwhile they
// took 187 and 148 us: warps cover the loads better than registers do.
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

// ONE: a row a sequence, which is that of its number.
template <class ST, class IT, int DK, bool ONE>
__global__ void __launch_bounds__(kWalkWarps * 32)
    linattn_walk_kernel(const Args p, const Seqs a) {
  using L = WalkLayout<ST, DK, ONE>;
  constexpr int U = L::U, E = L::E, VEC = L::VEC, CPL = L::CPL, LPR = L::LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ql = lane % LPR;
  const int s = blockIdx.x;
  const int h = blockIdx.y, g = h / p.hr;
  const int p0 = blockIdx.z * kWalkWarps * L::ROWS + warp * L::ROWS + lane / LPR;

  const Item it = packed_item<ONE>(a, s, p.pad, p.slots);
  if (it.len == 0) return;
  const bool from = it.read_ok && (!p.has_init || p.has_init[s]);

  // state rows p0 + u RPW; what a row does not have stays zero and is not stored
  float2 S[U][E / 2];  // in pairs: an instruction for two
  const int64_t head = (int64_t)p.dv * DK;
  const ST* src = static_cast<const ST*>(p.state) + (it.src * p.H + h) * head;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = p0 + u * L::RPW;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      Pack<ST, VEC> w = zero_pack<ST, VEC>();
      if (from && row < p.dv)
        w = load_pack<ST, VEC>(src + (int64_t)row * DK + (c * LPR + ql) * VEC);
#pragma unroll
      for (int e = 0; e < VEC; e += 2)
        S[u][(c * VEC + e) / 2] = make_float2(to_f(w.v[e]), to_f(w.v[e + 1]));
    }
  }

  const IT* qp = static_cast<const IT*>(p.q) + (int64_t)it.r0 * p.q_rs + (int64_t)g * p.q_gs;
  const IT* kp = static_cast<const IT*>(p.k) + (int64_t)it.r0 * p.k_rs + (int64_t)g * p.k_gs;
  const IT* vp = static_cast<const IT*>(p.v) + (int64_t)it.r0 * p.v_rs + (int64_t)h * p.v_hs;
  IT* op = static_cast<IT*>(p.out) + (int64_t)it.r0 * p.o_rs + (int64_t)h * p.o_hs;
  const float* lp = p.ld ? p.ld + (int64_t)it.r0 * p.ld_rs + (int64_t)h * p.ld_hs : nullptr;

  for (int t = 0; t < it.len; ++t) {
    float k[E], q[E];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      load_floats<IT, VEC>(kp + (c * LPR + ql) * VEC, p.qk_vec, k + c * VEC);
      load_floats<IT, VEC>(qp + (c * LPR + ql) * VEC, p.qk_vec, q + c * VEC);
    }
    const float decay = lp ? expf(*lp) : 1.0f;
    const float2 d = make_float2(decay, decay);
    float y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * L::RPW;
      const float one = row < p.dv ? to_f(vp[row]) : 0.0f;
      const float2 v = make_float2(one, one);
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        S[u][e] = __ffma2_rn(v, make_float2(k[2 * e], k[2 * e + 1]), __fmul2_rn(S[u][e], d));
        sum = __ffma2_rn(S[u][e], make_float2(q[2 * e], q[2 * e + 1]), sum);
      }
      y[u] = sum.x + sum.y;
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) y[u] += __shfl_xor_sync(0xffffffffu, y[u], o);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = p0 + u * L::RPW;
      if (ql == 0 && row < p.dv) op[row] = from_f<IT>(y[u] * p.scale);
    }
    int64_t to;
    const bool last = t == it.len - 1;
    if (it.read_ok && !p.disable && (last || !p.prompt) &&
        write_slot(a, s, p.prompt ? 0 : t, p.pad, p.slots, &to)) {
      ST* dst = static_cast<ST*>(p.state) + (to * p.H + h) * head;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = p0 + u * L::RPW;
        if (row >= p.dv) continue;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          Pack<ST, VEC> w;
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float2 f = S[u][(c * VEC + e) / 2];
            Words<ST, 2> two;
            two.set(&f);
            two.store(&w.v[e]);
          }
          store_pack<ST, VEC>(dst + (int64_t)row * DK + (c * LPR + ql) * VEC, w);
        }
      }
    }
    qp += p.q_rs;
    kp += p.k_rs;
    vp += p.v_rs;
    op += p.o_rs;
    if (lp) lp += p.ld_rs;
  }
}

template <class ST, class IT, int DK, bool ONE>
cudaError_t launch_walk_form(const Args& p, const Seqs& a, cudaStream_t stream) {
  constexpr int per = kWalkWarps * WalkLayout<ST, DK, ONE>::ROWS;
  const int tiles = (p.dv + per - 1) / per;
  // sequences along x, which has room for them all
  linattn_walk_kernel<ST, IT, DK, ONE>
      <<<dim3((unsigned)a.n, (unsigned)p.H, (unsigned)tiles), kWalkWarps * 32, 0, stream>>>(p, a);
  return cudaGetLastError();
}

template <class ST, class IT, int DK>
cudaError_t launch_walk_dk(const Args& p, const Seqs& a, cudaStream_t stream) {
  if (!a.cu && !a.na && a.steps == 1 && !p.prompt)
    return launch_walk_form<ST, IT, DK, true>(p, a, stream);
  return launch_walk_form<ST, IT, DK, false>(p, a, stream);
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
