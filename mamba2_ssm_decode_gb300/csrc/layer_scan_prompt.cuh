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
// Bound by the exponentials (dstate per row and channel, on the special-function
// pipe) and the packed fp32 products beside them, not by HBM.
#pragma once

#include "layer_scan.cuh"

namespace layer {

constexpr int kPromptThreads = 128;

template <int N>
struct PromptTile {
  static constexpr int NPT = N == 16 ? 4 : 8;           // state columns per thread
  static constexpr int LPC = N / NPT;                   // lanes per channel
  static constexpr int CH = kPromptThreads / LPC;       // channels per CTA
  static constexpr int TT = N <= 128 ? 32 : 16;         // rows per tile
  static constexpr int TPR = kPromptThreads / TT;       // staging threads per row
  static constexpr int SV = CH >= TPR ? CH / TPR : 1;   // channels per staging thread
  static constexpr int BV = N / TPR;                    // B (and C) columns per staging thread
  static constexpr int TG = LPC < 8 ? LPC : 8;          // rows whose sums are reduced together
  static constexpr int YS = CH + 32 / TG;               // row stride of the sums
};

template <int N>
struct alignas(16) PromptSmem {
  using K = PromptTile<N>;
  float d[K::TT][K::CH];    // dt'
  float dx[K::TT][K::CH];   // dt' x
  float B[K::TT][N];
  float C[K::TT][N];
  float y[K::TT][K::YS];    // sums over dstate
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

// V elements as stored: one access where `vec`, else those in [0, n) one by one, zeros beyond.
template <class T, int V>
__device__ __forceinline__ Pack<T, V> fetch(const T* p, bool vec, int n) {
  if (vec && n >= V) return load_pack<T, V>(p);
  Pack<T, V> r = zero_pack<T, V>();
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) r.v[i] = p[i];
  return r;
}

template <class IT, class DT, int N>
__global__ void __launch_bounds__(kPromptThreads)
    scan_prompt_kernel(const ScanArgs p, const VarlenArgs a, int64_t nseqs) {
  using K = PromptTile<N>;
  constexpr int NPT = K::NPT, LPC = K::LPC, TT = K::TT, SV = K::SV, BV = K::BV, TG = K::TG;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  PromptSmem<N>& sm = *reinterpret_cast<PromptSmem<N>*>(smem_raw);

  const int tid = threadIdx.x, lane = tid & 31;
  const int per = p.C / p.G, tiles = (per + K::CH - 1) / K::CH;
  const int g = blockIdx.x / tiles;                       // the CTA's channels are of one group
  const int c0 = g * per + (blockIdx.x - g * tiles) * K::CH;
  const int c_end = (g + 1) * per;

  // the chain's part: channel cc, columns n(j, i) = (j LPC + q) 4 + i
  const int q = lane % LPC;
  const int ch = tid / LPC;
  const int cc = c0 + ch;
  float2 A2[NPT / 2], h[NPT / 2];
#pragma unroll
  for (int j = 0; j < NPT / 4; ++j) {
    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (cc < c_end) load_floats<float, 4>(p.A + cc * p.A_rs + (j * LPC + q) * 4, p.a_vec, f);
    A2[2 * j] = make_float2(f[0] * kLog2e, f[1] * kLog2e);
    A2[2 * j + 1] = make_float2(f[2] * kLog2e, f[3] * kLog2e);
  }

  // the staging part: row tr of the tile, channels sc .. sc + SV
  const int tr = tid / K::TPR, tp = tid % K::TPR;
  const int sc = c0 + tp * SV;
  const int sn = tp * SV < K::CH ? (c_end - sc < SV ? c_end - sc : SV) : 0;
  const int b0 = tp * BV;
  float Dv[SV], bias[SV];
#pragma unroll
  for (int i = 0; i < SV; ++i) {
    Dv[i] = p.D && i < sn ? p.D[sc + i] : 0.0f;
    bias[i] = p.bias && i < sn ? p.bias[sc + i] : 0.0f;
  }
  const IT* xp = static_cast<const IT*>(p.x) + sc;
  const IT* zp = static_cast<const IT*>(p.z) + sc;
  const DT* dp = static_cast<const DT*>(p.dt) + sc;
  const IT* Bp = static_cast<const IT*>(p.B) + g * p.B_gs + b0;
  const IT* Cp = static_cast<const IT*>(p.Cm) + g * p.C_gs + b0;

  for (int64_t s = blockIdx.y; s < nseqs; s += gridDim.y) {
    const Item it = packed_item(a, s, p.pad, p.slots);
    if (it.len == 0) continue;
    const bool from = it.read_ok && (!p.has_init || p.has_init[s]);
#pragma unroll
    for (int j = 0; j < NPT / 4; ++j) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (from && cc < c_end)
        v = load_state4(p, (it.src * p.C + cc) * N + (j * LPC + q) * 4);
      h[2 * j] = make_float2(v.x, v.y);
      h[2 * j + 1] = make_float2(v.z, v.w);
    }

    Pack<IT, SV> x, z;
    Pack<DT, SV> dt;
    Pack<IT, BV> B, C;
    const int64_t r_end = it.r0 + it.len;
    auto load = [&](int64_t r) {
      const bool in = r < r_end;
      x = fetch<IT, SV>(xp + r * p.x_rs, p.x_vec, in ? sn : 0);
      if (p.z) z = fetch<IT, SV>(zp + r * p.z_rs, p.z_vec, in ? sn : 0);
      dt = fetch<DT, SV>(dp + r * p.dt_rs, p.dt_vec, in ? sn : 0);
      B = fetch<IT, BV>(Bp + r * p.B_rs, p.bc_vec, in ? BV : 0);
      C = fetch<IT, BV>(Cp + r * p.C_rs, p.bc_vec, in ? BV : 0);
    };
    load(it.r0 + tr);

    for (int64_t t0 = 0; t0 < it.len; t0 += TT) {
      const int64_t r = it.r0 + t0 + tr;
      const int n = it.len - t0 < TT ? (int)(it.len - t0) : TT;
      // stage: rows beyond the sequence get dt' = 0 and zeros, a step that changes nothing
      const bool in = tr < n;
      Pack<IT, SV> xk = x, zk = z;
      if (tp * SV < K::CH) {
#pragma unroll
        for (int i = 0; i < SV; i += 2) {
          const int k = i + 1 < SV ? i + 1 : i;
          float2 d = make_float2(to_f(dt.v[i]), to_f(dt.v[k]));
          const float2 bi = make_float2(bias[i], bias[k]);
          d = p.softplus ? softplus_sum2(d, bi) : __fadd2_rn(d, bi);
          if (!in) d = make_float2(0.0f, 0.0f);
          const float2 dx = __fmul2_rn(d, make_float2(to_f(x.v[i]), to_f(x.v[k])));
          sm.d[tr][tp * SV + i] = d.x;
          sm.dx[tr][tp * SV + i] = dx.x;
          if (k > i) {
            sm.d[tr][tp * SV + k] = d.y;
            sm.dx[tr][tp * SV + k] = dx.y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < BV; ++i) {
        sm.B[tr][b0 + i] = to_f(B.v[i]);
        sm.C[tr][b0 + i] = to_f(C.v[i]);
      }
      __syncthreads();
      if (t0 + TT < it.len) load(r + TT);

      for (int t = 0; t < n; t += TG) {
        float acc[TG];
#pragma unroll
        for (int k = 0; k < TG; ++k) {
          const float d = sm.d[t + k][ch], dx = sm.dx[t + k][ch];
          const float2 d2 = make_float2(d, d), dx2 = make_float2(dx, dx);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int j = 0; j < NPT / 4; ++j) {
            const float4 b = *reinterpret_cast<const float4*>(&sm.B[t + k][(j * LPC + q) * 4]);
            const float4 c = *reinterpret_cast<const float4*>(&sm.C[t + k][(j * LPC + q) * 4]);
            const float2 e0 = __fmul2_rn(A2[2 * j], d2), e1 = __fmul2_rn(A2[2 * j + 1], d2);
            h[2 * j] = __ffma2_rn(h[2 * j], make_float2(ex2(e0.x), ex2(e0.y)),
                                  __fmul2_rn(dx2, make_float2(b.x, b.y)));
            h[2 * j + 1] = __ffma2_rn(h[2 * j + 1], make_float2(ex2(e1.x), ex2(e1.y)),
                                      __fmul2_rn(dx2, make_float2(b.z, b.w)));
            sum = __ffma2_rn(h[2 * j], make_float2(c.x, c.y), sum);
            sum = __ffma2_rn(h[2 * j + 1], make_float2(c.z, c.w), sum);
          }
          acc[k] = sum.x + sum.y;
        }
        int base = 0, plain = 0;
        ssu::RowScatter<TG, LPC / 2>::run(acc, q, base, plain);
        if ((q & plain) == 0) sm.y[t + base][ch] = acc[0];
      }
      __syncthreads();

      if (in && sn > 0) {
        float y[SV];
#pragma unroll
        for (int i = 0; i < SV; ++i) {
          y[i] = fmaf(Dv[i], to_f(xk.v[i]), sm.y[tr][tp * SV + i]);
          if (p.z) y[i] *= silu(to_f(zk.v[i]));
        }
        if (p.out_f32) {
          float* o = static_cast<float*>(p.out) + r * p.o_rs + sc;
          if (p.o_vec && sn == SV) {
            Pack<float, SV> v;
#pragma unroll
            for (int i = 0; i < SV; ++i) v.v[i] = y[i];
            store_pack<float, SV>(o, v);
          } else {
#pragma unroll
            for (int i = 0; i < SV; ++i)
              if (i < sn) o[i] = y[i];
          }
        } else {
          IT* o = static_cast<IT*>(p.out) + r * p.o_rs + sc;
          Pack<IT, SV> v;
#pragma unroll
          for (int i = 0; i < SV; ++i) v.v[i] = from_f<IT>(y[i]);
          if (p.o_vec && sn == SV) {
            store_pack<IT, SV>(o, v);
          } else {
#pragma unroll
            for (int i = 0; i < SV; ++i)
              if (i < sn) o[i] = v.v[i];
          }
        }
      }
    }

    int64_t slot;
    if (it.read_ok && !p.disable && cc < c_end && write_slot(a, s, 0, p.pad, p.slots, &slot)) {
#pragma unroll
      for (int j = 0; j < NPT / 4; ++j)
        store_state4(p, (slot * p.C + cc) * N + (j * LPC + q) * 4, h[2 * j], h[2 * j + 1]);
    }
  }
}

template <class IT, class DT, int N>
cudaError_t launch_scan_prompt(const ScanArgs& p, const VarlenArgs& a, int64_t nseqs,
                               cudaStream_t stream) {
  using K = PromptTile<N>;
  const int per = p.C / p.G;
  const int64_t gx = (int64_t)p.G * ((per + K::CH - 1) / K::CH);
  const int64_t gy = nseqs < 65535 ? nseqs : 65535;
  auto kern = scan_prompt_kernel<IT, DT, N>;
  const int smem = (int)sizeof(PromptSmem<N>);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<dim3((unsigned)gx, (unsigned)gy), kPromptThreads, smem, stream>>>(p, a, nseqs);
  return cudaGetLastError();
}

template <class IT, class DT>
cudaError_t launch_scan_prompt_n(int N, const ScanArgs& p, const VarlenArgs& a, int64_t nseqs,
                                 cudaStream_t stream) {
  switch (N) {
    case 16: return launch_scan_prompt<IT, DT, 16>(p, a, nseqs, stream);
    case 32: return launch_scan_prompt<IT, DT, 32>(p, a, nseqs, stream);
    case 64: return launch_scan_prompt<IT, DT, 64>(p, a, nseqs, stream);
    case 128: return launch_scan_prompt<IT, DT, 128>(p, a, nseqs, stream);
    case 256: return launch_scan_prompt<IT, DT, 256>(p, a, nseqs, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace layer
