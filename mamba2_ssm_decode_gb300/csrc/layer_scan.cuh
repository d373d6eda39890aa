// layer_scan.cuh -- the selective scan with an A that varies along dstate:
// for channel c and state column n, over the rows of a sequence in order,
//     dt'  = dt[r][c] + dt_bias[c];  dt' = softplus(dt') if dt_softplus
//     h[c][n] <- exp(A[c][n] dt') h[c][n] + dt' x[r][c] B[r][g][n]
//     y[r][c]  = sum_n h[c][n] C[r][g][n] + D[c] x[r][c];  y *= silu(z[r][c])
// with g = c / (channels / groups).  The chain stays in fp32 registers; a
// state is rounded only where it is stored.
#pragma once

#include "layer_common.cuh"

namespace layer {

struct ScanArgs {
  void* state;
  int state_dtype;  // ssu_dtype
  int64_t slots;
  int C, G;
  ssu::FastDiv per;  // channels per group
  const void* x;
  int64_t x_rs;
  const void* z;
  int64_t z_rs;
  void* out;
  int64_t o_rs;
  int out_f32;
  const void* dt;
  int64_t dt_rs;
  int dt_f32;
  int rows_vec;  // every row of x, z, dt, out, B and C (and its groups) starts on a 16-byte boundary
  const void* B;
  int64_t B_rs, B_gs;
  const void* Cm;
  int64_t C_rs, C_gs;
  int bc_vec;  // every row of B and C starts on a 16-byte boundary
  const float* A;
  int64_t A_rs;
  int a_vec;  // so does every row of A
  const float* D;
  const float* bias;
  int softplus;
  int disable;
  int64_t pad;
  const uint8_t* has_init;
  int final_only;
};

// ---------------------------------------------------------------------------
// Decode.  LPR lanes share a channel's state row (16-byte pieces, as
// ssu::RowLayout lays them out) and a lane owns the same pieces of U channels,
// so that it has U CPL 16-byte loads in flight and A stays in registers over
// the sequences that the CTA walks.  What a channel needs once per row (dt',
// D x, the gate) is worked out by the lanes that end up with its sum, and
// handed to the others by shuffles.
// ---------------------------------------------------------------------------
constexpr int kScanWarps = 4;

template <class ST, int N>
struct ScanStep {
  using L = ssu::RowLayout<ST, N>;
  static constexpr int FIT = 32 / L::EPL > 1 ? 32 / L::EPL : 1;  // 32 state values per thread
  static constexpr int U = L::LPR < FIT ? L::LPR : FIT;
  static constexpr int CH = kScanWarps * L::RPW * U;  // channels per CTA
};

template <class ST, class IT, int N>
__global__ void __launch_bounds__(kScanWarps * 32)
    scan_step_kernel(const ScanArgs p, const Seqs a) {
  using K = ScanStep<ST, N>;
  using L = typename K::L;
  constexpr int U = K::U;
  constexpr int LPU = L::LPR / U;  // lanes of a row that own the same channel's sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % L::LPR, rr = lane / L::LPR;
  const int c0 = blockIdx.x * K::CH + warp * L::RPW * U + rr;  // channel of u: c0 + u RPW
  const int mine = q / LPU;                                    // the u whose sum this lane ends up with
  const int cm = c0 + mine * L::RPW;
  const bool cm_ok = cm < p.C;

  float2 A2[U][L::EPL / 2];  // A log2 e
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * L::RPW;
#pragma unroll
    for (int k = 0; k < L::CPL; ++k) {
      float f[L::VEC];
#pragma unroll
      for (int i = 0; i < L::VEC; ++i) f[i] = 0.0f;
      if (c < p.C)
        load_floats<float, L::VEC>(p.A + c * p.A_rs + (q + k * L::LPR) * L::VEC, p.a_vec, f);
#pragma unroll
      for (int i = 0; i < L::VEC / 2; ++i)
        A2[u][k * L::VEC / 2 + i] = make_float2(f[2 * i] * kLog2e, f[2 * i + 1] * kLog2e);
    }
  }
  const float Dc = p.D && cm_ok ? p.D[cm] : 0.0f;
  const float bias = p.bias && cm_ok ? p.bias[cm] : 0.0f;
  ST* state = static_cast<ST*>(p.state);
  const IT* Bp = static_cast<const IT*>(p.B);
  const IT* Cp = static_cast<const IT*>(p.Cm);

  for (int s = blockIdx.y; s < a.n; s += gridDim.y) {
    const Item it = packed_item(a, s, p.pad, p.slots);
    if (it.len == 0) continue;
    const bool from = it.read_ok && (!p.has_init || p.has_init[s]);
    float2 h[U][L::EPL / 2];
    {
      uint4 raw[U][L::CPL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * L::RPW;
#pragma unroll
        for (int k = 0; k < L::CPL; ++k)
          raw[u][k] = from && c < p.C
                          ? ssu::ld_stream(state + (it.src * p.C + c) * N +
                                           (q + k * L::LPR) * L::VEC)
                          : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < L::CPL; ++k)
          ssu::Elem<ST>::unpack2(raw[u][k], &h[u][k * L::VEC / 2]);
    }
    for (int64_t t = 0; t < it.len; ++t) {
      const int64_t r = it.r0 + t;
      float xv = 0.0f, dtv = 0.0f, gate = 1.0f;
      if (cm_ok) {
        xv = to_f(static_cast<const IT*>(p.x)[r * p.x_rs + cm]);
        dtv = p.dt_f32 ? static_cast<const float*>(p.dt)[r * p.dt_rs + cm]
                       : to_f(static_cast<const IT*>(p.dt)[r * p.dt_rs + cm]);
        dtv = p.softplus ? softplus_sum(dtv, bias) : dtv + bias;
        if (p.z) gate = silu(to_f(static_cast<const IT*>(p.z)[r * p.z_rs + cm]));
      }
      const float dtx = dtv * xv;
      float acc[U];
      float2 Bv[L::EPL / 2], Cv[L::EPL / 2];
      int have = -1;  // the group whose B and C are at hand
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * L::RPW;
        const int g = p.G == 1 ? 0 : (int)p.per.div((uint32_t)(c < p.C ? c : p.C - 1));
        if (u == 0 || g != have) {
          have = g;
#pragma unroll
          for (int k = 0; k < L::CPL; ++k) {
            const int64_t n = (q + k * L::LPR) * L::VEC;
            load_floats<IT, L::VEC>(Bp + r * p.B_rs + g * p.B_gs + n, p.bc_vec,
                                    reinterpret_cast<float*>(&Bv[k * L::VEC / 2]));
            load_floats<IT, L::VEC>(Cp + r * p.C_rs + g * p.C_gs + n, p.bc_vec,
                                    reinterpret_cast<float*>(&Cv[k * L::VEC / 2]));
          }
        }
        const int from_lane = (lane - q) + u * LPU;
        const float d = __shfl_sync(0xffffffffu, dtv, from_lane);
        const float dx = __shfl_sync(0xffffffffu, dtx, from_lane);
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < L::EPL / 2; ++i) {
          const float2 e = __fmul2_rn(A2[u][i], make_float2(d, d));
          const float2 hv = __ffma2_rn(h[u][i], make_float2(ex2(e.x), ex2(e.y)),
                                       __fmul2_rn(make_float2(dx, dx), Bv[i]));
          h[u][i] = hv;
          sum = __ffma2_rn(hv, Cv[i], sum);
        }
        acc[u] = sum.x + sum.y;
      }
      int base = 0, plain = 0;
      ssu::RowScatter<U, L::LPR / 2>::run(acc, q, base, plain);  // acc[0]: channel cm (base == mine)
      if (cm_ok && (q & plain) == 0) {
        const float y = (acc[0] + Dc * xv) * gate;
        if (p.out_f32) static_cast<float*>(p.out)[r * p.o_rs + cm] = y;
        else static_cast<IT*>(p.out)[r * p.o_rs + cm] = from_f<IT>(y);
      }
      int64_t slot;
      const bool now = !p.final_only || t == it.len - 1;
      if (now && it.read_ok && !p.disable &&
          write_slot(a, s, p.final_only ? 0 : t, p.pad, p.slots, &slot)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * L::RPW;
          if (c < p.C) {
#pragma unroll
            for (int k = 0; k < L::CPL; ++k)
              ssu::st_state(state + (slot * p.C + c) * N + (q + k * L::LPR) * L::VEC,
                            ssu::Elem<ST>::pack2(&h[u][k * L::VEC / 2]));
          }
        }
      }
    }
  }
}

// One row per sequence and one group of B and C: the lane layout of
// scan_step_kernel, walked as a pipeline.  While a sequence is worked on, the
// next one's state and row are on their way, and the slot of the one after it,
// so that a CTA always has loads in flight and waits for none of them twice.
template <class ST, class IT, int N>
__global__ void __launch_bounds__(kScanWarps * 32, ScanStep<ST, N>::L::EPL > 16 ? 2 : 3)
    scan_token_kernel(const ScanArgs p, const Seqs a) {
  using K = ScanStep<ST, N>;
  using L = typename K::L;
  constexpr int U = K::U, VEC = L::VEC, CPL = L::CPL, H = L::EPL / 2;
  constexpr int LPU = L::LPR / U;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % L::LPR, rr = lane / L::LPR;
  const int c0 = blockIdx.x * K::CH + warp * L::RPW * U + rr;
  const int cm = c0 + q / LPU * L::RPW;
  const bool cm_ok = cm < p.C;
  const int cl = cm_ok ? cm : p.C - 1;  // lanes beyond the channels read the last one's row

  float2 A2[U][H];  // A log2 e
  bool c_ok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * L::RPW;
    c_ok[u] = c < p.C;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      float f[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = 0.0f;
      if (c_ok[u]) load_floats<float, VEC>(p.A + c * p.A_rs + (q + k * L::LPR) * VEC, p.a_vec, f);
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i)
        A2[u][k * VEC / 2 + i] = make_float2(f[2 * i] * kLog2e, f[2 * i + 1] * kLog2e);
    }
  }
  const float Dc = p.D && cm_ok ? p.D[cm] : 0.0f;
  const float bias = p.bias && cm_ok ? p.bias[cm] : 0.0f;
  ST* state = static_cast<ST*>(p.state);
  const IT* xp = static_cast<const IT*>(p.x) + cl;
  const IT* zp = static_cast<const IT*>(p.z) + cl;
  const IT* Bp = static_cast<const IT*>(p.B) + q * VEC;
  const IT* Cp = static_cast<const IT*>(p.Cm) + q * VEC;

  uint4 raw[U][CPL];
  Words<IT, 1> x, z;
  uint32_t dt;  // as stored
  Words<IT, VEC> B[CPL], C[CPL];
  z.zero();
  // what sequence s needs, from the slot it reads
  auto fetch = [&](int s, int64_t slot, bool read) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < CPL; ++k) {
        raw[u][k] = make_uint4(0u, 0u, 0u, 0u);
        if (read && c_ok[u])
          raw[u][k] = ssu::ld_stream(state + (slot * p.C + c0 + u * L::RPW) * N +
                                     (q + k * L::LPR) * VEC);
      }
    x.load(xp + s * p.x_rs);
    if (p.z) z.load(zp + s * p.z_rs);
    if (p.dt_f32) dt = static_cast<const uint32_t*>(p.dt)[s * p.dt_rs + cl];
    else if constexpr (sizeof(IT) == 2)
      dt = static_cast<const uint16_t*>(p.dt)[s * p.dt_rs + cl];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      if (p.bc_vec) {
        B[k].load(Bp + s * p.B_rs + k * L::LPR * VEC);
        C[k].load(Cp + s * p.C_rs + k * L::LPR * VEC);
      } else {
        B[k].load_some(Bp + s * p.B_rs + k * L::LPR * VEC, VEC);
        C[k].load_some(Cp + s * p.C_rs + k * L::LPR * VEC, VEC);
      }
    }
  };

  int s = blockIdx.y;
  int next = s + gridDim.y;
  Slot from = load_slot(a.src, s, 0, a.idx64), to = load_slot(a.dst, s, 0, a.idx64);
  int64_t src = from.id(s, a.idx64);
  bool read = from.found && slot_ok(src, p.pad, p.slots);
  fetch(s, src, read);
  Slot from_n = from, to_n = to;
  if (next < a.n) {
    from_n = load_slot(a.src, next, 0, a.idx64);
    to_n = load_slot(a.dst, next, 0, a.idx64);
  }
  while (true) {
    float2 h[U][H], Bv[H], Cv[H];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < CPL; ++k) ssu::Elem<ST>::unpack2(raw[u][k], &h[u][k * VEC / 2]);
#pragma unroll
    for (int k = 0; k < CPL; ++k)
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        Bv[k * VEC / 2 + i] = B[k].pair(i);
        Cv[k * VEC / 2 + i] = C[k].pair(i);
      }
    const float xv = x.at(0), zv = z.at(0);
    Words<IT, 1> d16;
    d16.w[0] = dt;
    const float dv = p.dt_f32 ? __uint_as_float(dt) : d16.at(0);
    const int64_t dst = to.id(s, a.idx64);
    const bool write = read && !p.disable && to.found && slot_ok(dst, p.pad, p.slots);
    const int now = s;
    const bool more = next < a.n;
    if (more) {
      s = next;
      next += gridDim.y;
      src = from_n.id(s, a.idx64);
      read = from_n.found && slot_ok(src, p.pad, p.slots);
      to = to_n;
      fetch(s, src, read);
      if (next < a.n) {
        from_n = load_slot(a.src, next, 0, a.idx64);
        to_n = load_slot(a.dst, next, 0, a.idx64);
      }
    }

    const float dtv = p.softplus ? softplus_sum(dv, bias) : dv + bias;
    const float dtx = dtv * xv;
    float acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int from_lane = (lane - q) + u * LPU;
      const float d = __shfl_sync(0xffffffffu, dtv, from_lane);
      const float dx = __shfl_sync(0xffffffffu, dtx, from_lane);
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 e = __fmul2_rn(A2[u][i], make_float2(d, d));
        const float2 hv = __ffma2_rn(h[u][i], make_float2(ex2(e.x), ex2(e.y)),
                                     __fmul2_rn(make_float2(dx, dx), Bv[i]));
        h[u][i] = hv;
        sum = __ffma2_rn(hv, Cv[i], sum);
      }
      acc[u] = sum.x + sum.y;
    }
    int base = 0, plain = 0;
    ssu::RowScatter<U, L::LPR / 2>::run(acc, q, base, plain);
    if (write) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < CPL; ++k)
          if (c_ok[u])
            ssu::st_state(state + (dst * p.C + c0 + u * L::RPW) * N + (q + k * L::LPR) * VEC,
                          ssu::Elem<ST>::pack2(&h[u][k * VEC / 2]));
    }
    if (cm_ok && (q & plain) == 0) {
      const float y = (acc[0] + Dc * xv) * (p.z ? silu(zv) : 1.0f);
      if (p.out_f32) static_cast<float*>(p.out)[now * p.o_rs + cm] = y;
      else static_cast<IT*>(p.out)[now * p.o_rs + cm] = from_f<IT>(y);
    }
    if (!more) break;
  }
}

template <class ST, class IT, int N>
cudaError_t launch_scan_step(const ScanArgs& p, const Seqs& a, cudaStream_t stream) {
  using K = ScanStep<ST, N>;
  const bool token = !a.cu && !a.na && a.steps == 1 && p.G == 1;
  auto kern = token ? scan_token_kernel<ST, IT, N> : scan_step_kernel<ST, IT, N>;
  const int64_t gx = (p.C + K::CH - 1) / K::CH;
  // one wave: each CTA walks its share of the sequences with A in registers
  static int per_sm[2] = {0, 0};
  int& fit = per_sm[token];
  if (fit == 0) {
    const cudaError_t e =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, kScanWarps * 32, 0);
    if (e != cudaSuccess) return e;
  }
  int64_t gy = (int64_t)fit * ssu::sm_count() / gx;
  if (gy < 1) gy = 1;
  if (gy > a.n) gy = a.n;
  if (gy > 65535) gy = 65535;
  kern<<<dim3((unsigned)gx, (unsigned)gy), kScanWarps * 32, 0, stream>>>(p, a);
  return cudaGetLastError();
}

template <class ST, class IT>
cudaError_t launch_scan_n(int N, const ScanArgs& p, const Seqs& a,
                          cudaStream_t stream) {
  switch (N) {
    case 16: return launch_scan_step<ST, IT, 16>(p, a, stream);
    case 32: return launch_scan_step<ST, IT, 32>(p, a, stream);
    case 64: return launch_scan_step<ST, IT, 64>(p, a, stream);
    case 128: return launch_scan_step<ST, IT, 128>(p, a, stream);
    case 256: return launch_scan_step<ST, IT, 256>(p, a, stream);
  }
  return cudaErrorInvalidValue;
}

template <class IT>
cudaError_t launch_scan_io(int N, const ScanArgs& p, const Seqs& a,
                           cudaStream_t stream) {
  switch (p.state_dtype) {
    case SSU_F32: return launch_scan_n<float, IT>(N, p, a, stream);
    case SSU_BF16: return launch_scan_n<__nv_bfloat16, IT>(N, p, a, stream);
    case SSU_F16: return launch_scan_n<__half, IT>(N, p, a, stream);
    default: return cudaErrorInvalidValue;
  }
}

// one translation unit for each element type of the rows
cudaError_t launch_scan_f32(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream);
cudaError_t launch_prompt_f32(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream);
cudaError_t launch_scan_bf16(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream);
cudaError_t launch_prompt_bf16(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream);
cudaError_t launch_scan_f16(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream);
cudaError_t launch_prompt_f16(int N, const ScanArgs& p, const Seqs& a,
                         cudaStream_t stream);

}  // namespace layer
