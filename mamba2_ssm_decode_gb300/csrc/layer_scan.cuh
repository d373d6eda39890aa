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
  const uint8_t* has_init;  // per sequence, or NULL: every valid slot is read
};

// ---------------------------------------------------------------------------
// Decode.  LPR lanes share a channel's state row (16-byte pieces, as
// ssu::RowLayout lays them out) and a lane owns the same pieces of U channels,
// so that it has U CPL 16-byte loads in flight and A stays in registers over
// the sequences that the CTA walks.  What a channel needs once per row (dt',
// D x, the gate) is worked out by the lanes that end up with its sum, and
// handed to the others by shuffles.
//
// A CTA (its channels are of one group) walks its sequences as a pipeline:
// while a row is worked on, the next row is on its way, or the next sequence's
// state and first row, and before that the slot of the sequence after and the
// bounds of the one after that.  So it waits for none of them from the start,
// and one wave of CTAs keeps loads in flight throughout.  Bound by HBM: the
// state is read once a sequence and written once a row.  512 tokens x 5120
// channels x 16, fp32 state: 56.5 us, 357 MB, 6.3 TB/s; with drafted rows the
// chain of a row (softplus, shuffles, exponentials) shows, and the next
// sequence's state is asked for only in a sequence's last row: 128 sequences of 1
// to 4 rows take 46 us for 160 MB.
// ---------------------------------------------------------------------------
constexpr int kScanWarps = 4;

template <class ST, int N>
struct ScanStep {
  using L = ssu::RowLayout<ST, N>;
  // State values per thread: 16 of the short rows, 32 of those whose lanes own
  // more (64 tokens x 5120 channels x 128, fp32: 72 us with 32, 95 us with 16),
  // and the CTAs an SM that they leave room for (512 tokens x 5120 channels x
  // 16: fp32 state 65 us with four, bf16 47 us; three take 70 and 70, five 67
  // and 53).  The long rows have three, some registers spilled: with 16-bit x, B
  // and C 64 tokens x 5120 x 128 take 72 us where two take 109, 32 tokens x 256 81
  // us for 107.  fp32 rows pay more for the spills than two CTAs would cost them:
  // 103 us for 79, and 133 us for 88.
  static constexpr int MOST = L::EPL > 4 ? 32 : 16;
  static constexpr int FIT = MOST / L::EPL > 1 ? MOST / L::EPL : 1;
  static constexpr int U = L::LPR < FIT ? L::LPR : FIT;
  static constexpr int CTAS = U * L::EPL > 16 ? 3 : 4;
  static constexpr int CH = kScanWarps * L::RPW * U;  // channels per CTA
};

// The bounds and the slot of a sequence, in the order in which they can be
// asked for.  ONE: every sequence is one row and reads entry 0 of its table.
template <bool ONE>
struct Ahead {
  RawIndex b, e, n;  // bounds and accepted count, as stored
  int s, r0, len;
  Slot src;

  __device__ __forceinline__ void bounds(const Seqs& a, int seq) {
    s = seq;
    if (ONE || s >= a.n) return;
    b = load_index(a.cu, s, a.meta64);
    e = load_index(a.cu, s + 1, a.meta64);
    n = load_index(a.na, s, a.meta64);
  }
  __device__ __forceinline__ void slot(const Seqs& a) {
    if (s >= a.n) return;
    int pos = 0;
    if constexpr (ONE) {
      r0 = s;
      len = 1;
    } else {
      r0 = clamped(a.cu ? b.value(a.meta64) : (int64_t)s * a.steps, a.rows);
      const int end = clamped(a.cu ? e.value(a.meta64) : (int64_t)(s + 1) * a.steps, a.rows);
      len = end > r0 ? end - r0 : 0;
      const int64_t v = a.na ? n.value(a.meta64) - 1 : 0;
      pos = v < 0 || v > 0x7fffffff ? -1 : (int)v;
    }
    src = load_slot(a.src, s, pos, a.idx64);
  }
};

template <class ST, class IT, int N, bool ONE>
__global__ void __launch_bounds__(kScanWarps * 32, ScanStep<ST, N>::CTAS)
    scan_walk_kernel(const ScanArgs p, const Seqs a) {
  using K = ScanStep<ST, N>;
  using L = typename K::L;
  constexpr int U = K::U, VEC = L::VEC, CPL = L::CPL, H = L::EPL / 2;
  constexpr int LPU = L::LPR / U;  // lanes of a row that own the same channel's sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane % L::LPR, rr = lane / L::LPR;
  const int per = p.C / p.G, tiles = (per + K::CH - 1) / K::CH;
  const int g = blockIdx.x / tiles;
  const int t0 = (blockIdx.x - g * tiles) * K::CH + warp * L::RPW * U + rr;
  const int c0 = g * per + t0;                       // channel of u: c0 + u RPW
  const int cm = c0 + q / LPU * L::RPW;              // the one whose sum this lane ends up with
  const bool cm_ok = cm < (g + 1) * per;
  const int cl = cm_ok ? cm : (g + 1) * per - 1;     // lanes beyond the group read its last one's

  float2 A2[U][H];  // A log2 e
  bool c_ok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * L::RPW;
    c_ok[u] = c < (g + 1) * per;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      float f[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = 0.0f;
      if (c_ok[u]) load_floats<float, VEC>(p.A + c * p.A_rs + (q + k * L::LPR) * VEC, p.a_vec, f);
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i)
        A2[u][k * VEC / 2 + i] = make_float2(log2_rate(f[2 * i]), log2_rate(f[2 * i + 1]));
    }
  }
  const float Dc = p.D && cm_ok ? p.D[cm] : 0.0f;
  const float bias = p.bias && cm_ok ? p.bias[cm] : 0.0f;
  ST* state = static_cast<ST*>(p.state);
  const IT* xp = static_cast<const IT*>(p.x) + cl;
  const IT* zp = static_cast<const IT*>(p.z) + cl;
  const IT* Bp = static_cast<const IT*>(p.B) + g * p.B_gs + q * VEC;
  const IT* Cp = static_cast<const IT*>(p.Cm) + g * p.C_gs + q * VEC;

  uint4 raw[U][CPL];
  Words<IT, 1> x, z;
  uint32_t dt;  // as stored
  Words<IT, VEC> B[CPL], C[CPL];
  Slot to;
  z.zero();
  auto fetch_state = [&](int64_t slot, bool read) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < CPL; ++k) {
        raw[u][k] = make_uint4(0u, 0u, 0u, 0u);
        if (read && c_ok[u])
          raw[u][k] = ssu::ld_stream(state + (slot * p.C + c0 + u * L::RPW) * N +
                                     (q + k * L::LPR) * VEC);
      }
  };
  auto fetch_row = [&](int s, int t, int r) {
    x.load(xp + r * p.x_rs);
    if (p.z) z.load(zp + r * p.z_rs);
    if (p.dt_f32) dt = static_cast<const uint32_t*>(p.dt)[r * p.dt_rs + cl];
    else if constexpr (sizeof(IT) == 2)
      dt = static_cast<const uint16_t*>(p.dt)[r * p.dt_rs + cl];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      if (p.bc_vec) {
        B[k].load(Bp + r * p.B_rs + k * L::LPR * VEC);
        C[k].load(Cp + r * p.C_rs + k * L::LPR * VEC);
      } else {
        B[k].load_some(Bp + r * p.B_rs + k * L::LPR * VEC, VEC);
        C[k].load_some(Cp + r * p.C_rs + k * L::LPR * VEC, VEC);
      }
    }
    to = load_slot(a.dst, s, t, a.idx64);
  };

  const int stride = gridDim.y;
  Ahead<ONE> next, after;  // of the sequence after the one worked on, and of the one after that
  next.bounds(a, blockIdx.y);
  after.bounds(a, blockIdx.y + stride);
  // the next sequence that has rows, and its slot; the bounds of the one behind it
  auto advance = [&]() {
    while (true) {
      next.slot(a);
      if (next.s >= a.n || next.len > 0) return;
      next = after;
      after.bounds(a, next.s + stride);
    }
  };
  advance();
  if (next.s >= a.n) return;
  int64_t src = next.src.id(next.s, a.idx64);
  bool read = next.src.found && slot_ok(src, p.pad, p.slots);
  fetch_state(src, read);
  fetch_row(next.s, 0, next.r0);

  while (true) {
    const int s = next.s, r0 = next.r0, len = next.len;
    const bool keep = read && !p.disable;
    next = after;
    after.bounds(a, next.s + stride);
    advance();
    const bool more = next.s < a.n;
    float2 h[U][H];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < CPL; ++k) ssu::Elem<ST>::unpack2(raw[u][k], &h[u][k * VEC / 2]);

    for (int t = 0; t < len; ++t) {
      float2 Bv[H], Cv[H];
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
      const bool write = keep && to.found && slot_ok(dst, p.pad, p.slots);
      if (t + 1 < len) {
        fetch_row(s, t + 1, r0 + t + 1);
      } else if (more) {
        src = next.src.id(next.s, a.idx64);
        read = next.src.found && slot_ok(src, p.pad, p.slots);
        fetch_state(src, read);
        fetch_row(next.s, 0, next.r0);
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
      ssu::RowScatter<U, L::LPR / 2>::run(acc, q, base, plain);  // acc[0]: channel cm
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
        const int64_t o = (r0 + t) * p.o_rs + cm;
        if (p.out_f32) static_cast<float*>(p.out)[o] = y;
        else static_cast<IT*>(p.out)[o] = from_f<IT>(y);
      }
    }
    if (!more) break;
  }
}

template <class ST, class IT, int N>
cudaError_t launch_scan_step(const ScanArgs& p, const Seqs& a, cudaStream_t stream) {
  using K = ScanStep<ST, N>;
  const bool one = !a.cu && !a.na && a.steps == 1;
  auto kern = one ? scan_walk_kernel<ST, IT, N, true> : scan_walk_kernel<ST, IT, N, false>;
  const int per = p.C / p.G;
  const int64_t gx = (int64_t)p.G * ((per + K::CH - 1) / K::CH);
  if (gx > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // one wave: each CTA walks its share of the sequences with A in registers
  int fit = 0;
  const cudaError_t e =
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, kScanWarps * 32, 0);
  if (e != cudaSuccess) return e;
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
