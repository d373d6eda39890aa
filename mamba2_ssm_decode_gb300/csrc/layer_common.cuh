// layer_common.cuh -- what the kernels around the state update share: element
// types and vectors, the fast exponential and gate, the rows and slots of a
// packed sequence, and the host-side argument checks.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "../../include/ssu.h"
#include "ssu_kernel.cuh"

namespace ssu {
ssu_status record_error(ssu_status code, const char* message);  // ssu_abi.cu
int sm_count();                                                  // ssu_abi.cu
}  // namespace ssu

namespace layer {
using ssu::load_int;
using ssu::slot_ok;
using ssu::TableArgs;
using ssu::VarlenArgs;

// ---------------------------------------------------------------------------
// host: errors and checks
// ---------------------------------------------------------------------------
inline ssu_status fail(ssu_status code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return ssu::record_error(code, buf);
}

inline ssu_status ok() { return ssu::record_error(SSU_OK, ""); }

inline ssu_status launched(cudaError_t e) {
  if (e != cudaSuccess)
    return fail(SSU_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(e));
  return ok();
}

inline bool is_index(ssu_dtype d) { return d == SSU_I32 || d == SSU_I64; }
inline bool is_float(ssu_dtype d) { return d == SSU_F32 || d == SSU_BF16 || d == SSU_F16; }
inline int size_of(ssu_dtype d) { return d == SSU_F32 || d == SSU_I32 ? 4 : d == SSU_I64 ? 8 : 2; }
inline bool aligned(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// Sequence metadata shared by the decode-form calls (ssu_conv_update,
// ssu_scan_update): the checks of ssu_update_varlen.
ssu_status check_packed(int64_t slots, int64_t nseqs, int64_t rows, const void* cu,
                        int64_t dense_steps, const void* na, ssu_dtype meta_dtype,
                        const ssu_slot_table* src, const ssu_slot_table* dst,
                        ssu_dtype index_dtype, VarlenArgs* out);

// ... and by the prompt-form calls (ssu_conv_fwd_varlen, ssu_scan_fwd_varlen).
ssu_status check_prompts(bool pool, int64_t slots, int64_t nseqs, int64_t rows, const void* cu,
                         ssu_dtype meta_dtype, const void* src, const void* dst,
                         ssu_dtype index_dtype, VarlenArgs* out);

// ---------------------------------------------------------------------------
// device: elements
// ---------------------------------------------------------------------------
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
  return __float2half_rn(v);
}

// V consecutive elements of type T, moved in accesses of the largest power of
// two up to 16 bytes that divides their size.
template <class T, int V>
struct alignas((sizeof(T) * V & -(sizeof(T) * V)) < 16 ? (sizeof(T) * V & -(sizeof(T) * V)) : 16)
    Pack {
  T v[V];
};

template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}

template <class T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& v) {
  *reinterpret_cast<Pack<T, V>*>(p) = v;
}

template <class T, int V>
__device__ __forceinline__ Pack<T, V> zero_pack() {
  Pack<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) z.v[i] = from_f<T>(0.0f);
  return z;
}

// V consecutive elements as fp32: one vector access where `vec` says that the
// address allows it, else element by element.
template <class T, int V>
__device__ __forceinline__ void load_floats(const T* p, bool vec, float* f) {
  if (vec) {
    const Pack<T, V> r = load_pack<T, V>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f(r.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f(p[i]);
  }
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^v, results below the smallest normal flushed to zero
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float silu(float v) {
  return __fdividef(v, 1.0f + ex2(-v * kLog2e));
}

// softplus(a + b) = log(1 + e^v) = max(v, 0) + log1p(e^-|v|), v = a + b, for
// two values at once (the packed fp32 pipe).  Far below zero the result is e^v
// itself, which turns an error of v into a relative one: so the exponent's
// product with log2 e is carried in two parts (Dekker), what the sum a + b lost
// (Knuth's two-sum) is put back, and e^(v + d) = e^v (1 + d) to first order.
// log1p(u) = u P(u) on [0, 1], P the degree 8 least-maximum fit of log1p(u) / u
// (relative error 1.8e-7 in fp32).  NaN comes through `lost`; infinities have
// none.
__device__ __forceinline__ float2 softplus_sum2(float2 a, float2 b) {
  const float2 minus = make_float2(-1.0f, -1.0f);
  const float2 v = __fadd2_rn(a, b);
  const float2 part = __ffma2_rn(a, minus, v);
  float2 lost = __fadd2_rn(__ffma2_rn(__ffma2_rn(part, minus, v), minus, a),
                           __ffma2_rn(part, minus, b));
  if (fabsf(v.x) == INFINITY) lost.x = 0.0f;
  if (fabsf(v.y) == INFINITY) lost.y = 0.0f;
  // below -150 the exponential is zero in fp32
  const float2 m = make_float2(fmaxf(-fabsf(v.x), -150.0f), fmaxf(-fabsf(v.y), -150.0f));
  const float2 l2e = make_float2(1.44269502e+0f, 1.44269502e+0f);
  const float2 hi = __fmul2_rn(m, l2e);
  float2 d = __ffma2_rn(m, l2e, __fmul2_rn(hi, minus));
  d = __ffma2_rn(m, make_float2(1.92596299e-8f, 1.92596299e-8f), d);  // log2 e - l2e
  d = __ffma2_rn(d, make_float2(0.693147181f, 0.693147181f), lost);
  float2 u = make_float2(ex2(hi.x), ex2(hi.y));
  u = __ffma2_rn(u, d, u);
  constexpr float P[9] = {0.9999999403953552f, -0.4999949336051941f, 0.3331909775733948f,
                          -0.2484298199415207f, 0.19106005132198334f, -0.13663242757320404f,
                          0.07822591066360474f, -0.029505213722586632f, 0.0052326880395412445f};
  float2 l = make_float2(P[8], P[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) l = __ffma2_rn(l, u, make_float2(P[i], P[i]));
  return __ffma2_rn(l, u, make_float2(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
}

__device__ __forceinline__ float softplus_sum(float a, float b) {
  return softplus_sum2(make_float2(a, a), make_float2(b, b)).x;
}

// ---------------------------------------------------------------------------
// device: rows and slots of packed sequence s
// ---------------------------------------------------------------------------
struct Item {
  int64_t r0;      // first row
  int64_t len;     // rows (0: an empty sequence, nothing to do)
  int64_t src;     // slot read
  bool read_ok;    // ... when it is a valid one; else the sequence runs from zeros and writes none
};

__device__ __forceinline__ Item packed_item(const VarlenArgs& a, int64_t s, int64_t pad,
                                            int64_t slots) {
  Item it;
  int64_t begin, end;
  if (a.cu) {
    begin = load_int(a.cu, s, a.meta64);
    end = load_int(a.cu, s + 1, a.meta64);
  } else {
    begin = s * a.dense_steps;
    end = begin + a.dense_steps;
  }
  if (begin < 0) begin = 0;
  if (end > a.rows) end = a.rows;
  it.r0 = begin;
  it.len = end > begin ? end - begin : 0;
  it.src = s;
  bool found = true;
  if (a.src.idx) {
    const int64_t col = a.na ? load_int(a.na, s, a.meta64) - 1 : 0;
    found = ssu::table_entry(a.src, s, col, a.idx64, &it.src);
  }
  it.read_ok = found && slot_ok(it.src, pad, slots);
  return it;
}

// Slot that takes the state after row t of sequence s: entry t of the write
// table, of the read table without one, slot s without either.
__device__ __forceinline__ bool write_slot(const VarlenArgs& a, int64_t s, int64_t t, int64_t pad,
                                           int64_t slots, int64_t* slot) {
  bool found = true;
  if (a.dst.idx) found = ssu::table_entry(a.dst, s, t, a.idx64, slot);
  else if (a.src.idx) found = ssu::table_entry(a.src, s, t, a.idx64, slot);
  else *slot = s;
  return found && slot_ok(*slot, pad, slots);
}

}  // namespace layer
