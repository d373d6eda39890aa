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

// A slot table: entry (s, t) is idx[s ss + t ts], 0 <= t < steps, below numel.
struct Table {
  const void* idx;  // nullptr: slot s
  int64_t numel;
  int ss, ts, steps;
};

// The sequences of a call.
struct Seqs {
  int rows, n;
  const void* cu;  // nullptr: `steps` rows each
  int steps;
  const void* na;  // nullptr: the read table's entry 0
  int meta64, idx64;
  Table src, dst;  // slots read, slots written
};

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
                        ssu_dtype index_dtype, Seqs* out);

// ... and by the prompt-form calls (ssu_conv_fwd_varlen, ssu_scan_fwd_varlen).
ssu_status check_prompts(bool pool, int64_t slots, int64_t nseqs, int64_t rows, const void* cu,
                         ssu_dtype meta_dtype, const void* src, const void* dst,
                         ssu_dtype index_dtype, Seqs* out);

// An operand's memory: in each row `pieces` runs of `bytes` bytes, piece_stride apart.
struct Rows {
  const void* p;
  int64_t stride, bytes;
  int64_t pieces = 1, piece_stride = 0;
};

// Whether two operands of `rows` rows share a byte.  Columns of one wider tensor
// lie between each other's rows and do not.
bool overlap(const Rows& a, const Rows& b, int64_t rows);

// Rows of `n` elements, and of groups of them.
inline Rows rows_of(const void* p, int64_t stride, int64_t n, ssu_dtype d) {
  return Rows{p, stride * size_of(d), n * size_of(d)};
}
inline Rows rows_of(const void* p, int64_t stride, int64_t groups, int64_t group_stride, int64_t n,
                    ssu_dtype d) {
  const int64_t es = size_of(d);
  if (groups == 1 || group_stride == n) return Rows{p, stride * es, groups * n * es};
  return Rows{p, stride * es, n * es, groups, group_stride * es};
}

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

// V elements as stored, in 32-bit words.
template <class T, int V>
struct Words {
  static constexpr int BYTES = V * (int)sizeof(T), NW = (BYTES + 3) / 4;
  uint32_t w[NW];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    else return __half2float(__ushort_as_half((unsigned short)(w[i >> 1] >> (i & 1 ? 16 : 0))));
  }
  // elements 2 i and 2 i + 1 (zero beyond V)
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(at(2 * i), 2 * i + 1 < V ? at(2 * i + 1) : 0.0f);
  }
  // all V, from (V + 1) / 2 pairs, rounded to nearest even
  __device__ __forceinline__ void set(const float2* f) {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(f[i].x);
        if (2 * i + 1 < V) w[2 * i + 1] = __float_as_uint(f[i].y);
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 v = __float22bfloat162_rn(f[i]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __float22half2_rn(f[i]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  }
  __device__ __forceinline__ void load(const T* p) {  // from a multiple of 16 bytes, or of BYTES
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void load_some(const T* p, int n) {  // elements [0, n), zeros beyond
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (i & 1 ? 16 : 0);
      }
  }
};

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

// A log2 e, held to the largest finite value (NaN stays).  An infinite one would
// turn a step of zero, which has to change nothing, into 0 x infinity; held, a
// column with A = -infinity still forgets at once: 2^(A dt') is 0 for every dt'
// of 2^-120 or more (a smaller one, where infinity would do, forgets in part).
__device__ __forceinline__ float log2_rate(float a) {
  float r = a * kLog2e;
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(-3.402823466e38f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(3.402823466e38f));
  return r;
}

__device__ __forceinline__ float silu(float v) {
  return __fdividef(v, 1.0f + ex2(-v * kLog2e));
}

__device__ __forceinline__ float2 silu2(float2 v) {
  const float2 e = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
  const float2 s = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), make_float2(1.0f, 1.0f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(s.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(s.y));
  return __fmul2_rn(v, r);
}

// softplus(a + b) = log(1 + e^v) = max(v, 0) + log1p(e^-|v|), v = a + b.  Far
// below zero the result is e^v itself, which turns an error of v into a
// relative one: so the exponent's product with log2 e is carried in two parts
// (Dekker), what the sum a + b lost (Knuth's two-sum) is put back, and e^(v + d)
// = e^v (1 + d) to first order.  log1p(u) = u P(u) on [0, 1], P the degree 8
// least-maximum fit of log1p(u) / u (relative error 1.8e-7 in fp32).  NaN comes
// through `lost`; infinities have none.
__device__ __forceinline__ float softplus_from(float v, float lost) {
  const float m = fmaxf(-fabsf(v), -150.0f);  // below, the exponential is zero in fp32
  const float hi = m * kLog2e;
  float d = fmaf(m, kLog2e, -hi);
  d = fmaf(m, 1.92596299e-8f, d);  // log2 e - kLog2e
  d = fmaf(d, 0.693147181f, lost);
  float u = ex2(hi);
  u = fmaf(u, d, u);
  float l = 0.0052326880395412445f;
  l = fmaf(l, u, -0.029505213722586632f);
  l = fmaf(l, u, 0.07822591066360474f);
  l = fmaf(l, u, -0.13663242757320404f);
  l = fmaf(l, u, 0.19106005132198334f);
  l = fmaf(l, u, -0.2484298199415207f);
  l = fmaf(l, u, 0.3331909775733948f);
  l = fmaf(l, u, -0.4999949336051941f);
  l = fmaf(l, u, 0.9999999403953552f);
  return fmaf(l, u, fmaxf(v, 0.0f));
}

__device__ __forceinline__ float softplus_sum(float a, float b) {
  const float v = a + b;
  const float part = v - a;
  const float lost = (a - (v - part)) + (b - part);
  return softplus_from(v, fabsf(v) == INFINITY ? 0.0f : lost);
}

// ... of V sums at once.  What a sum lost is below 2^-21 of the result unless v
// is below -16 (or not finite): only then is it put back, for each sum by itself,
// so that no channel's bits depend on its neighbours'.
template <int V>
__device__ __forceinline__ void softplus_sums(float* a, const float* b) {
  float v[V];
  bool near = true;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = a[i] + b[i];
    near = near && v[i] > -16.0f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = softplus_from(v[i], 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float part = v[i] - a[i];
      const float lost = (a[i] - (v[i] - part)) + (b[i] - part);
      a[i] = softplus_from(v[i], v[i] > -16.0f || v[i] == -INFINITY ? 0.0f : lost);
    }
  }
}

// ---------------------------------------------------------------------------
// device: rows and slots of packed sequence s
// ---------------------------------------------------------------------------
// An index as stored: two 32-bit words (one twice where indices are 32 bits
// wide).  Absent arrays read zeros.  Loading and looking at it are apart, with
// no choice between kinds of load in between, so that the loads of a call's
// metadata wait for each other only where one needs the other's value.
__device__ const int kNoIndex[2] = {0, 0};

struct RawIndex {
  int lo, hi;
  __device__ __forceinline__ int64_t value(int is64) const {
    return is64 ? (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo) : (int64_t)lo;
  }
};

__device__ __forceinline__ RawIndex load_index(const void* p, int64_t i, int is64) {
  const int* w = p ? static_cast<const int*>(p) + (i << is64) : kNoIndex;
  return RawIndex{w[0], w[is64]};
}

// Entry (s, pos) of a slot table, as stored; `found` is false where the table
// has no such entry.  Without a table the slot is s itself.
struct Slot {
  RawIndex raw;
  bool found, table;
  __device__ __forceinline__ int64_t id(int s, int is64) const {
    return table ? raw.value(is64) : s;
  }
};

__device__ __forceinline__ Slot load_slot(const Table& t, int s, int pos, int is64) {
  const int64_t e = (int64_t)s * t.ss + (int64_t)pos * t.ts;
  Slot slot;
  slot.table = t.idx != nullptr;
  const bool inside = (unsigned)pos < (unsigned)t.steps && e < t.numel;
  slot.found = inside || !slot.table;
  slot.raw = load_index(inside ? t.idx : nullptr, e, is64);
  return slot;
}

struct Item {
  int r0, len;   // first row, rows (0: an empty sequence, nothing to do)
  int64_t src;   // slot read
  bool read_ok;  // ... when it is a valid one; else the sequence runs from zeros and writes none
};

__device__ __forceinline__ int clamped(int64_t v, int most) {
  return v < 0 ? 0 : v < most ? (int)v : most;
}

// ONE: every sequence is one row and reads entry 0 of its table.
template <bool ONE = false>
__device__ __forceinline__ Item packed_item(const Seqs& a, int s, int64_t pad, int64_t slots) {
  Item it;
  Slot read;
  if constexpr (ONE) {
    read = load_slot(a.src, s, 0, a.idx64);
    it.r0 = s;
    it.len = 1;
  } else {
    const RawIndex b = load_index(a.cu, s, a.meta64), e = load_index(a.cu, s + 1, a.meta64);
    const RawIndex n = load_index(a.na, s, a.meta64);
    const int64_t pos = a.na ? n.value(a.meta64) - 1 : 0;
    read = load_slot(a.src, s, pos < 0 || pos > 0x7fffffff ? -1 : (int)pos, a.idx64);
    it.r0 = clamped(a.cu ? b.value(a.meta64) : (int64_t)s * a.steps, a.rows);
    const int end = clamped(a.cu ? e.value(a.meta64) : (int64_t)(s + 1) * a.steps, a.rows);
    it.len = end > it.r0 ? end - it.r0 : 0;
  }
  it.src = read.id(s, a.idx64);
  it.read_ok = read.found && slot_ok(it.src, pad, slots);
  return it;
}

// Slot that takes the state after row t of sequence s.
__device__ __forceinline__ bool write_slot(const Seqs& a, int s, int t, int64_t pad, int64_t slots,
                                           int64_t* slot) {
  const Slot to = load_slot(a.dst, s, t, a.idx64);
  *slot = to.id(s, a.idx64);
  return to.found && slot_ok(*slot, pad, slots);
}

}  // namespace layer
