// layer_conv.cu -- the depthwise causal convolution in front of the state
// update, with its own per-slot cache of rows.
//
// For channel c and row t of a sequence, with W taps and xs the rows that the
// slot held followed by the call's rows,
//     y[t][c] = act(bias[c] + sum_{j < W} weight[c][j] xs[t - (W - 1) + j][c])
// and the slot afterwards holds the last W - 1 rows of xs.  About 2 W + 4
// operations per element against 2 elements moved: bound by HBM.
#include "layer_common.cuh"

namespace layer {

struct ConvArgs {
  void* state;
  int64_t slots;
  int64_t C;
  const void* x;
  int64_t x_rs;
  void* out;
  int64_t o_rs;
  const void* weight;
  const void* bias;
  int w_vec;                // weight starts on a 16-byte boundary
  int silu;
  int disable;
  int64_t pad;
  const uint8_t* has_init;  // per sequence, or NULL: every valid slot is read
  int final_only;           // prompts: the state is written after a sequence's last row only
};

template <class WT, int W, int V>
__device__ __forceinline__ void load_weights(const ConvArgs& p, int64_t c, float (&w)[W][V],
                                             float (&bias)[V]) {
  const WT* wp = static_cast<const WT*>(p.weight) + c * W;
  // a thread's V W weights are side by side: whole 16 bytes where V channels are
  Pack<WT, V * W> raw;
  if (V > 1 && p.w_vec) {
    raw = load_pack<WT, V * W>(wp);
  } else {
#pragma unroll
    for (int i = 0; i < V * W; ++i) raw.v[i] = wp[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = to_f(raw.v[i * W + j]);
#pragma unroll
  for (int i = 0; i < V; ++i)
    bias[i] = p.bias ? to_f(static_cast<const WT*>(p.bias)[c + i]) : 0.0f;
}

// One row: xs holds the W rows that its taps read, oldest first.
template <class IT, int W, int V>
__device__ __forceinline__ Pack<IT, V> conv_row(const Pack<IT, V>* xs, const float (&w)[W][V],
                                                const float (&bias)[V], int act) {
  Pack<IT, V> y;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float acc = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) acc = fmaf(w[j][i], to_f(xs[j].v[i]), acc);
    y.v[i] = from_f<IT>(act ? silu(acc) : acc);
  }
  return y;
}

// Decode: a thread owns V channels of one sequence after another and walks the
// sequence's rows with the window of W - 1 rows in registers.
template <class IT, class WT, int W, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvArgs p, const VarlenArgs a,
                                                        int64_t nseqs) {
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (c >= p.C) return;
  float w[W][V], bias[V];
  load_weights<WT, W, V>(p, c, w, bias);
  const IT* x = static_cast<const IT*>(p.x) + c;
  IT* out = static_cast<IT*>(p.out) + c;
  IT* state = static_cast<IT*>(p.state) + c;
  for (int64_t s = blockIdx.y; s < nseqs; s += gridDim.y) {
    const Item it = packed_item(a, s, p.pad, p.slots);
    if (it.len == 0) continue;
    Pack<IT, V> xs[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      xs[j] = it.read_ok ? load_pack<IT, V>(state + (it.src * (W - 1) + j) * p.C) : zero_pack<IT, V>();
    for (int64_t t = 0; t < it.len; ++t) {
      xs[W - 1] = load_pack<IT, V>(x + (it.r0 + t) * p.x_rs);
      store_pack<IT, V>(out + (it.r0 + t) * p.o_rs, conv_row<IT, W, V>(xs, w, bias, p.silu));
      int64_t slot;
      if (it.read_ok && !p.disable && write_slot(a, s, t, p.pad, p.slots, &slot)) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
          store_pack<IT, V>(state + (slot * (W - 1) + j) * p.C, xs[j + 1]);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) xs[j] = xs[j + 1];
    }
  }
}

// First sequence s with cu[s + 1] > row (nseqs if there is none): the warp's
// lanes probe 32 places at a time.
__device__ __forceinline__ int64_t find_sequence(const VarlenArgs& a, int64_t nseqs, int64_t row) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, n = nseqs;
  while (n > 0) {
    const int64_t step = (n + 31) / 32;
    const int64_t last = (lane + 1) * step - 1;  // of this lane's block
    const bool before = last < n && load_int(a.cu, lo + last + 1, a.meta64) <= row;
    const int64_t skip = __popc(__ballot_sync(0xffffffffu, before)) * step;
    lo += skip;
    n = n - skip < step - 1 ? n - skip : step - 1;
  }
  return lo;
}

// Prompts: a thread owns V channels of a tile of rows, whatever sequences they
// belong to, and takes them kConvRows at a time: that many loads in flight,
// then the sliding window of W - 1 rows in fp32 registers.  Rows that reach
// back to a sequence's slot (its first W - 1) are all done by the tile that
// holds the sequence's first row, which also writes the slot afterwards: no
// other CTA reads a slot, so it may be written in place.
constexpr int kConvRows = 8;

template <class IT, class WT, int W, int V>
__global__ void __launch_bounds__(128) conv_prompt_kernel(const ConvArgs p, const VarlenArgs a,
                                                          int64_t nseqs, int tile_rows,
                                                          int ctiles) {
  const int64_t tile = blockIdx.x / ctiles;
  const int64_t c = ((int64_t)(blockIdx.x - tile * ctiles) * blockDim.x + threadIdx.x) * V;
  const int64_t t0 = tile * tile_rows;
  const int64_t t1 = t0 + tile_rows < a.rows ? t0 + tile_rows : a.rows;
  int64_t s = find_sequence(a, nseqs, t0);
  if (c >= p.C) return;
  float w[W][V], bias[V];
  load_weights<WT, W, V>(p, c, w, bias);
  const IT* x = static_cast<const IT*>(p.x) + c;
  IT* out = static_cast<IT*>(p.out) + c;
  IT* state = static_cast<IT*>(p.state) + c;

  for (; s < nseqs; ++s) {
    const Item it = packed_item(a, s, p.pad, p.slots);
    if (it.r0 >= t1) break;
    if (it.len == 0) continue;
    const int64_t end = it.r0 + it.len;
    const int64_t reach = it.r0 + W - 1 < end ? it.r0 + W - 1 : end;  // rows that see the slot
    const bool owner = it.r0 >= t0;
    int64_t r = owner ? it.r0 : (t0 > reach ? t0 : reach);
    const int64_t stop = end < t1 ? end : (owner && reach > t1 ? reach : t1);
    if (!owner && r >= stop) continue;
    const bool from = owner && it.read_ok && (!p.has_init || p.has_init[s]);
    Pack<IT, V> first[W - 1];  // the rows in front of r
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      if (!owner) first[j] = load_pack<IT, V>(x + (r - (W - 1) + j) * p.x_rs);
      else if (from) first[j] = load_pack<IT, V>(state + (it.src * (W - 1) + j) * p.C);
      else first[j] = zero_pack<IT, V>();
    }
    float xs[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) xs[j][i] = to_f(first[j].v[i]);
    auto row = [&](const Pack<IT, V>& in, int64_t at) {
      Pack<IT, V> y;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xs[W - 1][i] = to_f(in.v[i]);
        float acc = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) acc = fmaf(w[j][i], xs[j][i], acc);
        y.v[i] = from_f<IT>(p.silu ? silu(acc) : acc);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) xs[j][i] = xs[j + 1][i];
      }
      store_pack<IT, V>(out + at * p.o_rs, y);
    };
    for (; r + kConvRows <= stop; r += kConvRows) {
      Pack<IT, V> in[kConvRows];
#pragma unroll
      for (int k = 0; k < kConvRows; ++k) in[k] = load_pack<IT, V>(x + (r + k) * p.x_rs);
#pragma unroll
      for (int k = 0; k < kConvRows; ++k) row(in[k], r + k);
    }
    for (; r < stop; ++r) row(load_pack<IT, V>(x + r * p.x_rs), r);

    int64_t slot;
    if (owner && it.read_ok && !p.disable && write_slot(a, s, 0, p.pad, p.slots, &slot)) {
      Pack<IT, V> last[W - 1];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        last[j] = zero_pack<IT, V>();
        if (it.len + j >= W - 1) {
          last[j] = load_pack<IT, V>(x + (end - (W - 1) + j) * p.x_rs);
        } else {  // shorter than the window: rows of the slot are left in it
#pragma unroll
          for (int k = 0; k < W - 1; ++k)
            if (k == it.len + j) last[j] = first[k];
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        store_pack<IT, V>(state + (slot * (W - 1) + j) * p.C, last[j]);
    }
  }
}

constexpr int kStepThreads = 128;

template <class IT, class WT, int W, int V>
cudaError_t launch_step(const ConvArgs& p, const VarlenArgs& a, int64_t nseqs,
                        cudaStream_t stream) {
  const int64_t gx = (p.C / V + kStepThreads - 1) / kStepThreads;
  const int64_t gy = nseqs < 65535 ? nseqs : 65535;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  conv_step_kernel<IT, WT, W, V>
      <<<dim3((unsigned)gx, (unsigned)gy), kStepThreads, 0, stream>>>(p, a, nseqs);
  return cudaGetLastError();
}

template <class IT, class WT, int W, int V>
cudaError_t launch_prompt(const ConvArgs& p, const VarlenArgs& a, int64_t nseqs,
                          cudaStream_t stream) {
  const int64_t ctiles = (p.C / V + kStepThreads - 1) / kStepThreads;
  // rows per thread: fewer than 64 while the SMs are not full (16 CTAs each)
  int rows = 64;
  while (rows > kConvRows && a.rows / rows * ctiles < 16LL * ssu::sm_count()) rows /= 2;
  const int64_t grid = ctiles * ((a.rows + rows - 1) / rows);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  conv_prompt_kernel<IT, WT, W, V>
      <<<(unsigned)grid, kStepThreads, 0, stream>>>(p, a, nseqs, rows, (int)ctiles);
  return cudaGetLastError();
}

// Channels per thread: 16 bytes of a row where every row starts on a 16-byte
// boundary, 4 bytes (two 16-bit channels) on 4-byte boundaries, else one.
template <class IT, class WT, int W>
cudaError_t launch_width(const ConvArgs& p, const VarlenArgs& a, int64_t nseqs,
                         cudaStream_t stream) {
  constexpr int B = (int)sizeof(IT);
  auto rows_on = [&](int64_t bytes) {
    return aligned(p.x, bytes) && aligned(p.out, bytes) && aligned(p.state, bytes) &&
           p.x_rs * B % bytes == 0 && p.o_rs * B % bytes == 0 && p.C * B % bytes == 0;
  };
  auto launch = [&](auto v) {
    constexpr int V = decltype(v)::value;
    return p.final_only ? launch_prompt<IT, WT, W, V>(p, a, nseqs, stream)
                        : launch_step<IT, WT, W, V>(p, a, nseqs, stream);
  };
  if (rows_on(16)) return launch(std::integral_constant<int, 16 / B>{});
  if constexpr (B == 2) {
    if (rows_on(4)) return launch(std::integral_constant<int, 2>{});
  }
  return launch(std::integral_constant<int, 1>{});
}

template <class IT, class WT>
cudaError_t launch_types(int W, const ConvArgs& p, const VarlenArgs& a, int64_t nseqs,
                         cudaStream_t stream) {
  switch (W) {
    case 2: return launch_width<IT, WT, 2>(p, a, nseqs, stream);
    case 3: return launch_width<IT, WT, 3>(p, a, nseqs, stream);
    case 4: return launch_width<IT, WT, 4>(p, a, nseqs, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_conv(const ssu_conv_params* c, const ConvArgs& p, const VarlenArgs& a,
                        int64_t nseqs, cudaStream_t stream) {
  const int W = (int)c->width;
  const bool f32w = c->weight_dtype == SSU_F32;
  switch (c->io_dtype) {
    case SSU_F32: return launch_types<float, float>(W, p, a, nseqs, stream);
    case SSU_BF16:
      return f32w ? launch_types<__nv_bfloat16, float>(W, p, a, nseqs, stream)
                  : launch_types<__nv_bfloat16, __nv_bfloat16>(W, p, a, nseqs, stream);
    case SSU_F16:
      return f32w ? launch_types<__half, float>(W, p, a, nseqs, stream)
                  : launch_types<__half, __half>(W, p, a, nseqs, stream);
    default: return cudaErrorInvalidValue;
  }
}

ssu_status check_conv(const ssu_conv_params* c, int64_t rows, bool pool_needed, ConvArgs* p) {
  if (!c) return fail(SSU_ERR_INVALID_ARGUMENT, "params must not be NULL");
  if (!is_float(c->io_dtype))
    return fail(SSU_ERR_UNSUPPORTED, "x must be f32, bf16 or f16");
  if (c->weight_dtype != c->io_dtype && c->weight_dtype != SSU_F32)
    return fail(SSU_ERR_INVALID_ARGUMENT, "weight and bias must have the x dtype or be f32");
  if (c->channels < 1 || c->slots < 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "channels must be positive and slots >= 0, got %lld, %lld",
                (long long)c->channels, (long long)c->slots);
  if (c->channels > (1 << 24)) return fail(SSU_ERR_UNSUPPORTED, "channels must not exceed 2^24");
  if (c->width < 2 || c->width > 4)
    return fail(SSU_ERR_UNSUPPORTED, "width %lld is not one of 2, 3, 4", (long long)c->width);
  if (c->activation != SSU_ACT_NONE && c->activation != SSU_ACT_SILU)
    return fail(SSU_ERR_INVALID_ARGUMENT, "activation must be none or silu, got %d", c->activation);
  if (rows > 0 && (!c->x || !c->out || !c->weight))
    return fail(SSU_ERR_INVALID_ARGUMENT, "x, out and weight must not be NULL");
  if (rows > 1 && c->out_row_stride < c->channels)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out rows overlap: a stride of %lld for %lld channels",
                (long long)c->out_row_stride, (long long)c->channels);
  if (pool_needed && !c->conv_state && c->slots > 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "conv_state must not be NULL");
  const int es = size_of(c->io_dtype);
  if (!aligned(c->x, es) || !aligned(c->out, es) || !aligned(c->conv_state, es) ||
      !aligned(c->weight, size_of(c->weight_dtype)) || !aligned(c->bias, size_of(c->weight_dtype)))
    return fail(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their element size");
  *p = ConvArgs{};
  p->state = c->conv_state;
  p->slots = c->conv_state ? c->slots : 0;
  p->C = c->channels;
  p->x = c->x;
  p->x_rs = c->x_row_stride;
  p->out = c->out;
  p->o_rs = c->out_row_stride;
  p->weight = c->weight;
  p->bias = c->bias;
  p->w_vec = aligned(c->weight, 16);
  p->silu = c->activation == SSU_ACT_SILU;
  p->disable = c->disable_state_update != 0;
  p->pad = c->pad_slot_id;
  return SSU_OK;
}

}  // namespace layer

#pragma GCC visibility push(default)
extern "C" {

ssu_status ssu_conv_update(const ssu_conv_params* c, int64_t nseqs, int64_t rows,
                           const void* cu_seqlens, int64_t dense_steps,
                           const void* num_accepted_tokens, ssu_dtype meta_dtype,
                           const ssu_slot_table* src, const ssu_slot_table* dst,
                           ssu_dtype index_dtype, struct CUstream_st* stream) {
  using namespace layer;
  ConvArgs p;
  VarlenArgs a;
  ssu_status st = check_conv(c, rows, true, &p);
  if (st == SSU_OK)
    st = check_packed(c->slots, nseqs, rows, cu_seqlens, dense_steps, num_accepted_tokens,
                      meta_dtype, src, dst, index_dtype, &a);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  return launched(launch_conv(c, p, a, nseqs, (cudaStream_t)stream));
}

ssu_status ssu_conv_fwd_varlen(const ssu_conv_params* c, int64_t nseqs, int64_t rows,
                               const void* cu_seqlens, ssu_dtype meta_dtype,
                               const void* state_batch_indices,
                               const void* dst_state_batch_indices, ssu_dtype index_dtype,
                               const uint8_t* has_initial_state, struct CUstream_st* stream) {
  using namespace layer;
  ConvArgs p;
  VarlenArgs a;
  ssu_status st = check_conv(c, rows, false, &p);
  if (st == SSU_OK)
    st = check_prompts(c->conv_state != nullptr, c->slots, nseqs, rows, cu_seqlens, meta_dtype,
                       state_batch_indices, dst_state_batch_indices, index_dtype, &a);
  if (st != SSU_OK) return st;
  if (rows > 0 && c->x == c->out)
    return fail(SSU_ERR_INVALID_ARGUMENT, "out must not be x: rows are read by several blocks");
  if (nseqs == 0 || rows == 0) return ok();
  p.has_init = has_initial_state;
  p.final_only = 1;
  return launched(launch_conv(c, p, a, nseqs, (cudaStream_t)stream));
}

}  // extern "C"
#pragma GCC visibility pop
