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
  int w_vec;                // weight and bias start on 16-byte boundaries
  int silu;
  int disable;
  int64_t pad;
  const uint8_t* has_init;  // per sequence, or NULL: every valid slot is read
  int prompt;               // the prompt form: the state is written after a sequence's last row only
};

// A thread's V W weights and V biases are side by side: whole vectors where V
// channels are, fp32 pairs of neighbouring channels in registers.
template <class WT, int W, int V>
__device__ __forceinline__ void load_weights(const ConvArgs& p, int64_t c,
                                             float2 (&w)[W][(V + 1) / 2],
                                             float2 (&bias)[(V + 1) / 2]) {
  const WT* wp = static_cast<const WT*>(p.weight) + c * W;
  const WT* bp = static_cast<const WT*>(p.bias) + c;
  Pack<WT, V * W> raw;
  Pack<WT, V> b = zero_pack<WT, V>();
  if (V > 1 && p.w_vec) {
    raw = load_pack<WT, V * W>(wp);
    if (p.bias) b = load_pack<WT, V>(bp);
  } else {
#pragma unroll
    for (int i = 0; i < V * W; ++i) raw.v[i] = wp[i];
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (p.bias) b.v[i] = bp[i];
  }
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) {
    const int k = 2 * i + 1 < V ? 2 * i + 1 : 2 * i;
#pragma unroll
    for (int j = 0; j < W; ++j)
      w[j][i] = make_float2(to_f(raw.v[2 * i * W + j]), to_f(raw.v[k * W + j]));
    bias[i] = make_float2(to_f(b.v[2 * i]), to_f(b.v[k]));
  }
}

// One row: xs holds the W rows that its taps read, oldest first.
template <class IT, int W, int V>
__device__ __forceinline__ void conv_row(IT* out, const float2 (&xs)[W][(V + 1) / 2],
                                         const float2 (&w)[W][(V + 1) / 2],
                                         const float2 (&bias)[(V + 1) / 2], int act) {
  float2 y[(V + 1) / 2];
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) {
    y[i] = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) y[i] = __ffma2_rn(w[j][i], xs[j][i], y[i]);
    if (act) y[i] = silu2(y[i]);
  }
  Words<IT, V> r;
  r.set(y);
  r.store(out);
}

// Decode: a thread owns V channels of one sequence after another and walks the
// sequence's rows with the window of W - 1 rows in registers.  What it needs
// of up to ROWS rows (the rows, and the slots that take the state after them)
// is asked for at once, beside the slot's rows.  ROWS 1: one row a sequence.
// Bound by the latency of three dependent loads (count, slot, rows) in two or
// three waves of CTAs: 640 drafted rows x 5376 channels take 14.4 us for 43 MB.
// Eight CTAs an SM (64 registers, at which the drafted instance spills 28
// bytes): 1024 one-row sequences 22.5 us where the 6 that registers would leave
// take 26; with drafted rows the two are alike (256 sequences 12.5 us both, 1024
// sequences 42.3 and 43.3, on inputs partly in L2).
constexpr int kStepThreads = 128;

template <class IT, class WT, int W, int V, int ROWS>
__global__ void __launch_bounds__(kStepThreads, sizeof(IT) == 2 ? 8 : 5)
    conv_step_kernel(const ConvArgs p, const Seqs a) {
  const int64_t c = ((int64_t)blockIdx.x * kStepThreads + threadIdx.x) * V;
  if (c >= p.C) return;
  constexpr int P = (V + 1) / 2;
  float2 w[W][P], bias[P];
  load_weights<WT, W, V>(p, c, w, bias);
  const IT* x = static_cast<const IT*>(p.x) + c;
  IT* out = static_cast<IT*>(p.out) + c;
  IT* state = static_cast<IT*>(p.state) + c;
  for (int s = blockIdx.y; s < a.n; s += gridDim.y) {
    const Item it = packed_item<ROWS == 1>(a, s, p.pad, p.slots);
    if (it.len == 0) continue;
    Words<IT, V> in[W - 1 + ROWS];  // the window, then the rows, as stored
    float2 xs[W][P];
    for (int t0 = 0; t0 < it.len; t0 += ROWS) {
      const int n = it.len - t0 < ROWS ? it.len - t0 : ROWS;
      Slot to[ROWS];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        if (k < n) {
          in[W - 1 + k].load(x + (it.r0 + t0 + k) * p.x_rs);
          to[k] = load_slot(a.dst, s, t0 + k, a.idx64);
        }
      }
      if (t0 == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          if (it.read_ok) in[j].load(state + (it.src * (W - 1) + j) * p.C);
          else in[j].zero();
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int i = 0; i < P; ++i) xs[j][i] = in[j].pair(i);
      }
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int i = 0; i < P; ++i) xs[W - 1][i] = in[W - 1 + k].pair(i);
        conv_row<IT, W, V>(out + (it.r0 + t0 + k) * p.o_rs, xs, w, bias, p.silu);
        const int64_t slot = to[k].id(s, a.idx64);
        if (it.read_ok && !p.disable && to[k].found && slot_ok(slot, p.pad, p.slots)) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            in[k + 1 + j].store(state + (slot * (W - 1) + j) * p.C);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int i = 0; i < P; ++i) xs[j][i] = xs[j + 1][i];
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) in[j] = in[ROWS + j];
    }
  }
}

// First sequence s with cu[s + 1] > row (a.n if there is none): the warp's
// lanes probe 32 places at a time.
__device__ __forceinline__ int find_sequence(const Seqs& a, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int64_t last = (int64_t)(lane + 1) * step - 1;  // of this lane's block
    const bool before = last < n && load_int(a.cu, lo + last + 1, a.meta64) <= row;
    const int64_t skip = (int64_t)__popc(__ballot_sync(0xffffffffu, before)) * step;
    lo += (int)skip;
    n = n - skip < step - 1 ? (int)(n - skip) : step - 1;
  }
  return lo;
}

// Prompts: a thread owns V channels of a tile of rows, whatever sequences they
// belong to, and takes them kConvRows at a time: that many loads in flight,
// then the sliding window of W - 1 rows in fp32 registers.  Rows that reach
// back to a sequence's slot (its first W - 1) are all done by the tile that
// holds the sequence's first row, which also writes the slot afterwards: no
// other CTA reads a slot, so it may be written in place.
//
// Bound by HBM and the latency of its loads: 20634 x 5376 bf16 rows take 85 us,
// 444 MB at 5.2 TB/s; the same walk without the arithmetic takes 73 us.
template <class IT>
constexpr int kRowsInFlight = sizeof(IT) == 2 ? 8 : 4;
constexpr int kPromptThreads = 128;

template <class IT, class WT, int W, int V>
__global__ void __launch_bounds__(kPromptThreads, sizeof(IT) == 2 ? 6 : 4)
    conv_prompt_kernel(const ConvArgs p, const Seqs a, int tile_rows,
                       int ctiles) {
  constexpr int kConvRows = kRowsInFlight<IT>;
  const int tile = blockIdx.x / ctiles;
  const int64_t c = ((int64_t)(blockIdx.x - tile * ctiles) * kPromptThreads + threadIdx.x) * V;
  const int t0 = tile * tile_rows;  // below a.rows
  const int t1 = a.rows - t0 < tile_rows ? a.rows : t0 + tile_rows;
  int s = find_sequence(a, t0);
  if (c >= p.C) return;
  constexpr int P = (V + 1) / 2;
  float2 w[W][P], bias[P];
  load_weights<WT, W, V>(p, c, w, bias);
  const IT* x = static_cast<const IT*>(p.x) + c;
  IT* out = static_cast<IT*>(p.out) + c;
  IT* state = static_cast<IT*>(p.state) + c;

  for (; s < a.n; ++s) {
    const Item it = packed_item(a, s, p.pad, p.slots);
    if (it.r0 >= t1) break;
    if (it.len == 0) continue;
    const int end = it.r0 + it.len;
    const int reach = it.len > W - 1 ? it.r0 + W - 1 : end;  // rows that see the slot
    const bool owner = it.r0 >= t0;
    int r = owner ? it.r0 : (t0 > reach ? t0 : reach);
    const int stop = end < t1 ? end : (owner && reach > t1 ? reach : t1);
    if (!owner && r >= stop) continue;
    const bool from = owner && it.read_ok && (!p.has_init || p.has_init[s]);
    Words<IT, V> first[W - 1];  // the rows in front of r
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      if (!owner) first[j].load(x + (r - (W - 1) + j) * p.x_rs);
      else if (from) first[j].load(state + (it.src * (W - 1) + j) * p.C);
      else first[j].zero();
    }
    float2 xs[W][P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) xs[j][i] = first[j].pair(i);
    // kConvRows loads are always in flight: a row's place takes the row
    // kConvRows on (the last one again beyond the end) as soon as it is in xs
    Words<IT, V> in[kConvRows];
    const IT* xf = x + r * p.x_rs;  // the row to fetch next
    int behind = stop - 1 - r;      // rows behind it
    IT* o = out + r * p.o_rs;
    auto fetch = [&](int k) {
      in[k].load(xf);
      if (behind > 0) {
        xf += p.x_rs;
        --behind;
      }
    };
    auto row = [&](int k) {
#pragma unroll
      for (int i = 0; i < P; ++i) xs[W - 1][i] = in[k].pair(i);
      fetch(k);
      conv_row<IT, W, V>(o, xs, w, bias, p.silu);
      o += p.o_rs;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) xs[j][i] = xs[j + 1][i];
    };
#pragma unroll
    for (int k = 0; k < kConvRows; ++k) fetch(k);
    for (; stop - r >= kConvRows; r += kConvRows) {
#pragma unroll
      for (int k = 0; k < kConvRows; ++k) row(k);
    }
#pragma unroll
    for (int k = 0; k < kConvRows - 1; ++k)
      if (stop - r > k) row(k);

    int64_t slot;
    if (owner && it.read_ok && !p.disable && write_slot(a, s, 0, p.pad, p.slots, &slot)) {
      Words<IT, V> last[W - 1];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        if (it.len + j >= W - 1) {
          last[j].load(x + (end - (W - 1) + j) * p.x_rs);
        } else {  // shorter than the window: rows of the slot are left in it
          last[j].zero();
#pragma unroll
          for (int k = 0; k < W - 1; ++k)
            if (k == it.len + j) last[j] = first[k];
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) last[j].store(state + (slot * (W - 1) + j) * p.C);
    }
  }
}

template <class IT, class WT, int W, int V, int ROWS>
cudaError_t launch_step_as(const ConvArgs& p, const Seqs& a, cudaStream_t stream) {
  const int64_t gx = (p.C / V + kStepThreads - 1) / kStepThreads;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // a CTA keeps its weights over several sequences once the SMs are full
  int64_t gy = (16LL * ssu::sm_count() + gx - 1) / gx;
  if (gy > a.n) gy = a.n;
  if (gy > 65535) gy = 65535;
  conv_step_kernel<IT, WT, W, V, ROWS>
      <<<dim3((unsigned)gx, (unsigned)gy), kStepThreads, 0, stream>>>(p, a);
  return cudaGetLastError();
}

template <class IT, class WT, int W, int V>
cudaError_t launch_step(const ConvArgs& p, const Seqs& a, cudaStream_t stream) {
  if (!a.cu && !a.na && a.steps == 1) return launch_step_as<IT, WT, W, V, 1>(p, a, stream);
  return launch_step_as<IT, WT, W, V, 4>(p, a, stream);
}

template <class IT, class WT, int W, int V>
cudaError_t launch_prompt(const ConvArgs& p, const Seqs& a,
                          cudaStream_t stream) {
  const int64_t ctiles = (p.C / V + kPromptThreads - 1) / kPromptThreads;
  // rows per thread: fewer than 64 while the SMs are not full (16 CTAs each)
  int rows = 64;
  while (rows > kRowsInFlight<IT> && a.rows / rows * ctiles < 16LL * ssu::sm_count()) rows /= 2;
  const int64_t grid = ctiles * (((int64_t)a.rows + rows - 1) / rows);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  conv_prompt_kernel<IT, WT, W, V>
      <<<(unsigned)grid, kPromptThreads, 0, stream>>>(p, a, rows, (int)ctiles);
  return cudaGetLastError();
}

// Channels per thread: four where every row starts on a multiple of four (at
// 20634 x 5376 bf16 rows they leave 24 warps an SM and take 84 us; eight take
// 128 registers, 16 warps and 100 us; two fp32 ones 191 us where four take
// 171), two 16-bit ones on 4 bytes, else one.
template <class IT, class WT, int W>
cudaError_t launch_width(const ConvArgs& p, const Seqs& a, cudaStream_t stream) {
  constexpr int B = (int)sizeof(IT);
  auto launch = [&](auto v) {
    constexpr int V = decltype(v)::value;
    return p.prompt ? launch_prompt<IT, WT, W, V>(p, a, stream)
                    : launch_step<IT, WT, W, V>(p, a, stream);
  };
  auto rows_on = [&](int64_t bytes) {
    return aligned(p.x, bytes) && aligned(p.out, bytes) && aligned(p.state, bytes) &&
           p.x_rs * B % bytes == 0 && p.o_rs * B % bytes == 0 && p.C * B % bytes == 0;
  };
  if (rows_on(4 * B)) return launch(std::integral_constant<int, 4>{});
  if constexpr (B == 2) {
    if (rows_on(4)) return launch(std::integral_constant<int, 2>{});
  }
  return launch(std::integral_constant<int, 1>{});
}

template <class IT, class WT>
cudaError_t launch_types(int W, const ConvArgs& p, const Seqs& a,
                         cudaStream_t stream) {
  switch (W) {
    case 2: return launch_width<IT, WT, 2>(p, a, stream);
    case 3: return launch_width<IT, WT, 3>(p, a, stream);
    case 4: return launch_width<IT, WT, 4>(p, a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_conv(const ssu_conv_params* c, const ConvArgs& p, const Seqs& a, cudaStream_t stream) {
  const int W = (int)c->width;
  const bool f32w = c->weight_dtype == SSU_F32;
  switch (c->io_dtype) {
    case SSU_F32: return launch_types<float, float>(W, p, a, stream);
    case SSU_BF16:
      return f32w ? launch_types<__nv_bfloat16, float>(W, p, a, stream)
                  : launch_types<__nv_bfloat16, __nv_bfloat16>(W, p, a, stream);
    case SSU_F16:
      return f32w ? launch_types<__half, float>(W, p, a, stream)
                  : launch_types<__half, __half>(W, p, a, stream);
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
  p->w_vec = aligned(c->weight, 16) && aligned(c->bias, 16);
  p->silu = c->activation == SSU_ACT_SILU;
  p->disable = c->disable_state_update != 0;
  p->pad = c->pad_slot_id;
  return SSU_OK;
}

// out against x: a row of x is read by the threads of several rows of out in the
// prompt form; in the decode form out may be x itself, but no other view of it.
ssu_status check_conv_out(const ssu_conv_params* c, int64_t rows, bool in_place) {
  const Rows x = rows_of(c->x, c->x_row_stride, c->channels, c->io_dtype);
  const Rows out = rows_of(c->out, c->out_row_stride, c->channels, c->io_dtype);
  if (in_place && x.p == out.p && (rows == 1 || x.stride == out.stride)) return SSU_OK;
  if (overlap(out, x, rows))
    return fail(SSU_ERR_INVALID_ARGUMENT, "out must not overlap x%s",
                in_place ? " (it may be the very same rows)" : "");
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
  Seqs a;
  ssu_status st = check_conv(c, rows, true, &p);
  if (st == SSU_OK)
    st = check_packed(c->slots, nseqs, rows, cu_seqlens, dense_steps, num_accepted_tokens,
                      meta_dtype, src, dst, index_dtype, &a);
  if (st == SSU_OK) st = check_conv_out(c, rows, true);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  return launched(launch_conv(c, p, a, (cudaStream_t)stream));
}

ssu_status ssu_conv_fwd_varlen(const ssu_conv_params* c, int64_t nseqs, int64_t rows,
                               const void* cu_seqlens, ssu_dtype meta_dtype,
                               const void* state_batch_indices,
                               const void* dst_state_batch_indices, ssu_dtype index_dtype,
                               const uint8_t* has_initial_state, struct CUstream_st* stream) {
  using namespace layer;
  ConvArgs p;
  Seqs a;
  ssu_status st = check_conv(c, rows, false, &p);
  if (st == SSU_OK)
    st = check_prompts(c->conv_state != nullptr, c->slots, nseqs, rows, cu_seqlens, meta_dtype,
                       state_batch_indices, dst_state_batch_indices, index_dtype, &a);
  if (st == SSU_OK) st = check_conv_out(c, rows, false);
  if (st != SSU_OK) return st;
  if (nseqs == 0 || rows == 0) return ok();
  p.has_init = has_initial_state;
  p.prompt = 1;
  return launched(launch_conv(c, p, a, (cudaStream_t)stream));
}

}  // extern "C"
#pragma GCC visibility pop
