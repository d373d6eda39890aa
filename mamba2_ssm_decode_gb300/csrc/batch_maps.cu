// batch_maps.cu -- what the packed calls need to know about a batch, built on
// the GPU from its lengths: sequence starts, the chunks of the SSD prefill, each
// row's sequence and position; and slot tables, filled with the lowest free slots.
//
// Integers only, a few bytes a row: what the calls cost is latency.  16 sequences 6 us,
// 2048 sequences of 524288 rows 10.3 us; 20 entries 6 us, 8000 entries of a pool of 16384
// 14.3 us (one CTA: its two passes over the table).
#include "layer_common.cuh"

namespace maps {
using namespace layer;

__device__ __forceinline__ void store_int(void* p, int64_t i, int is64, int64_t v) {
  if (is64) static_cast<int64_t*>(p)[i] = v;
  else static_cast<int32_t*>(p)[i] = (int32_t)v;
}

// Inclusive sum over the CTA's threads, and the total.  `warps`: one word a warp.
template <int THREADS, class T>
__device__ __forceinline__ T block_scan(T v, T* warps, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // `warps` may still be read from the scan before
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = all;
    all += warps[w];
  }
  *total = all;
  return v + before;
}

// ---------------------------------------------------------------------------
// maps of a batch of prompts
// ---------------------------------------------------------------------------
struct Args {
  const void* lens;
  const void* context;  // nullptr: zeros
  int is64;
  int n, chunk, most;  // sequences, chunk size, room for chunks
  int rows;
  void *cu, *cu_chunk, *seq_idx, *last, *num_chunks, *row_seq, *row_pos;
  uint8_t* has_init;
};

constexpr int kThreads = 512;

struct Span {
  int64_t len;  // tokens, not below zero
  int off;      // of the first within its chunk
};

__device__ __forceinline__ int64_t context_of(const Args& a, int s) {
  const int64_t c = a.context ? load_int(a.context, s, a.is64) : 0;
  return c > 0 ? c : 0;
}

// Its place within its chunk.
__device__ __forceinline__ int offset_of(const Args& a, int64_t context) {
  // a 64-bit remainder takes a hundred instructions
  return (int)(context >> 32 ? context % a.chunk : (uint32_t)context % (uint32_t)a.chunk);
}

// Starts cu[0 .. n] (cut at `rows`) and chunk ends end[0 .. n) of every
// sequence, to shared memory; kPer sequences a thread.
template <int kPer>
__device__ __forceinline__ void plan(const Args& a, int* cu, int* end) {
  __shared__ long long warps[kThreads / 32];
  long long rows = 0, chunks = 0;
  if (threadIdx.x == 0) cu[0] = 0;
  for (int s0 = 0; s0 < a.n; s0 += kPer * kThreads) {
    const int s = s0 + kPer * threadIdx.x;
    long long len[kPer], sum = 0, total;
    int off[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      len[i] = s + i < a.n ? load_int(a.lens, s + i, a.is64) : 0;
      off[i] = s + i < a.n ? offset_of(a, context_of(a, s + i)) : 0;
      len[i] = len[i] > 0 ? (len[i] < a.rows ? len[i] : a.rows) : 0;  // more is cut all the same
      sum += len[i];
    }
    long long from = rows + block_scan<kThreads>(sum, warps, &total) - sum;
    rows += total;
    // a sequence's chunks end at multiples of the chunk size of its own positions; it has one
    // at least, which carries its state through
    int many[kPer], all = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = (int)(from < a.rows ? from : a.rows);
      from += len[i];
      const int e = (int)(from < a.rows ? from : a.rows);
      many[i] = e == b ? 1 : (int)(((uint32_t)off[i] + (uint32_t)(e - b) + (uint32_t)a.chunk - 1u) /
                                   (uint32_t)a.chunk);
      if (s + i >= a.n) continue;
      cu[s + i + 1] = e;
      all += many[i];
    }
    long long c = chunks + block_scan<kThreads>((long long)all, warps, &total) - all;
    chunks += total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (s + i >= a.n) continue;
      c += many[i];
      end[s + i] = (int)c;
    }
  }
  __syncthreads();
}

// The first of n ascending values that is above v (n: none).
__device__ __forceinline__ int first_above(const int* values, int n, int v) {
  int lo = 0;
  for (int left = n; left > 0;) {  // as many steps whatever v is
    const int half = left >> 1;
    if (values[lo + half] <= v) lo += left - half, left = half;
    else left = half;
  }
  return lo;
}

// cu, end: as plan() leaves them
__device__ __forceinline__ void write_chunk(const Args& a, const int* cu, const int* end, int c) {
  const int chunks = a.n ? end[a.n - 1] : 0;
  const int s = min(first_above(end, a.n, c), a.n - 1);
  int64_t at = a.n ? cu[a.n] : 0;
  if (c < chunks) {
    const int nth = c - (s > 0 ? end[s - 1] : 0);
    at = cu[s];
    if (nth > 0) at += (int64_t)nth * a.chunk - offset_of(a, context_of(a, s));
  }
  store_int(a.cu_chunk, c, a.is64, at);
  if (c < a.most) store_int(a.seq_idx, c, a.is64, s > 0 ? s : 0);
}

// Rows r, r + step, ...: kRows of them, whose searches and loads overlap.
template <int kRows>
__device__ __forceinline__ void write_rows(const Args& a, const int* cu, int64_t r, int64_t step) {
  int s[kRows];
  int64_t pos[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    s[i] = r + i * step < a.rows ? first_above(cu + 1, a.n, (int)(r + i * step)) : a.n;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    pos[i] = s[i] < a.n ? context_of(a, s[i]) + r + i * step - cu[s[i]] : -1;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (r + i * step >= a.rows) continue;
    if (a.row_seq) store_int(a.row_seq, r + i * step, a.is64, s[i] < a.n ? s[i] : -1);
    if (a.row_pos) store_int(a.row_pos, r + i * step, a.is64, pos[i]);
  }
}

__device__ __forceinline__ void write_sequence(const Args& a, const int* cu, const int* end, int s) {
  if (s == 0) store_int(a.cu, 0, a.is64, 0);
  if (s == 0) store_int(a.num_chunks, 0, a.is64, a.n ? end[a.n - 1] : 0);
  if (s >= a.n) return;
  store_int(a.cu, s + 1, a.is64, cu[s + 1]);
  store_int(a.last, s, a.is64, end[s] - 1);
  a.has_init[s] = context_of(a, s) > 0;
}

// Every CTA plans for itself and writes its share.  MANY: more than a sequence (S) or
// a row (R) a thread; one at a time is 2 us faster where there are few.
template <bool MANY_S, bool MANY_R>
__global__ void __launch_bounds__(kThreads) prompt_maps_kernel(const Args a) {
  constexpr int kRows = MANY_R ? 4 : 1;
  extern __shared__ int plan_smem[];
  int* cu = plan_smem;
  int* end = plan_smem + a.n + 1;
  plan<MANY_S ? 4 : 1>(a, cu, end);
  const int t = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  for (int s = t; s <= a.n; s += step) write_sequence(a, cu, end, s);
  for (int c = t; c <= a.most; c += step) write_chunk(a, cu, end, c);
  if (a.row_seq || a.row_pos)
    for (int64_t r = t; r < a.rows; r += (int64_t)kRows * step) write_rows<kRows>(a, cu, r, step);
}

// ---------------------------------------------------------------------------
// slot tables
// ---------------------------------------------------------------------------
struct AssignArgs {
  const void* table;
  const void* counts;
  void* out;
  void* fresh;
  int* missing;
  int is64;
  int n, steps, slots;
  int64_t pad;
};

constexpr int kAssignThreads = 1024;
// Bit k (from 0) of those set in v.
__device__ __forceinline__ int nth_bit(unsigned long long v, int k) {
  int at = 0;
#pragma unroll
  for (int w = 32; w > 0; w >>= 1) {
    const int low = __popcll(v & ((1ull << w) - 1));
    if (k >= low) {
      k -= low;
      at += w;
      v >>= w;
    }
  }
  return at;
}

// One CTA: a bitmap of the slots that are kept, the free ones before each of its
// words, and then, in the table's order, the k-th place without a slot takes the
// k-th free one.  kEntries of the table a thread at a time.  LIST: the free slots are
// listed in shared memory, where there is room for kListed of them; else each place
// searches the words (8000 entries of a pool of 16384: 14.3 and 18 us).
constexpr int kListed = 1 << 15;
constexpr int kMostSlots = 1 << 20;

template <int kEntries, bool LIST>
__global__ void __launch_bounds__(kAssignThreads) slots_assign_kernel(const AssignArgs a) {
  extern __shared__ unsigned long long held[];
  __shared__ int warps[kAssignThreads / 32];
  const int words = (a.slots + 63) / 64;
  int* before = reinterpret_cast<int*>(held + words);
  for (int w = threadIdx.x; w < words; w += kAssignThreads) {
    const int rest = a.slots - w * 64;  // beyond the last slot: held
    held[w] = rest < 64 ? ~0ull << rest : 0;
  }
  __syncthreads();
  if (threadIdx.x == 0 && a.pad >= 0 && a.pad < a.slots)
    atomicOr(&held[a.pad >> 6], 1ull << (a.pad & 63));  // never handed out
  const int entries = a.n * a.steps;  // at most 2^24
  // the table's entry e; `wanted`: its row is to hold it
  auto entry = [&](int e, bool* wanted) {
    const uint32_t s = (uint32_t)e / (uint32_t)a.steps;
    *wanted = (int64_t)(e - (int)s * a.steps) < load_int(a.counts, s, a.is64);
    return load_int(a.table, e, a.is64);
  };
  for (int e0 = threadIdx.x; e0 < entries; e0 += kEntries * kAssignThreads) {
    int64_t v[kEntries];
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
      const int e = e0 + i * kAssignThreads;
      bool wanted = false;
      v[i] = e < entries ? entry(e, &wanted) : 0;
      if (!wanted) v[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
      if (slot_ok(v[i], a.pad, a.slots)) atomicOr(&held[v[i] >> 6], 1ull << (v[i] & 63));
  }
  __syncthreads();
  int free = 0;
  for (int w0 = 0; w0 < words; w0 += kAssignThreads) {
    const int w = w0 + threadIdx.x;
    const int mine = w < words ? 64 - __popcll(held[w]) : 0;
    int total;
    const int inc = free + block_scan<kAssignThreads>(mine, warps, &total);
    if (w < words) before[w] = inc - mine;
    free += total;
  }
  __syncthreads();
  int* list = before + words;
  if constexpr (LIST) {
    for (int i = threadIdx.x; i < 4 * words; i += kAssignThreads) {  // 16 slots a thread
      const int w = i >> 2, part = (i & 3) * 16;
      const unsigned long long open = ~held[w];
      int k = before[w] + __popcll(open & ((1ull << part) - 1));
      for (unsigned m = (unsigned)(open >> part) & 0xffffu; m; m &= m - 1)
        list[k++] = w * 64 + part + __ffs((int)m) - 1;
    }
    __syncthreads();
  }
  // a warp has kEntries times 32 consecutive entries, 32 at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int given = 0;
  for (int e0 = 0; e0 < entries; e0 += kEntries * kAssignThreads) {
    const int first = e0 + warp * kEntries * 32 + lane;
    int64_t v[kEntries];
    unsigned need[kEntries], kept = 0;
    int mine = 0;  // of the warp
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
      const int e = first + i * 32;
      bool wanted = false;
      v[i] = e < entries ? entry(e, &wanted) : 0;
      const bool keeps = wanted && slot_ok(v[i], a.pad, a.slots);
      kept |= (unsigned)keeps << i;
      need[i] = __ballot_sync(0xffffffffu, wanted && !keeps);
      mine += __popc(need[i]);
    }
    __syncthreads();  // `warps` may still be read
    if (lane == 0) warps[warp] = mine;
    __syncthreads();
    static_assert(kAssignThreads / 32 == 32, "a lane a warp");
    const int theirs = warps[lane];
    const int total = __reduce_add_sync(0xffffffffu, theirs);
    int rank = given + __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0);
    given += total;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
      const int e = first + i * 32;
      const int k = rank + __popc(need[i] & ((1u << lane) - 1));
      rank += __popc(need[i]);
      if (e >= entries) continue;
      int64_t got = a.pad;
      if ((need[i] >> lane & 1) && k < free) {
        if constexpr (LIST) {
          got = list[k];
        } else {
          int lo = 0, hi = words;  // the last word with no more than k free ones before it
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= k) lo = mid;
            else hi = mid;
          }
          got = lo * 64 + nth_bit(~held[lo], k - before[lo]);
        }
      }
      store_int(a.out, e, a.is64, kept >> i & 1 ? v[i] : got);
      store_int(a.fresh, e, a.is64, got);
    }
  }
  if (threadIdx.x == 0) *a.missing = given > free ? given - free : 0;
}

static ssu_status prompt_maps(const ssu_prompt_maps_params* c, cudaStream_t stream) {
  if (!c) return fail(SSU_ERR_INVALID_ARGUMENT, "params must not be NULL");
  if (!is_index(c->index_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "lengths and maps must be int32 or int64");
  if (c->nseqs < 0 || c->rows < 0 || c->chunk_size < 1 || c->max_chunks < 0)
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "nseqs, rows and max_chunks must be >= 0, chunk_size positive");
  if (c->nseqs > SSU_PROMPT_MAPS_MAX_SEQS || c->rows > 0x7fffffffLL - 1024 ||
      c->chunk_size > (1 << 20) || c->max_chunks >= 1 << 30)
    return fail(SSU_ERR_UNSUPPORTED,
                "at most %d sequences, 2^31 - 1025 rows, chunks of 2^20 and 2^30 - 1 of them",
                SSU_PROMPT_MAPS_MAX_SEQS);
  // what the lengths can come to, so that no chunk is lost
  const int64_t need = c->rows / c->chunk_size + (c->context_lens ? 2 : 1) * c->nseqs;
  if (c->max_chunks < need)
    return fail(SSU_ERR_INVALID_ARGUMENT, "%lld rows of %lld sequences may need %lld chunks, got "
                "room for %lld", (long long)c->rows, (long long)c->nseqs, (long long)need,
                (long long)c->max_chunks);
  if ((c->nseqs > 0 && (!c->lens || !c->last_chunk_indices || !c->has_initial_state)) ||
      !c->cu_seqlens || !c->cu_chunk_seqlens || !c->num_chunks ||
      (c->max_chunks > 0 && !c->seq_idx))
    return fail(SSU_ERR_INVALID_ARGUMENT, "lens and the maps must not be NULL");
  const int es = size_of(c->index_dtype);
  const void* all[] = {c->lens, c->context_lens, c->cu_seqlens, c->cu_chunk_seqlens, c->seq_idx,
                       c->last_chunk_indices, c->num_chunks, c->row_seq, c->row_pos};
  for (const void* p : all)
    if (!aligned(p, es))
      return fail(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their element size");
  const struct {
    const void* p;
    int64_t bytes;
  } out[] = {{c->cu_seqlens, (c->nseqs + 1) * es},
             {c->cu_chunk_seqlens, (c->max_chunks + 1) * es},
             {c->seq_idx, c->max_chunks * es},
             {c->last_chunk_indices, c->nseqs * es},
             {c->has_initial_state, c->nseqs},
             {c->num_chunks, es},
             {c->row_seq, c->rows * es},
             {c->row_pos, c->rows * es},
             {c->lens, c->nseqs * es},
             {c->context_lens, c->nseqs * es}};
  for (int i = 0; i < 8; ++i)
    for (int j = i + 1; j < 10; ++j)
      if (out[i].bytes > 0 && out[j].bytes > 0 &&
          overlap(Rows{out[i].p, 0, out[i].bytes}, Rows{out[j].p, 0, out[j].bytes}, 1))
        return fail(SSU_ERR_INVALID_ARGUMENT, "the maps must not overlap each other or the lengths");
  Args a{};
  a.lens = c->lens;
  a.context = c->context_lens;
  a.is64 = c->index_dtype == SSU_I64;
  a.n = (int)c->nseqs;
  a.chunk = (int)c->chunk_size;
  a.most = (int)c->max_chunks;
  a.rows = (int)c->rows;
  a.cu = c->cu_seqlens;
  a.cu_chunk = c->cu_chunk_seqlens;
  a.seq_idx = c->seq_idx;
  a.last = c->last_chunk_indices;
  a.num_chunks = c->num_chunks;
  a.has_init = c->has_initial_state;
  a.row_seq = c->row_seq;
  a.row_pos = c->row_pos;
  auto smem_of = [](int n) { return (2 * n + 1) * (int)sizeof(int); };
  const int smem = smem_of(a.n);
  const int64_t rows = a.row_seq || a.row_pos ? a.rows : 0;
  const int64_t items = rows > a.most ? rows : a.most;
  const int64_t fit = ssu::sm_count();
  int64_t ctas = items / kThreads + 1;
  const bool many_s = a.n > kThreads, many_r = ctas > fit;
  if (many_r) ctas = fit;
  auto kernel = many_s ? (many_r ? prompt_maps_kernel<true, true> : prompt_maps_kernel<true, false>)
                       : (many_r ? prompt_maps_kernel<false, true> : prompt_maps_kernel<false, false>);
  if (smem > 48 * 1024) {
    // the most of any call: the limit is the kernel's, and another thread's call sets it too
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               smem_of(SSU_PROMPT_MAPS_MAX_SEQS));
    if (e != cudaSuccess) return launched(e);
  }
  kernel<<<(unsigned)ctas, kThreads, smem, stream>>>(a);
  return launched(cudaGetLastError());
}

static ssu_status assign(const void* table, const void* counts, ssu_dtype index_dtype,
                         int64_t nseqs, int64_t steps, int64_t slots, int64_t pad, void* out,
                         void* fresh, int32_t* missing, cudaStream_t stream) {
  if (!is_index(index_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "the slot table and counts must be int32 or int64");
  if (nseqs < 0 || steps < 0 || slots < 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "nseqs, steps and slots must be >= 0");
  // it is written into the tables
  if (index_dtype == SSU_I32 && pad != (int32_t)pad)
    return fail(SSU_ERR_INVALID_ARGUMENT, "pad_slot_id %lld is no int32, which the table holds",
                (long long)pad);
  if (slots > kMostSlots) return fail(SSU_ERR_UNSUPPORTED, "slots must not exceed 2^20");
  if (nseqs > 0x7fffffffLL || steps > 0x7fffffffLL || (steps > 0 && nseqs > (1 << 24) / steps))
    return fail(SSU_ERR_UNSUPPORTED, "the table must not exceed 2^24 entries");
  const int64_t entries = nseqs * steps;
  if (!missing || (entries > 0 && (!table || !counts || !out || !fresh)))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "table, counts, out, fresh and num_missing must not be NULL");
  const int es = size_of(index_dtype);
  if (!aligned(table, es) || !aligned(counts, es) || !aligned(out, es) || !aligned(fresh, es) ||
      !aligned(missing, 4))
    return fail(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their element size");
  auto span = [&](const void* p, int64_t n) { return Rows{p, 0, n * es}; };
  const Rows t = span(table, entries), o = span(out, entries), f = span(fresh, entries),
             n = span(counts, nseqs), m = Rows{missing, 0, 4};
  if (entries > 0 && ((table != out && overlap(t, o, 1)) || overlap(o, f, 1) || overlap(t, f, 1) ||
                      overlap(n, o, 1) || overlap(n, f, 1) || overlap(m, o, 1) ||
                      overlap(m, f, 1) || overlap(m, t, 1) || overlap(m, n, 1)))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "out may be table itself; else table, counts, out, fresh and num_missing must not "
                "overlap");
  AssignArgs a{table, counts, out, fresh, missing, index_dtype == SSU_I64, (int)nseqs, (int)steps,
               (int)slots, pad};
  const bool list = a.slots <= kListed;
  auto smem_of = [list](int n) { return (n + 63) / 64 * 12 + (list ? n * 4 : 0); };
  const int smem = smem_of(a.slots);
  const bool few = entries <= kAssignThreads;
  auto kernel = list ? (few ? slots_assign_kernel<1, true> : slots_assign_kernel<8, true>)
                     : (few ? slots_assign_kernel<1, false> : slots_assign_kernel<8, false>);
  if (smem > 40 * 1024) {  // the most of any call, as above
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               smem_of(list ? kListed : kMostSlots));
    if (e != cudaSuccess) return launched(e);
  }
  kernel<<<1, kAssignThreads, smem, stream>>>(a);
  return launched(cudaGetLastError());
}

}  // namespace maps

#pragma GCC visibility push(default)
extern "C" {

ssu_status ssu_prompt_maps(const ssu_prompt_maps_params* c, struct CUstream_st* stream) {
  return maps::prompt_maps(c, (cudaStream_t)stream);
}

ssu_status ssu_slots_assign(const void* table, const void* counts, ssu_dtype index_dtype,
                            int64_t nseqs, int64_t steps, int64_t slots, int64_t pad_slot_id,
                            void* table_out, void* fresh, int32_t* num_missing,
                            struct CUstream_st* stream) {
  return maps::assign(table, counts, index_dtype, nseqs, steps, slots, pad_slot_id, table_out,
                      fresh, num_missing, (cudaStream_t)stream);
}

}  // extern "C"
#pragma GCC visibility pop
