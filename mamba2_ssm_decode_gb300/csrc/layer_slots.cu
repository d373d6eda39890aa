// layer_slots.cu -- moves of whole slots inside the pools that the other calls
// index: copies (a sequence forked, a beam step), clears, and the compaction
// that closes a pool up, over any number of pools (every layer's state,
// convolution rows, ring caches and trackers) in one call.
//
// Pure data movement: a slot is read once and written once.
#include "layer_common.cuh"

namespace layer {

constexpr int kMaxPools = SSU_SLOTS_MAX_POOLS;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kChunk = kCopyThreads * kCopyUnroll * 16;  // bytes of a slot per work item

struct Pool {
  uint8_t* data;
  int64_t bytes, stride;
};

// Pools by value in the launch's parameters: nothing has to be copied to the
// device before the kernel, and nothing kept alive after the call.  Calls of a
// few pools have a smaller list to hand over.
constexpr int kFewPools = 16;

template <int MOST>
struct Pools {
  Pool pool[MOST];
  int first[MOST + 1];  // first chunk of each pool within a slot; the total at the end
  uint32_t wide[(MOST + 31) / 32];  // bit set: 16-byte accesses
  int n;
  int64_t slots;
};

enum class Fill { kCopy, kZero };

template <class T, Fill F>
__device__ __forceinline__ void move_bytes(uint8_t* dst, const uint8_t* src, int bytes) {
  const int n = bytes / (int)sizeof(T);
  T* d = reinterpret_cast<T*>(dst);
  const T* s = reinterpret_cast<const T*>(src);
  for (int i0 = threadIdx.x; i0 < n; i0 += kCopyThreads * kCopyUnroll) {
    T v[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
      const int i = i0 + k * kCopyThreads;
      v[k] = T{};
      if (F == Fill::kCopy && i < n) v[k] = s[i];
    }
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
      const int i = i0 + k * kCopyThreads;
      if (i < n) d[i] = v[k];
    }
  }
}

// Chunk `chunk` of a slot: which pool's bytes, from where.
template <Fill F, int MOST>
__device__ __forceinline__ void move_chunk(const Pools<MOST>& ps, int chunk, int64_t from, int64_t to) {
  int lo = 0, hi = ps.n - 1;  // the pool with first[lo] <= chunk < first[lo + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ps.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  const Pool& p = ps.pool[lo];
  const int64_t at = (int64_t)(chunk - ps.first[lo]) * kChunk;
  const int64_t left = p.bytes - at;
  const int bytes = left < kChunk ? (int)left : kChunk;
  uint8_t* d = p.data + to * p.stride + at;
  const uint8_t* s = p.data + from * p.stride + at;
  if (ps.wide[lo >> 5] >> (lo & 31) & 1) move_bytes<uint4, F>(d, s, bytes);
  else if (((uintptr_t)p.data | (uintptr_t)p.bytes | (uintptr_t)p.stride) % 4 == 0)
    move_bytes<uint32_t, F>(d, s, bytes);
  else move_bytes<uint8_t, F>(d, s, bytes);
}

// Bound by HBM: 24 copies of 8 slots over four layers' pools, 340 MB, take 51
// us, 6.7 TB/s, what a plain copy reaches.
// grid: x = pairs (several CTAs that copy the same piece of one source run side
// by side, so a fork reads it from HBM once), y = chunks of a slot.
template <Fill F, int MOST>
__global__ void __launch_bounds__(kCopyThreads)
    slots_copy_kernel(const __grid_constant__ Pools<MOST> ps, const void* src, const void* dst,
                      int idx64, int64_t pad) {
  const int64_t to = load_int(dst, blockIdx.x, idx64);
  const int64_t from = F == Fill::kCopy ? load_int(src, blockIdx.x, idx64) : to;
  if (!slot_ok(to, pad, ps.slots) || !slot_ok(from, pad, ps.slots)) return;
  if (F == Fill::kCopy && from == to) return;
  for (int chunk = blockIdx.y; chunk < ps.first[ps.n]; chunk += gridDim.y)
    move_chunk<F, MOST>(ps, chunk, from, to);
}

// Which slots are live, and where each that lies beyond the first `live` goes:
// the k-th of them to the k-th free slot below.  A bitmap of the slots in
// shared memory, a running count per 64 slots, then ranks.
struct Plan {
  unsigned long long* bits;  // [words]
  int* before;               // [words] live slots in front of word w
  int words, slots, live, kept;  // kept: live slots that stay where they are

  // live slots in front of slot id < slots
  __device__ __forceinline__ int rank(int id) const {
    return before[id >> 6] + __popcll(bits[id >> 6] & ((1ull << (id & 63)) - 1));
  }
  __device__ __forceinline__ bool is_live(int id) const { return bits[id >> 6] >> (id & 63) & 1; }
};

static __host__ __device__ inline int plan_words(int64_t slots) { return (int)((slots + 63) / 64); }

// All threads of the CTA; `smem` holds 12 bytes a word.
template <int THREADS>
__device__ __forceinline__ Plan make_plan(void* smem, const void* table, int idx64, int64_t n,
                                          int64_t pad, int slots) {
  __shared__ int warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Plan p;
  p.words = plan_words(slots);
  p.slots = slots;
  p.bits = static_cast<unsigned long long*>(smem);
  p.before = reinterpret_cast<int*>(p.bits + p.words);
  for (int w = tid; w < p.words; w += THREADS) p.bits[w] = 0;
  __syncthreads();
  for (int64_t i = tid; i < n; i += THREADS) {
    const int64_t v = load_int(table, i, idx64);
    if (slot_ok(v, pad, slots)) atomicOr(&p.bits[v >> 6], 1ull << (v & 63));
  }
  __syncthreads();
  // exclusive prefix of the words' counts: a run of words for each thread
  const int run = (p.words + THREADS - 1) / THREADS;
  const int w0 = tid * run < p.words ? tid * run : p.words;
  const int w1 = w0 + run < p.words ? w0 + run : p.words;
  int sum = 0;
  for (int w = w0; w < w1; ++w) sum += __popcll(p.bits[w]);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int front = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int v = warp_sum[w];
    front += w < warp ? v : 0;
    total += v;
  }
  int at = inc - sum + front;
  for (int w = w0; w < w1; ++w) {
    p.before[w] = at;
    at += __popcll(p.bits[w]);
  }
  __syncthreads();
  p.live = total;
  p.kept = total < slots ? p.rank(total) : total;
  return p;
}

// The two slots of every move, in order.
template <int THREADS, class T>
__device__ __forceinline__ void list_moves(const Plan& p, T* src, T* dst) {
  for (int id = threadIdx.x; id < p.slots; id += THREADS) {
    const bool live = p.is_live(id);
    if (id < p.live && !live) dst[id - p.rank(id)] = (T)id;
    if (id >= p.live && live) src[p.rank(id) - p.kept] = (T)id;
  }
  __syncthreads();  // they are read by other threads than wrote them
}

// The table under the new ids, and the number of live slots.
template <int THREADS, class T>
__device__ __forceinline__ void write_table(const Plan& p, const T* dst, const void* table,
                                            void* table_out, int idx64, int64_t n, int64_t pad,
                                            int* num_live) {
  for (int64_t i = threadIdx.x; i < n; i += THREADS) {
    const int64_t v = load_int(table, i, idx64);
    int64_t to = v;
    if (slot_ok(v, pad, p.slots) && v >= p.live) to = (int64_t)dst[p.rank((int)v) - p.kept];
    if (idx64) static_cast<int64_t*>(table_out)[i] = to;
    else static_cast<int32_t*>(table_out)[i] = (int32_t)to;
  }
  if (threadIdx.x == 0) *num_live = p.live;
}

// Large pools: one CTA plans, a second launch moves.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
    slots_plan_kernel(const void* table, void* table_out, int idx64, int64_t n, int64_t pad,
                      int slots, int* num_live, int* moves, int* src, int* dst) {
  extern __shared__ __align__(16) unsigned char plan_smem_raw[];
  const Plan p = make_plan<kPlanThreads>(plan_smem_raw, table, idx64, n, pad, slots);
  list_moves<kPlanThreads>(p, src, dst);
  if (threadIdx.x == 0) *moves = p.live - p.kept;
  write_table<kPlanThreads>(p, dst, table, table_out, idx64, n, pad, num_live);
}

// As many CTAs as fit walk the moves, the pieces of one slot side by side.
template <int MOST>
__global__ void __launch_bounds__(kCopyThreads)
    slots_move_kernel(const __grid_constant__ Pools<MOST> ps, const int* moves, const int* src,
                      const int* dst) {
  const int64_t chunks = ps.first[ps.n], half = ps.slots / 2;
  const int64_t listed = *moves;  // at most half the slots, as the plan leaves them ...
  const int64_t items = (listed < half ? listed : half) * chunks;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int64_t m = i / chunks;
    const unsigned from = src[m], to = dst[m];
    // ... and ids below `slots`: a workspace that something else wrote moves nothing elsewhere
    if (from < ps.slots && to < ps.slots)
      move_chunk<Fill::kCopy, MOST>(ps, (int)(i - m * chunks), from, to);
  }
}

// Small ones, in one launch: every CTA makes the plan for itself (a few
// thousand table entries out of L2, less than a launch takes) and moves its
// share; the last one writes the table, which must not be the one that the
// others are still reading.  With half the slots live and 8 KB a slot: 256 slots
// 6.4 us where two launches take 11.9, 1024 slots 8.4 and 10.5, but 4096 slots
// 24.7 and 16.5 (57.7 and 54.5 with 128 KB a slot): the plan is worth repeating up
// to about 2000 slots.
constexpr int kSmallSlots = 4096, kSmallEntries = 8192;

template <int MOST>
__global__ void __launch_bounds__(kCopyThreads)
    slots_compact_kernel(const __grid_constant__ Pools<MOST> ps, const void* table,
                         void* table_out, int idx64, int n, int64_t pad, int slots,
                         int* num_live) {
  __shared__ unsigned long long plan[kSmallSlots / 64 * 12 / 8];
  __shared__ unsigned short src[kSmallSlots / 2], dst[kSmallSlots / 2];
  const Plan p = make_plan<kCopyThreads>(plan, table, idx64, n, pad, slots);
  list_moves<kCopyThreads>(p, src, dst);
  if (blockIdx.x == gridDim.x - 1)
    write_table<kCopyThreads>(p, dst, table, table_out, idx64, n, pad, num_live);
  const int64_t chunks = ps.first[ps.n];
  const int64_t items = (p.live - p.kept) * chunks;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int64_t m = i / chunks;
    move_chunk<Fill::kCopy, MOST>(ps, (int)(i - m * chunks), src[m], dst[m]);
  }
}

template <int MOST>
static ssu_status check_pools(const ssu_pool* pools, int npools, int64_t slots, Pools<MOST>* ps) {
  if (npools < 0 || slots < 0)
    return fail(SSU_ERR_INVALID_ARGUMENT, "npools and slots must be >= 0");
  if (npools > kMaxPools)
    return fail(SSU_ERR_UNSUPPORTED, "at most %d pools per call, got %d", kMaxPools, npools);
  if (slots > (1 << 20)) return fail(SSU_ERR_UNSUPPORTED, "slots must not exceed 2^20");
  if (npools > 0 && !pools) return fail(SSU_ERR_INVALID_ARGUMENT, "pools must not be NULL");
  *ps = Pools<MOST>{};
  int64_t chunks = 0;
  int n = 0;
  for (int i = 0; i < npools; ++i) {
    const ssu_pool& p = pools[i];
    if (p.slot_bytes < 0 || (slots > 1 && p.slot_stride_bytes < p.slot_bytes))
      return fail(SSU_ERR_INVALID_ARGUMENT,
                  "pool %d: a slot of %lld bytes does not fit a stride of %lld", i,
                  (long long)p.slot_bytes, (long long)p.slot_stride_bytes);
    if (p.slot_bytes == 0 || slots == 0) continue;
    if (!p.data) return fail(SSU_ERR_INVALID_ARGUMENT, "pool %d must not be NULL", i);
    ps->pool[n] = Pool{static_cast<uint8_t*>(p.data), p.slot_bytes, p.slot_stride_bytes};
    if (aligned(p.data, 16) && p.slot_bytes % 16 == 0 && p.slot_stride_bytes % 16 == 0)
      ps->wide[n >> 5] |= 1u << (n & 31);
    ps->first[n] = (int)chunks;
    chunks += (p.slot_bytes + kChunk - 1) / kChunk;
    if (chunks > 0x3fffffffLL)
      return fail(SSU_ERR_UNSUPPORTED, "a slot of all pools must stay below 2^45 bytes");
    ++n;
  }
  ps->first[n] = (int)chunks;
  ps->n = n;
  ps->slots = slots;
  return SSU_OK;
}

template <Fill F, int MOST>
static ssu_status move_slots_as(const ssu_pool* pools, int npools, int64_t slots, const void* src,
                             const void* dst, ssu_dtype index_dtype, int64_t pairs, int64_t pad,
                             cudaStream_t stream) {
  Pools<MOST> ps;
  ssu_status st = check_pools(pools, npools, slots, &ps);
  if (st != SSU_OK) return st;
  if (!is_index(index_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "slot ids must be int32 or int64");
  if (pairs < 0) return fail(SSU_ERR_INVALID_ARGUMENT, "the number of slot ids must be >= 0");
  if (pairs > 0x7fffffffLL) return fail(SSU_ERR_UNSUPPORTED, "at most 2^31 - 1 slot ids per call");
  if (pairs > 0 && (!dst || (F == Fill::kCopy && !src)))
    return fail(SSU_ERR_INVALID_ARGUMENT, "slot ids must not be NULL");
  if (pairs == 0 || ps.n == 0) return ok();
  const int chunks = ps.first[ps.n];
  const dim3 grid((unsigned)pairs, (unsigned)(chunks < 65535 ? chunks : 65535));
  slots_copy_kernel<F, MOST><<<grid, kCopyThreads, 0, stream>>>(ps, src, dst, index_dtype == SSU_I64,
                                                         pad);
  return launched(cudaGetLastError());
}

template <Fill F>
static ssu_status move_slots(const ssu_pool* pools, int npools, int64_t slots, const void* src,
                             const void* dst, ssu_dtype index_dtype, int64_t pairs, int64_t pad,
                             cudaStream_t stream) {
  return npools <= kFewPools ? move_slots_as<F, kFewPools>(pools, npools, slots, src, dst,
                                                           index_dtype, pairs, pad, stream)
                             : move_slots_as<F, kMaxPools>(pools, npools, slots, src, dst,
                                                           index_dtype, pairs, pad, stream);
}

static int plan_smem(int64_t slots) { return plan_words(slots) * 12; }

static bool in_one_launch(int64_t slots, int64_t entries, bool in_place) {
  return slots <= kSmallSlots && entries <= kSmallEntries && !in_place;
}

static int64_t workspace_bytes_of(int64_t slots, int64_t entries, bool in_place) {
  if (slots < 0 || entries < 0) return -1;
  if (in_one_launch(slots, entries, in_place)) return 0;
  // the number of moves, and the two slots of each (at most half the pool moves)
  return 16 + 2 * 4 * ((slots + 1) / 2);
}

template <int MOST>
static ssu_status compact_as(const ssu_pool* pools, int npools, int64_t slots, const void* table,
                             void* table_out, ssu_dtype index_dtype, int64_t entries,
                             int64_t pad_slot_id, int32_t* num_live, void* workspace,
                             int64_t workspace_bytes, cudaStream_t stream) {
  Pools<MOST> ps;
  ssu_status st = check_pools(pools, npools, slots, &ps);
  if (st != SSU_OK) return st;
  if (!is_index(index_dtype))
    return fail(SSU_ERR_INVALID_ARGUMENT, "the slot table must be int32 or int64");
  if (entries < 0) return fail(SSU_ERR_INVALID_ARGUMENT, "entries must be >= 0");
  if ((entries > 0 && (!table || !table_out)) || !num_live)
    return fail(SSU_ERR_INVALID_ARGUMENT, "table, table_out and num_live must not be NULL");
  if (table != table_out && overlap(rows_of(table, 0, entries, index_dtype),
                                    rows_of(table_out, 0, entries, index_dtype), 1))
    return fail(SSU_ERR_INVALID_ARGUMENT, "table_out must be table or not overlap it");
  const int64_t need = workspace_bytes_of(slots, entries, table == table_out);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return fail(SSU_ERR_INVALID_ARGUMENT,
                "ssu_slots_compact needs a 16-byte aligned workspace of %lld bytes, got %lld",
                (long long)need, (long long)workspace_bytes);
  // at most half the slots move, and no more than the table has entries
  const int64_t most = slots / 2 < entries ? slots / 2 : entries;
  const int64_t items = most * ps.first[ps.n];
  const int64_t fit = 8LL * ssu::sm_count();
  const int64_t ctas = items < 1 ? 1 : items < fit ? items : fit;
  // 244 of 1024 slots moved, 201 MB: 44.7 us in two launches, 41.6 us in one; 12
  // of 48, 10 MB: 16 us and 11 us
  if (need == 0) {
    slots_compact_kernel<MOST><<<(unsigned)ctas, kCopyThreads, 0, stream>>>(
        ps, table, table_out, index_dtype == SSU_I64, (int)entries, pad_slot_id, (int)slots,
        num_live);
    return launched(cudaGetLastError());
  }
  int* moves = static_cast<int*>(workspace);
  int* src = moves + 4;
  int* dst = src + (slots + 1) / 2;
  const int smem = plan_smem(slots);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(slots_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return launched(e);
  }
  slots_plan_kernel<<<1, kPlanThreads, smem, stream>>>(
      table, table_out, index_dtype == SSU_I64, entries, pad_slot_id, (int)slots, num_live, moves,
      src, dst);
  e = cudaGetLastError();
  if (e != cudaSuccess || items == 0) return launched(e);
  slots_move_kernel<MOST><<<(unsigned)ctas, kCopyThreads, 0, stream>>>(ps, moves, src, dst);
  return launched(cudaGetLastError());
}

}  // namespace layer

#pragma GCC visibility push(default)
extern "C" {

ssu_status ssu_slots_copy(const ssu_pool* pools, int npools, int64_t slots, const void* src,
                          const void* dst, ssu_dtype index_dtype, int64_t pairs,
                          int64_t pad_slot_id, struct CUstream_st* stream) {
  return layer::move_slots<layer::Fill::kCopy>(pools, npools, slots, src, dst, index_dtype, pairs,
                                               pad_slot_id, (cudaStream_t)stream);
}

ssu_status ssu_slots_clear(const ssu_pool* pools, int npools, int64_t slots, const void* ids,
                           ssu_dtype index_dtype, int64_t count, int64_t pad_slot_id,
                           struct CUstream_st* stream) {
  return layer::move_slots<layer::Fill::kZero>(pools, npools, slots, nullptr, ids, index_dtype,
                                               count, pad_slot_id, (cudaStream_t)stream);
}

int64_t ssu_slots_compact_workspace_bytes(int64_t slots, int64_t entries, int in_place) {
  return layer::workspace_bytes_of(slots, entries, in_place != 0);
}

ssu_status ssu_slots_compact(const ssu_pool* pools, int npools, int64_t slots, const void* table,
                             void* table_out, ssu_dtype index_dtype, int64_t entries,
                             int64_t pad_slot_id, int32_t* num_live, void* workspace,
                             int64_t workspace_bytes, struct CUstream_st* stream) {
  using namespace layer;
  auto f = npools <= kFewPools ? compact_as<kFewPools> : compact_as<kMaxPools>;
  return f(pools, npools, slots, table, table_out, index_dtype, entries, pad_slot_id, num_live,
           workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"
#pragma GCC visibility pop
