// linattn_prompt.cu -- linear attention over prompts: the workspace, the plan and
// the launches.
#include "linattn_prompt.cuh"

namespace ssu {
unsigned* device_error_word();  // ssu_abi.cu
}

namespace linattn {

cudaError_t launch_pieces_bf16(const PromptArgs& g, int ctas, cudaStream_t stream);
cudaError_t launch_pieces_f16(const PromptArgs& g, int ctas, cudaStream_t stream);
cudaError_t launch_chunks_bf16(const PromptArgs& g, int ctas, cudaStream_t stream);
cudaError_t launch_chunks_f16(const PromptArgs& g, int ctas, cudaStream_t stream);

// How a call is cut, and where its workspace holds what.
struct Layout {
  int fair, cut;
  int64_t entries, pieces, split;  // most states, pieces, sequences in pieces
  int64_t piece_at[2], cut_at, decay_at, state_at, bytes;

  Layout(int64_t rows, int64_t nseqs, int64_t heads, int64_t dv, int64_t dk) {
    const int64_t sms = ssu::sm_count();
    const int64_t chunks = (rows + kC - 1) / kC;
    // every SM's share of the chunks; sequences beyond it are cut into pieces of a third of it
    const int64_t all = (chunks * heads + sms - 1) / sms;
    const int64_t share = all < 1 << 30 ? all : 1 << 30;  // (a single SM's of 2^31 rows)
    cut = (int)((share + 2) / 3 > 4 ? (share + 2) / 3 : 4);
    // ... where that saves more than the two launches it takes, some four chunks' time
    const int64_t worth = 2 * (int64_t)cut + 4;
    fair = (int)(share > worth ? share : worth);
    // a cut sequence has more than 64 `fair` rows, c > fair chunks and at most c / cut + 1
    // pieces; all of them together have at most rows / 64 + 1 chunks each
    const int64_t most = rows / ((int64_t)kC * fair);
    split = nseqs < most ? nseqs : most;
    entries = split ? (rows / kC + split) / cut + split : 0;
    pieces = nseqs + entries;
    auto round = [](int64_t n) { return (n + 255) / 256 * 256; };
    int64_t at = 256;  // the header
    for (int i = 0; i < 2; ++i) {
      piece_at[i] = at;
      at += round((i ? pieces : entries) * (int64_t)sizeof(Piece));
    }
    cut_at = at;
    at += round(split * (int64_t)sizeof(CutSeq));
    decay_at = at;
    at += round(entries * heads * 4);
    state_at = at;
    at += entries * heads * dv * dk * 4;
    bytes = at;
  }
};

bool takes_prompt(int64_t rows, int64_t nseqs, int64_t heads, int64_t dv, int64_t dk,
                  ssu_dtype io) {
  if ((io != SSU_BF16 && io != SSU_F16) || (dv != 64 && dv != 128) || (dk != 64 && dk != 128))
    return false;
  return nseqs * heads < 1LL << 30;  // items are counted in 32 bits
}

int64_t prompt_workspace(int64_t rows, int64_t nseqs, int64_t heads, int64_t dv, int64_t dk) {
  return Layout(rows, nseqs, heads, dv, dk).bytes;
}

using Encode = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder, which is not linked against; looked up once.
static Encode encoder() {
  static const Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

// [rows][n][dim] 16-bit elements, strides in elements, as boxes of 64 rows x 1 x 64.
static bool map_of(CUtensorMap* map, bool bf16, const void* p, int64_t rows, int64_t n, int64_t dim,
                   int64_t row_stride, int64_t stride) {
  const Encode f = encoder();
  if (!f) return false;
  // a stride that is never taken may be anything the call allows
  if (n == 1) stride = dim;
  if (rows == 1) row_stride = n * stride;
  const cuuint64_t size[3] = {(cuuint64_t)dim, (cuuint64_t)n, (cuuint64_t)rows};
  const cuuint64_t bytes[2] = {(cuuint64_t)stride * 2, (cuuint64_t)row_stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)kC}, step[3] = {1, 1, 1};
  return f(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
           const_cast<void*>(p), size, bytes, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_prompt(const Args& p, const Seqs& a, ssu_dtype io, void* workspace,
                          cudaStream_t stream) {
  const Layout l(a.rows, a.n, p.H, p.dv, p.dk);
  char* ws = static_cast<char*>(workspace);
  PromptArgs g{};
  g.p = p;
  g.a = a;
  g.head = reinterpret_cast<Header*>(ws);
  for (int i = 0; i < 2; ++i) g.pieces[i] = reinterpret_cast<Piece*>(ws + l.piece_at[i]);
  g.cuts = reinterpret_cast<CutSeq*>(ws + l.cut_at);
  g.decay = reinterpret_cast<float*>(ws + l.decay_at);
  g.state = reinterpret_cast<float*>(ws + l.state_at);
  g.fair = l.fair;
  g.cut = l.cut;
  g.entries = (int)l.entries;
  g.splits = (int)l.split;
  g.err = ssu::device_error_word();
  if (!g.err) return cudaErrorInvalidValue;
  if (!map_of(&g.q, io == SSU_BF16, p.q, a.rows, p.G, p.dk, p.q_rs, p.q_gs) ||
      !map_of(&g.k, io == SSU_BF16, p.k, a.rows, p.G, p.dk, p.k_rs, p.k_gs) ||
      !map_of(&g.v, io == SSU_BF16, p.v, a.rows, p.H, p.dv, p.v_rs, p.v_hs))
    return cudaErrorInvalidValue;
  linattn_plan_kernel<<<1, kPlanThreads, 0, stream>>>(g);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t sms = ssu::sm_count();
  auto ctas = [&](int64_t pieces) {
    const int64_t items = pieces * p.H;
    return (int)(items < sms ? items : sms);
  };
  const bool bf16 = io == SSU_BF16;
  if (l.entries > 0) {
    e = (bf16 ? launch_pieces_bf16 : launch_pieces_f16)(g, ctas(l.entries), stream);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)p.H * p.dv * p.dk / 4;
    e = launch_after(linattn_join_kernel,
                     dim3((unsigned)((items + kJoinThreads - 1) / kJoinThreads), (unsigned)l.split),
                     kJoinThreads, 0, stream, g);
    if (e != cudaSuccess) return e;
  }
  return (bf16 ? launch_chunks_bf16 : launch_chunks_f16)(g, ctas(l.pieces), stream);
}

}  // namespace linattn
