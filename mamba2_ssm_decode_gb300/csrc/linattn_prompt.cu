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
  int64_t entries, pieces;  // most states, most pieces
  int64_t piece_at[2], decay_at, state_at, bytes;

  Layout(int64_t rows, int64_t nseqs, int64_t heads, int64_t dv, int64_t dk) {
    const int64_t sms = ssu::sm_count();
    const int64_t chunks = (rows + kC - 1) / kC;
    // every SM's share of the chunks; sequences beyond it are cut into pieces of a third of it
    const int64_t share = (chunks * heads + sms - 1) / sms;
    cut = (int)(share / 3 > 4 ? share / 3 : 4);
    fair = (int)(share > cut ? share : cut);
    // a cut sequence has more than 64 `fair` rows, c > fair chunks and at most c / cut + 1
    // pieces; all of them together have at most rows / 64 + 1 chunks each
    const int64_t most = rows / ((int64_t)kC * fair);
    const int64_t split = nseqs < most ? nseqs : most;
    entries = split ? (rows / kC + split) / cut + split : 0;
    pieces = nseqs + entries;
    auto round = [](int64_t n) { return (n + 255) / 256 * 256; };
    int64_t at = 256;  // the header
    for (int i = 0; i < 2; ++i) {
      piece_at[i] = at;
      at += round((i ? pieces : entries) * (int64_t)sizeof(Piece));
    }
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

cudaError_t launch_prompt(const Args& p, const Seqs& a, ssu_dtype io, void* workspace,
                          cudaStream_t stream) {
  const Layout l(a.rows, a.n, p.H, p.dv, p.dk);
  char* ws = static_cast<char*>(workspace);
  PromptArgs g{};
  g.p = p;
  g.a = a;
  g.head = reinterpret_cast<Header*>(ws);
  for (int i = 0; i < 2; ++i) g.pieces[i] = reinterpret_cast<Piece*>(ws + l.piece_at[i]);
  g.decay = reinterpret_cast<float*>(ws + l.decay_at);
  g.state = reinterpret_cast<float*>(ws + l.state_at);
  g.fair = l.fair;
  g.cut = l.cut;
  g.entries = (int)l.entries;
  g.err = ssu::device_error_word();
  if (!g.err) return cudaErrorInvalidValue;
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
  }
  return (bf16 ? launch_chunks_bf16 : launch_chunks_f16)(g, ctas(l.pieces), stream);
}

}  // namespace linattn
