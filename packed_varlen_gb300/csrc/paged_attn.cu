// Attention of packed new tokens over a paged K/V cache: the entry point.
//
// Sequences of few query rows are bound by the cache's bytes and take the
// streaming kernel (paged_decode.cu), longer ones by tensor operations and
// take the tiled one (paged_chunk.cu); a mixed batch launches both, and each
// skips the other's sequences.
#include <math.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_chunk_work.cuh"
#include "paged_launch.h"

namespace pa {
namespace {

// Largest token counts and lengths: sums of two stay within 32 bits.
constexpr int32_t kMostTokens = 1 << 30;

// Bytes of widened rows up to which a call over an 8-bit cache widens ahead.
constexpr int64_t kWidenMost = int64_t{1} << 30;

// The most workspace that a call asks for.  Where the bounds could need more for the
// whole batch at once, the sequences go in several turns that use the same memory, as
// few as fit (a sequence's bits are its own, so the turns change none); a caller
// that gives more gets fewer.  GPU time of two turns against one: 100 sequences of
// 60-64 tokens over 2-30k keys 1811 / 1772 us, 128 of 1-12 over 0-40k 1409 / 1376.
constexpr int64_t kWorkspaceMost = int64_t{1} << 31;

// Where the partial results of a turn lie in the workspace.
struct WorkspacePlan {
  int64_t dec_slots;
  int dec_parts, dec_rows;
  int64_t chunk_rows, chunk_row0_rest;
  int chunk_cuts, chunk_cut0_rest;
  int64_t flat_pages;
  int flat_seqs;
  int64_t dec_o, dec_ml, chunk_o, chunk_ml, chunk_join, chunk_n_cuts;   // byte offsets
  int64_t flat_k, flat_v, flat_page;
  int64_t bytes;
};

WorkspacePlan workspace_plan(int batch, int total_q, int max_q, int max_k, int Hq, int Hkv, int D,
                             int format) {
  WorkspacePlan w{};
  const int G = Hq / Hkv;
  int tokens = max_q < total_q ? max_q : total_q;   // of a sequence in the streaming kernel
  if (tokens > kFewRows / G) tokens = kFewRows / G;
  w.dec_parts = 1;
  w.dec_rows = tokens * Hq;
  if (tokens > 0 && !paged_decode_is_local(batch, tokens, max_k, G, Hkv)) {
    for (int groups = 1; groups <= row_groups(tokens, G); ++groups) {
      const int parts = decode_parts_bound(max_k, groups, Hkv);
      const int rows = groups * kGroupRows < tokens * G ? groups * kGroupRows : tokens * G;
      if (parts > w.dec_parts) w.dec_parts = parts;
      if (parts > 1 && static_cast<int64_t>(rows) * Hkv * parts > w.dec_slots)
        w.dec_slots = static_cast<int64_t>(rows) * Hkv * parts;
    }
  }
  const int64_t slots = w.dec_slots * batch;

  const int item_tokens = 2 * (kChunkTile / G);
  const int few = kFewRows / G;   // tokens up to which no sequence takes the tiled kernel
  const int64_t tiles_k = (static_cast<int64_t>(max_k) + kChunkTile - 1) / kChunkTile;
  auto most_seqs = [&](int least) -> int64_t {   // sequences of at least so many tokens
    const int64_t n = max_q < least ? 0 : total_q / least;
    return n < batch ? n : batch;
  };
  // Shares of a sequence of i items a head, of at least kChunkMinShare key tiles each;
  // none where no sequence can have enough keys to be cut.
  auto shares_of = [&](int64_t i) -> int64_t {
    if (i * Hkv > kChunkShares * kChunkMinShare) return kChunkShares;   // (nothing overflows)
    const int64_t n = (i * Hkv * tiles_k + kChunkMinShare - 1) / kChunkMinShare;
    return n < kChunkShares ? n : kChunkShares;
  };
  // Cuts and workspace rows of so many sequences of i_from to i_to items a head: the
  // rows are bounded by the sequences and by the tokens, of which few make few items
  // and these few shares.
  auto add_cuts = [&](int64_t seqs, int64_t i_from, int64_t i_to) {
    if (tiles_k <= kChunkMinShare || seqs == 0) return;
    auto slots_of = [&](int64_t i) { return chunk_slots(shares_of(i), i * Hkv); };
    const int64_t all = static_cast<int64_t>(G) * total_q;
    int64_t by_tokens = 0;
    for (int64_t i = i_from; i <= i_to; ++i) {
      // rows of sequences of the least tokens that have i items, as many as the call
      // can have (one item: rows go with its tokens)
      auto rows = [&](int64_t slots) {
        return i == 1 ? slots * all : slots * all * item_tokens / ((i - 1) * item_tokens + 1) + 1;
      };
      if (rows(2 * kChunkShares) <= by_tokens) break;   // nor has any i after this one more
      if (rows(slots_of(i)) > by_tokens) by_tokens = rows(slots_of(i));
    }
    const int64_t by_seqs = slots_of(i_to) * seqs * G * (max_q < item_tokens ? max_q : item_tokens);
    w.chunk_cuts += static_cast<int>(seqs * shares_of(i_to));
    w.chunk_rows += by_seqs < by_tokens ? by_seqs : by_tokens;
  };
  const int64_t items = (static_cast<int64_t>(max_q) + item_tokens - 1) / item_tokens;
  if (format == PA_CACHE_E4M3) {
    const int64_t seqs = most_seqs(2 * item_tokens + 1), pages = seqs * tiles_k;
    if (pages * kChunkTile * Hkv * D * 4 <= kWidenMost && pages < (1 << 24)) w.flat_pages = pages;
    w.flat_seqs = static_cast<int>(seqs);
  }
  if (w.flat_pages > 0) {
    add_cuts(most_seqs(2 * item_tokens + 1), 3, items);
    w.chunk_row0_rest = w.chunk_rows;
    w.chunk_cut0_rest = w.chunk_cuts;
    add_cuts(most_seqs(few + 1), 1, items < 2 ? items : 2);
  } else {
    add_cuts(most_seqs(few + 1), 1, items);
  }
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 15) & ~int64_t{15};
    return here;
  };
  w.dec_o = take(slots * D * 4);
  w.dec_ml = take(slots * 8);
  w.chunk_o = take(w.chunk_rows * D * 4);
  w.chunk_ml = take(w.chunk_rows * 8);
  w.chunk_join = take(static_cast<int64_t>(w.chunk_cuts) * 32);
  w.chunk_n_cuts = take(w.chunk_cuts > 0 ? 16 : 0);
  w.flat_page = take(w.flat_pages > 0 ? static_cast<int64_t>(batch) * 4 : 0);
  w.flat_k = take(w.flat_pages * kChunkTile * Hkv * D * 2);
  w.flat_v = take(w.flat_pages * kChunkTile * Hkv * D * 2);
  w.bytes = at;
  return w;
}

// The turns of a call: `batch` sequences each, the last one the rest.
struct TurnPlan {
  int batch, last;
  WorkspacePlan w, w_last;
};
// As few as `most` bytes have room for (a sequence alone takes 1.1 GB at most).
TurnPlan turn_plan(int batch, int total_q, int max_q, int max_k, int Hq, int Hkv, int D, int format,
                   int64_t most) {
  auto plan = [&](int n) { return workspace_plan(n, total_q, max_q, max_k, Hq, Hkv, D, format); };
  TurnPlan t{batch, batch, plan(batch), {}};
  for (int turns = 2; (t.w.bytes > most || t.w_last.bytes > most) && t.batch > 1; ++turns) {
    t.batch = (batch + turns - 1) / turns;
    t.last = (batch - 1) % t.batch + 1;
    t.w = plan(t.batch);
    t.w_last = plan(t.last);
  }
  return t;
}

// Launches of one turn, whose sequences p.cu_q, p.seq_lens and p.c.table begin at.
cudaError_t launch_turn(PagedAttnParams &p, const WorkspacePlan &w, uint8_t *ws, bool quant, int sms,
                        cudaStream_t s) {
  p.dec_parts = w.dec_parts;
  p.dec_rows = w.dec_rows;
  p.dec_slots = w.dec_slots;
  p.dec_o = reinterpret_cast<float *>(ws + w.dec_o);
  p.dec_ml = reinterpret_cast<float2 *>(ws + w.dec_ml);
  p.chunk_o = reinterpret_cast<float *>(ws + w.chunk_o);
  p.chunk_ml = reinterpret_cast<float2 *>(ws + w.chunk_ml);
  p.chunk_join = reinterpret_cast<int4 *>(ws + w.chunk_join);
  p.chunk_n_cuts = reinterpret_cast<int32_t *>(ws + w.chunk_n_cuts);
  p.chunk_rows = w.chunk_rows;
  p.chunk_cuts = w.chunk_cuts;
  p.chunk_row0_rest = w.chunk_row0_rest;
  p.chunk_cut0_rest = w.chunk_cut0_rest;
  p.flat_k = reinterpret_cast<__nv_bfloat16 *>(ws + w.flat_k);
  p.flat_v = reinterpret_cast<__nv_bfloat16 *>(ws + w.flat_v);
  p.flat_page = reinterpret_cast<int32_t *>(ws + w.flat_page);
  p.flat_pages = static_cast<int>(w.flat_pages);
  p.flat_seqs = w.flat_seqs;
  // The long sequences first; the streaming kernel fills the SMs that they leave.
  const bool chunk = !decode_takes(p.max_q, p.G), few = p.G <= kFewRows;
  cudaError_t e = cudaSuccess;
  if (chunk) e = launch_paged_chunk(p, quant, sms, s);
  if (e == cudaSuccess && few) e = launch_paged_decode(p, quant, sms, chunk, s);
  if (e == cudaSuccess && (p.dec_parts > 1 || p.chunk_cuts > 0)) e = launch_paged_join(p, sms, s);
  return e;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int64_t pa_paged_attn_workspace_bytes(int32_t batch, int32_t total_q, int32_t max_q,
                                                 int32_t max_k, int32_t Hq, int32_t Hkv,
                                                 int32_t D, int32_t format) {
  if (batch < 1 || batch > PA_MAX_BATCH || total_q < 0 || max_q < 0 || max_k < 0 || Hkv < 1 ||
      Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > kChunkTile || Hkv > 4096 || total_q > kMostTokens ||
      max_q > kMostTokens || max_k > kMostTokens || (D != 64 && D != 128) ||
      (format != PA_CACHE_BF16 && format != PA_CACHE_E4M3))
    return -1;
  const int64_t bytes = workspace_plan(batch, total_q, max_q, max_k, Hq, Hkv, D, format).bytes;
  return bytes < kWorkspaceMost ? bytes : kWorkspaceMost;
}

extern "C" pa_status pa_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache,
                                       const uint8_t *k_exp, const uint8_t *v_exp, void *out,
                                       const int32_t *cu_seqlens_q, const int32_t *seq_lens,
                                       const int32_t *page_table, int32_t batch,
                                       int32_t total_q, int32_t max_q, int32_t max_k,
                                       int64_t q_stride, int32_t num_pages, int32_t page_size,
                                       int32_t table_pages, int64_t page_stride, int32_t Hq,
                                       int32_t Hkv, int32_t D, int32_t format, int32_t causal,
                                       float scale, void *workspace, int64_t workspace_bytes,
                                       pa_stream_t stream) {
  if (!cu_seqlens_q || !seq_lens) return PA_ERR_INVALID_ARG;
  if (batch < 1 || total_q < 0 || max_q < 0 || max_k < 0 || Hq < 1) return PA_ERR_INVALID_ARG;
  if (total_q > 0 && (!q || !out)) return PA_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;   // of weights as powers of two
  if (!isfinite(scale_log2)) return PA_ERR_INVALID_ARG;
  PagedAttnParams p;
  const PagedCacheArgs a{const_cast<void *>(k_cache), const_cast<void *>(v_cache),
                         const_cast<uint8_t *>(k_exp), const_cast<uint8_t *>(v_exp),
                         page_table, num_pages, page_size, table_pages, page_stride, Hkv, D,
                         format};
  const pa_status st = check_cache(a, p.c);
  if (st != PA_OK) return st;
  if (Hq % Hkv != 0 || q_stride < static_cast<int64_t>(Hq) * D) return PA_ERR_INVALID_ARG;
  if (batch > PA_MAX_BATCH || Hq / Hkv > kChunkTile || q_stride > (int64_t{1} << 38) ||
      total_q > kMostTokens || max_q > kMostTokens || max_k > kMostTokens)
    return PA_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(cu_seqlens_q, 4) ||
      !aligned_to(seq_lens, 4) || (q_stride & 7) != 0 || !aligned_to(workspace, 16))
    return PA_ERR_MISALIGNED;
  // (every size that the plan needs has been checked by now)
  const TurnPlan turns =
      turn_plan(batch, total_q, max_q, max_k, Hq, Hkv, D, format,
                workspace_bytes > kWorkspaceMost ? workspace_bytes : kWorkspaceMost);
  const int64_t need = turns.batch < batch ? kWorkspaceMost : turns.w.bytes;
  if (workspace_bytes < need || (need > 0 && !workspace)) return PA_ERR_INVALID_ARG;
  if (total_q == 0 || max_q == 0) return PA_OK;
  int sms;
  cudaError_t e = device_context(&p.status, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.q_stride = q_stride;
  p.total_q = total_q;
  p.max_q = max_q;
  p.max_k = max_k;
  p.Hq = Hq;
  p.causal = causal;
  p.scale_log2 = scale_log2;
  p.G = Hq / Hkv;
  p.g_inv = (1 << 16) / p.G + 1;
  p.dec_most = decode_most_parts(Hkv);
  p.capacity = static_cast<int64_t>(table_pages) * page_size;
  p.chunk_set = kSetAll;
  p.chunk_row0 = p.chunk_cut0 = 0;
  auto s = reinterpret_cast<cudaStream_t>(stream);
  for (p.batch0 = 0; p.batch0 < batch && e == cudaSuccess; p.batch0 += turns.batch) {
    const bool rest = batch - p.batch0 < turns.batch;
    p.batch = rest ? turns.last : turns.batch;
    p.cu_q = cu_seqlens_q + p.batch0;
    p.seq_lens = seq_lens + p.batch0;
    p.c.table = page_table + static_cast<int64_t>(p.batch0) * table_pages;
    e = launch_turn(p, rest ? turns.w_last : turns.w, static_cast<uint8_t *>(workspace),
                    format == PA_CACHE_E4M3, sms, s);
  }
  return from_cuda(e);
}
