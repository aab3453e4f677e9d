// Paged attention of sequences with many query rows, on the 5th-generation
// tensor cores: chunks of long inputs over everything cached before them.
//
// Bound by the tensor pipe once a K/V head's rows fill its tiles, and by what a
// piece of work costs around its tiles where it has few: GPU time, 32 query
// heads on 8 of 128, 2048 tokens over 14k keys 320 us (504 GFLOP, 1577
// TFLOP/s; some 2900 cycles for a key tile of 256 rows, of which the products
// are 2100); two 8-bit chunks of 600 tokens over 7000, 28 heads on 4, 124 us
// (975 TFLOP/s).  A call's first weights come 20,000 cycles after its start, a
// third of them cold instructions, and a piece ends with 5000 cycles in
// which its 128 KB go out.  Grouped
// query heads share their K/V head's keys, so a 128-row tile holds the whole
// group of 128 / G tokens (row = token * G + head of the group): each K/V
// byte brought to shared memory serves G heads.  Otherwise the kernel is the
// single-CTA packed attention kernel (attn_tc.cu) with its K/V tiles
// assembled from pages: one persistent CTA per SM, two 128-row tiles that
// share every K/V tile, S and O of both in TMEM, P over S.
//   warp 0       TMA producer: Q once per item, then K0, V0, K1, V1, ..., each
//                tile one copy per page (or per 128 rows of a larger page) and
//                64 columns; pages past the sequence's last key are fetched
//                from an out-of-range page, so they land as zeros.
//   warps 1, 2   issue tile 0's and tile 1's tcgen05.mma in turn.  Where an item
//                has rows for one tile only, the two take its even and its odd
//                key tiles, and the epilogue adds the two outputs up.
//   warps 3..6   softmax of tile 0, a thread per row; warps 7..10 of tile 1.
//   warps 11..18 (8-bit caches) widen the rows that the producer fetched into
//                the bf16 tiles that the products read.
// A unit of work is whole items or a share of the sequence's key tiles
// (paged_chunk_work.cuh); a part of an item leaves its unnormalised output,
// maximum and sum in the workspace, and paged_join_kernel joins them.
// Keys that a row does not see are masked to -inf; V rows past the sequence's
// last key are cleared in shared memory before any product reads them (0 *
// NaN would be NaN); rows of a tile beyond its tokens are computed from
// whatever lies there and never stored.  Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_chunk_work.cuh"
#include "paged_launch.h"
#include "tc_ptx.cuh"
#include "tma_map.h"

namespace pa {
namespace {

using namespace tc;

constexpr int kTile = kChunkTile;
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (~2 s)
constexpr long long kDrainLimit = 400000000LL;  // teardown after an abort (~0.2 s)
constexpr float kRescaleThreshold = 8.0f;       // log2 units

template <int D, bool kQuant>
struct Cfg {
  static constexpr int kSoftmaxWarp = 3;                    // first of eight
  static constexpr int kWidenWarp = kSoftmaxWarp + 8;       // first of kWideners (8-bit caches)
  static constexpr int kWideners = 8;
  static constexpr int kThreads = (kWidenWarp + (kQuant ? kWideners : 0)) * 32;
  // columns of S that a softmax thread holds at a time: the whole row where 352
  // threads share the registers (read once: 2048 tokens over 14k keys in 336 us,
  // 360 with two passes over 64), a quarter where 608 do
  static constexpr int kCols = kQuant ? 32 : 128;
  static constexpr int kSlots = kQuant ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 8);
  static constexpr int kRaws = kQuant ? kSlots : 0;         // 8-bit tiles as they arrive
  static constexpr int kRawBytes = kTile * D;
  static constexpr int kPieces = 4;                         // told ahead by the producer
  static constexpr int kReaders = 2 + 8 + (kQuant ? kWideners : 0);   // warps that read them
  static constexpr int kHalfBytes = kTile * 64 * 2;         // 128 rows x 128 B
  static constexpr int kTileBytes = kTile * D * 2;          // one Q/K/V tile
  static constexpr int kQOff = 0;                           // Q0, Q1
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kRawOff = kRingOff + kSlots * kTileBytes;
  static constexpr int kBarOff = kRawOff + kRaws * kRawBytes;
  // barriers: per Q tile t an S-full, a P-ready and an O-full barrier
  static constexpr int kQFull = 0, kQEmpty = 1, kSFull = 2, kPReady = 4, kOFull = 6,
                       kFinal = 8, kTurn = 10, kSlotFull = 12, kSlotEmpty = 12 + kSlots,
                       kRawFull = 12 + 2 * kSlots, kRawEmpty = kRawFull + kRaws,
                       kPieceFull = kRawEmpty + kRaws, kPieceEmpty = kPieceFull + kPieces,
                       kBothDone = kPieceEmpty + kPieces, kBothRead = kBothDone + 1;
  static constexpr int kNumBars = kBothRead + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;   // tmem base, abort flag, counter
  static constexpr int kSchedOff = (kMiscOff + 16 + 127) / 128 * 128;
  // order, first part row, first cut unit and first unit of each sequence in the list
  static constexpr int kPieceOff = kSchedOff + ((4 * PA_MAX_BATCH + 2) * 4 + 15) / 16 * 16;
  static constexpr int kStatOff = kPieceOff + kPieces * 64;   // (maximum, sum) of [tile][row]
  static constexpr int kSmemBytes = kStatOff + 2 * kTile * 8;
  static_assert(kSmemBytes <= 232448, "shared memory plan exceeds the per-CTA limit");
  // TMEM columns: S_t at 128 t (P_t over its first 64), O_t at 256 + D t
  static constexpr uint32_t kColS = 0;
  static constexpr uint32_t kColO = 256;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(kTile, kTile, false);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(kTile, D, true);
  // V (MN-major): next 64-column half at LBO, next 8 keys at SBO = 1024.  With
  // D = 64 the MMA spans a single half and LBO is never used.
  static constexpr uint32_t kVLbo = D == 128 ? kHalfBytes : 1024;
};

// Whole warp: zero key rows [valid, 128) of a V tile in shared memory (its
// column halves are 128 rows of 128 bytes; the swizzle permutes 16-byte chunks
// inside a row only).  The fences order the stores after the bytes that
// landed and before the tensor core's reads.
template <int D>
__device__ __forceinline__ void zero_v_tail(uint8_t *tile, int valid, int lane) {
  fence_proxy_async();
  const int per_half = (kTile - valid) * 8;   // 16-byte chunks per half
  for (int c = lane; c < per_half * (D / 64); c += 32) {
    const int hf = c / per_half, r = c - hf * per_half;
    *reinterpret_cast<uint4 *>(tile + hf * (kTile * 128) + (valid + (r >> 3)) * 128 +
                               (r & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async();
  __syncwarp();
}

// Loads that are issued where they are written, ahead of their use (a plain
// __ldg may be moved down to it).
__device__ __forceinline__ int32_t load_now(const int32_t *p) {
  int32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int load_now(const uint8_t *p) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];\n" : "=r"(v) : "l"(p));
  return static_cast<int>(v);
}

// Two e4m3 bytes of w, as `sel` puts them in bytes 0 and 2, to bf16: times 16
// their seven low bits lie in bf16's place and the sign at bit 11, which the sum
// carries on to bit 15.  That is the value times 2^-120, subnormals included, and
// one packed multiply by 2^(120 + e) makes it the exact stored value.
__device__ __forceinline__ uint32_t widen_pair(uint32_t w, uint32_t scale, uint32_t sel) {
  return mul_bf16x2((__byte_perm(w, 0u, sel) * 16u + 0x78007800u) & 0x87f087f0u, scale);
}
// A byte of 0x7f or 0xff is e4m3's NaN, which a write never makes but a cache
// filled elsewhere may hold; widen_pair takes it for 480.  Not 0 where 16 bytes hold one:
__device__ __forceinline__ uint32_t holds_nan(const uint4 &y) {
  auto carry = [](uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; };
  return (carry(y.x) | carry(y.y) | carry(y.z) | carry(y.w)) & 0x80808080u;
}
// widen_pair with NaN in its place; scale 0: no row of the sequence, and zeros.
__device__ __forceinline__ uint32_t widen_pair_nan(uint32_t w, uint32_t scale, uint32_t sel) {
  uint32_t r = widen_pair(w, scale, sel);
  const uint32_t y = __byte_perm(w, 0u, sel);
  if (scale != 0u && (y & 0x7fu) == 0x7fu) r |= 0x7fffu;
  if (scale != 0u && (y & 0x7f0000u) == 0x7f0000u) r |= 0x7fff0000u;
  return r;
}

// The sequences of the call that take this launch, most keys first, with the
// prefixes of their units, of those that may cut items (shares), and of the
// workspace rows of their parts: first[n] = all units, cut0[n] = all shares.
// Only the producer reads it.  Up to 32 sequences that warp makes it alone, a
// sequence to a lane, while the other warps go on; more are ranked by all of
// the CTA's threads first.
struct WorkList {
  int32_t *order, *first, *cut0, *part0;   // in shared memory
  int32_t *units, *rows;                   // temporaries: units, rows of all parts (0: never cut)
};
__device__ __forceinline__ bool in_launch(const PagedAttnParams &p, int lq) {
  return !decode_takes(lq, p.G) &&
         (p.chunk_set == kSetAll || chunk_widens(lq, p.G) == (p.chunk_set == kSetFlat));
}
__device__ __forceinline__ ChunkWork note_units(const PagedAttnParams &p, const WorkList &x, int at,
                                                const PagedSeq &s) {
  const ChunkWork w = chunk_work(s.lq, s.lk, p.causal, p.G, p.c.Hkv);
  x.units[at] = w.units;
  x.rows[at] = w.share ? static_cast<int32_t>(chunk_slots(w.units, w.items_head * p.c.Hkv)) *
                             chunk_part_rows(s.lq, p.G)
                       : 0;
  return w;
}
// One warp.  Returns the sequences; lane b keeps sequence b and its work.
__device__ __forceinline__ int rank_few(const PagedAttnParams &p, const WorkList &x, PagedSeq &s,
                                        ChunkWork &w, bool report) {
  const int lane = threadIdx.x & 31;
  int err = 0;
  if (lane < p.batch)
    s = paged_seq(p, lane, err);
  if (err && report) record_error(p.status, err);
  const bool in = lane < p.batch && in_launch(p, s.lq);
  const uint32_t all = __ballot_sync(0xffffffffu, in);
  int rank = 0;
#pragma unroll 1
  for (uint32_t rest = all; rest; rest &= rest - 1) {
    const int y = __ffs(rest) - 1;
    const int lk = __shfl_sync(0xffffffffu, s.lk, y);
    rank += lk > s.lk || (lk == s.lk && y < lane);
  }
  if (in) {
    x.order[rank] = lane;
    w = note_units(p, x, rank, s);
  }
  __syncwarp();
  return __popc(all);
}
// All threads; ends with __syncthreads().
__device__ __forceinline__ int rank_many(const PagedAttnParams &p, const WorkList &x,
                                         int32_t *count, bool report) {
  const int tid = threadIdx.x, nt = blockDim.x;
  int32_t *seq = x.units, *keys = x.rows;
  for (int b = tid; b < p.batch; b += nt) {
    int err;
    const PagedSeq s = paged_seq(p, b, err);
    if (err && report) record_error(p.status, err);
    if (in_launch(p, s.lq)) {
      const int at = atomicAdd(count, 1);   // any order: the ranks below are the list's
      seq[at] = b;
      keys[at] = s.lk;
    }
  }
  __syncthreads();
  const int n = *count;
  for (int y = tid; y < n; y += nt) {
    const int b = seq[y], lb = keys[y];
    int rank = 0;
    for (int z = 0; z < n; ++z) rank += (keys[z] > lb) || (keys[z] == lb && seq[z] < b);
    x.order[rank] = b;
  }
  __syncthreads();
  for (int y = tid; y < n; y += nt) {
    int err;
    note_units(p, x, y, paged_seq(p, x.order[y], err));
  }
  fence_proxy_async();   // the ring's copies come after every access to the temporaries there
  __syncthreads();
  return n;
}
// One warp, after either: the prefixes.  Returns the sequences that are worked on.
__device__ __forceinline__ int add_up(const PagedAttnParams &p, const WorkList &x, int n, bool report) {
  const int lane = threadIdx.x & 31;
  // Boundaries that overlap can name more tokens than the call has, and so
  // more parts than the workspace has room for: the list ends before those.
  const int most_cuts = p.chunk_set == kSetFlat ? p.chunk_cut0_rest : p.chunk_cuts;
  const int64_t most_rows = p.chunk_set == kSetFlat ? p.chunk_row0_rest : p.chunk_rows;
  int units = 0, cuts = p.chunk_cut0, rows = static_cast<int>(p.chunk_row0), fit = n;
#pragma unroll 1
  for (int base = 0; base < n; base += 32) {
    const int y = base + lane;
    const int u = y < n ? x.units[y] : 0, r = y < n ? x.rows[y] : 0;
    const int k = r > 0 ? u : 0;
    int iu = u, ik = k, ir = r;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
      const int yu = __shfl_up_sync(0xffffffffu, iu, off);
      const int yk = __shfl_up_sync(0xffffffffu, ik, off);
      const int yr = __shfl_up_sync(0xffffffffu, ir, off);
      if (lane >= off) {
        iu += yu;
        ik += yk;
        ir += yr;
      }
    }
    if (y < n) {
      x.first[y] = units + iu - u;
      x.cut0[y] = cuts + ik - k;
      x.part0[y] = rows + ir - r;
      if (r > 0 && (cuts + ik > most_cuts || rows + ir > most_rows) && y < fit) fit = y;
    }
    units += __shfl_sync(0xffffffffu, iu, 31);
    cuts += __shfl_sync(0xffffffffu, ik, 31);
    rows += __shfl_sync(0xffffffffu, ir, 31);
  }
  if (lane == 0) {
    x.first[n] = units;
    x.cut0[n] = cuts;
  }
  fit = __reduce_min_sync(0xffffffffu, fit);
  if (fit < n && lane == 0 && report) record_error(p.status, PA_DEVICE_ERR_CU_SEQLENS);
  fence_proxy_async();   // as in rank_many
  __syncwarp();
  return fit;
}

// A piece as the producer tells the other warps of it: finding a unit's place
// takes some 10,000 cycles the first time (mostly instruction fetch), so one
// warp does it, ahead of the others.
struct Piece {
  int32_t j0, j1;       // key tiles; j1 = 0: no more pieces
  int32_t q0, tok0;     // the sequence's first row of q, the item's first token
  int32_t tokens, head;
  int32_t lk, before;   // the sequence's keys, and those before its first query
  int32_t slot;         // workspace row of a part, or -1: the item is whole
  int32_t b;            // the sequence
  int32_t part_rows;    // rows of a part in the workspace
  int32_t pad[5];
};
static_assert(sizeof(Piece) == 64, "four 16-byte reads");

// A unit's sequence, and the walk over its pieces.
struct Unit {
  PagedSeq s;
  int b, local;       // sequence, unit within it
  int at;             // place of the sequence in the list
  int part_rows;      // workspace rows of one part
  bool by_piece;      // how its parts are placed (chunk_slots)
  int flat_page;      // first page of its widened rows (kSetFlat)
  int64_t part0;      // workspace row of the sequence's first part
  ChunkWork w;
  ChunkCursor cur;
};
// Whole warp.  `s` and `w`: sequence `lane` and its work, where the call has 32 at most.
__device__ __forceinline__ void open_unit(const PagedAttnParams &p, const WorkList &list, int n, int u,
                                          const PagedSeq &s, const ChunkWork &w, Unit &x) {
  int lo = 0, hi = n;   // largest i < n with first[i] <= u (every sequence has a unit)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list.first[mid] <= u) lo = mid; else hi = mid;
  }
  x.b = list.order[lo];
  if (p.batch <= 32) {
    auto from = [&](auto v) { return __shfl_sync(0xffffffffu, v, x.b); };
    x.s = PagedSeq{from(s.q0), from(s.lq), from(s.lk)};
    x.w.lq = x.s.lq;
    x.w.lk = x.s.lk;
    x.w.causal = p.causal;
    x.w.item_tokens = 2 * (kChunkTile / p.G);
    x.w.items_head = from(w.items_head);
    x.w.few = from(w.few);
    x.w.head_keys = from(w.head_keys);
    x.w.share = from(w.share);
  } else {
    int err;
    x.s = paged_seq(p, x.b, err);
    x.w = chunk_work(x.s.lq, x.s.lk, p.causal, p.G, p.c.Hkv);
  }
  x.local = u - list.first[lo];
  x.at = lo;
  x.part0 = list.part0[lo];
  x.part_rows = chunk_part_rows(x.s.lq, p.G);
  x.by_piece = x.w.items_head * p.c.Hkv < list.first[lo + 1] - list.first[lo];
  x.flat_page = p.chunk_set == kSetFlat ? p.flat_page[x.b] : 0;
  if (x.w.share == 0) {
    x.cur.start_whole(x.w, x.local, p.c.Hkv);
  } else {   // even lanes find the share's start, odd ones its end
    const ChunkPlace y = x.w.place_at((x.local + (threadIdx.x & 1)) * x.w.share, p.c.Hkv);
    auto from = [](int v, int lane) { return __shfl_sync(0xffffffffu, v, lane); };
    x.cur.at = ChunkPlace{from(y.head, 0), from(y.item, 0), from(y.j, 0)};
    x.cur.end = ChunkPlace{from(y.head, 1), from(y.item, 1), from(y.j, 1)};
  }
}

template <int D, bool kQuant>
__global__ void __launch_bounds__(Cfg<D, kQuant>::kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedAttnParams p) {
  using C = Cfg<D, kQuant>;
  extern __shared__ uint8_t smem_raw[];
  // 128-byte swizzle atoms need a 1024-byte aligned base
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {
    if (threadIdx.x == 0) record_error(p.status, PA_DEVICE_ERR_SMEM_ALIGN);
    griddep_wait();
    return;
  }
  uint8_t *gbase = smem_raw;
  const uint32_t sQ = base + C::kQOff;
  const uint32_t sRing = base + C::kRingOff;
  auto bar = [&](int idx) -> uint32_t { return base + C::kBarOff + 8u * idx; };
  uint32_t *tmem_base_ptr = reinterpret_cast<uint32_t *>(gbase + C::kMiscOff);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(gbase + C::kMiscOff + 4);
  int32_t *counter = reinterpret_cast<int32_t *>(gbase + C::kMiscOff + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();   // the streaming kernel may take the SMs that this one leaves
  // ---- set-up: barriers (warp 2), TMEM (warp 1), work list (warp 0) -------
  // (the ring is free until the first load: the list's temporaries lie there)
  int32_t *sched = reinterpret_cast<int32_t *>(gbase + C::kSchedOff);
  int32_t *tmp = reinterpret_cast<int32_t *>(gbase + C::kRingOff);
  const WorkList list{sched, sched + 3 * PA_MAX_BATCH + 1, sched + 2 * PA_MAX_BATCH,
                      sched + PA_MAX_BATCH, tmp, tmp + PA_MAX_BATCH};
  PagedSeq lane_seq{0, 0, 0};   // of sequence `lane`, where the call has 32 at most
  ChunkWork lane_work;
  int n_seqs = 0;
  if (tid == 64) {
    mbar_init(bar(C::kQFull), 1);
    mbar_init(bar(C::kQEmpty), 2);   // one arrival per MMA issuer
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(C::kSFull + t), 1);
      mbar_init(bar(C::kPReady + t), 128);
      mbar_init(bar(C::kOFull + t), 1);
      mbar_init(bar(C::kFinal + t), 1);
      mbar_init(bar(C::kTurn + t), 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(bar(C::kSlotFull + s), kQuant ? C::kWideners : 1);   // the widening warps, or the copy
      mbar_init(bar(C::kSlotEmpty + s), 2);   // one arrival per MMA issuer
    }
    for (int s = 0; s < C::kRaws; ++s) {
      mbar_init(bar(C::kRawFull + s), 1);
      mbar_init(bar(C::kRawEmpty + s), C::kWideners);
    }
    mbar_init(bar(C::kBothDone), 8);
    mbar_init(bar(C::kBothRead), 8);
    for (int s = 0; s < C::kPieces; ++s) {
      mbar_init(bar(C::kPieceFull + s), 1);
      mbar_init(bar(C::kPieceEmpty + s), C::kReaders);
    }
    *abort_flag = 0;
    if (p.batch > 32) *counter = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(base + C::kMiscOff, C::kTmemCols);
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    if (p.batch <= 32) {
      n_seqs = rank_few(p, list, lane_seq, lane_work, blockIdx.x == 0);
      if (lane == 0) *counter = n_seqs;
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_base_ptr;
  const int tile_tokens = kTile / p.G, tile_rows = tile_tokens * p.G;
  if (p.batch > 32) n_seqs = rank_many(p, list, counter, blockIdx.x == 0);
  if (*counter == 0) {   // none for this launch, as in a call whose bounds allow for them only
    if (blockIdx.x == 0 && tid == 0 && p.chunk_cuts > 0)
      p.chunk_n_cuts[p.chunk_set == kSetRest] = p.chunk_cut0;
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
    griddep_wait();
    return;
  }

  Piece *pieces = reinterpret_cast<Piece *>(gbase + C::kPieceOff);
  uint32_t pieces_read = 0;
  // the next piece, for each of the reading warps
  auto next_piece = [&](Piece &x) -> bool {
    const uint32_t at = pieces_read % C::kPieces;
    const bool told = bounded_wait(bar(C::kPieceFull + at), (pieces_read / C::kPieces) & 1u,
                                   abort_flag, p.status, kWaitLimit);
    if (!__all_sync(0xffffffffu, told)) return false;
    ++pieces_read;
    x = pieces[at];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kPieceEmpty + at));
    return x.j1 > 0;
  };

  if (warp == 0) {
    // ================= TMA producer =================
    // fills K/V slots, or (8-bit caches) the buffers that the widening warps read
    constexpr int kBufs = kQuant ? C::kRaws : C::kSlots;
    constexpr int kFull = kQuant ? C::kRawFull : C::kSlotFull;
    constexpr int kEmpty = kQuant ? C::kRawEmpty : C::kSlotEmpty;
    constexpr int kBufBytes = kQuant ? C::kRawBytes : C::kTileBytes;
    const uint32_t sBuf = base + (kQuant ? C::kRawOff : C::kRingOff);
    const bool lead = elect_one();
    n_seqs = add_up(p, list, n_seqs, blockIdx.x == 0);
    const int n_units = list.first[n_seqs];
    if (blockIdx.x == 0 && lead && p.chunk_cuts > 0)
      p.chunk_n_cuts[p.chunk_set == kSetRest] = list.cut0[n_seqs];
    // rows that the launch before this one widens
    if (p.chunk_set == kSetFlat) griddep_wait();
    uint32_t q_loads = 0, slot_loads = 0;
    bool ok = true;
    auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
      const bool w = bounded_wait(b, parity, abort_flag, p.status, kWaitLimit);
      return __all_sync(0xffffffffu, w);
    };
    const int box_rows = min(1 << p.c.page_shift, kTile), boxes = kTile / box_rows;
    const int page_mask = (1 << p.c.page_shift) - 1;
    // A tile's copies are one to a lane: box x of its rows and column half y
    // belong to lane x * kHalves + y, which also holds the box's page.
    constexpr int kHalves = kQuant ? 1 : D / 64;
    const int box = lane / kHalves, half = lane % kHalves;
    uint32_t told = 0;
    auto tell = [&](const Piece &x) -> bool {
      const uint32_t at = told % C::kPieces;
      if (!wait_all(bar(C::kPieceEmpty + at), ((told / C::kPieces) & 1u) ^ 1u)) return false;
      if (lead) {
        pieces[at] = x;
        mbar_arrive(bar(C::kPieceFull + at));
      }
      ++told;
      return true;
    };
    auto load_pages = [&](const Unit &x, int j) -> int32_t {
      const int64_t key = static_cast<int64_t>(j) * kTile + box * box_rows;
      if (box >= boxes || key >= x.s.lk) return -1;
      if (p.chunk_set == kSetFlat) return x.flat_page + j < p.flat_pages ? x.flat_page + j : -1;
      const int32_t page = load_now(p.c.table + static_cast<int64_t>(x.b) * p.c.table_pages +
                                    (key >> p.c.page_shift));
      if (!page_ok(p.c, page)) {
        record_error(p.status, PA_DEVICE_ERR_PAGE);
        return -1;
      }
      return page;
    };
    auto load_kv = [&](const CUtensorMap *tm, int32_t page, int j, int head) -> bool {
      const uint32_t s = slot_loads % kBufs;
      const uint32_t use = slot_loads / kBufs;
      if (!wait_all(bar(kEmpty + s), (use & 1u) ^ 1u)) return false;
      const uint32_t dst = sBuf + s * kBufBytes;
      if (lead) mbar_arrive_expect_tx(bar(kFull + s), kBufBytes);
      const int row = (j * kTile) & page_mask;   // not 0 only where a page spans several tiles
      __syncwarp();   // no byte of a copy is counted before all are announced
      if (box < boxes)
        tma_load_4d(dst + box * box_rows * (kQuant ? D : 128) + half * C::kHalfBytes, tm,
                    bar(kFull + s), half * 64, head, row, page);
      ++slot_loads;
      return true;
    };
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      Unit x;
      open_unit(p, list, n_seqs, u, lane_seq, lane_work, x);
      int4 join_a = make_int4(0, 0, 0, 0), join_b = join_a;   // no item is cut at this unit's end
      ChunkPiece pc;
      while (ok && x.cur.next(x.w, pc)) {
        int32_t pages = load_pages(x, pc.j0);
        const int tok0 = pc.item * x.w.item_tokens;
        Piece piece;
        piece.j0 = pc.j0;
        piece.j1 = pc.j1;
        piece.q0 = x.s.q0;
        piece.tok0 = tok0;
        piece.tokens = min(x.w.item_tokens, x.s.lq - tok0);
        piece.head = pc.head;
        piece.lk = x.s.lk;
        piece.before = x.s.lk - x.s.lq;
        piece.b = x.b;
        piece.part_rows = x.part_rows;
        const int part = x.by_piece ? x.local + pc.head * x.w.items_head + pc.item
                                    : 2 * x.local + (pc.j0 == 0);
        piece.slot = pc.j0 == 0 && pc.j1 == pc.nk ? -1
                                                  : static_cast<int>(x.part0) + part * x.part_rows;
        const int ntq = piece.tokens > tile_tokens ? 2 : 1;
        if (!wait_all(bar(C::kQEmpty), (q_loads & 1u) ^ 1u)) {
          ok = false;
          break;
        }
        if (lead) {
          mbar_arrive_expect_tx(bar(C::kQFull), ntq * (D / 64) * tile_rows * 128);
          for (int t = 0; t < ntq; ++t) {
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              tma_load_4d(sQ + t * C::kTileBytes + hf * C::kHalfBytes, &tm_q, bar(C::kQFull),
                          hf * 64, 0, pc.head, x.s.q0 + tok0 + t * tile_tokens);
          }
        }
        ++q_loads;
        if (!tell(piece)) {
          ok = false;
          break;
        }
        if (pc.j0 == 0 && pc.j1 < pc.nk) {
          // this share begins the item, later ones go on with it: how many
          const int more = x.w.shares_after(x.local, pc.head, pc.item);
          join_a = make_int4(1 + more, piece.slot, x.part_rows, x.by_piece);
          join_b = make_int4(piece.tokens * p.G, x.s.q0 + tok0, pc.head, 0);
        }
        for (int j = pc.j0; j < pc.j1 && ok; ++j) {
          const int32_t next = j + 1 < pc.j1 ? load_pages(x, j + 1) : -1;
          ok = load_kv(&tm_k, pages, j, pc.head);
          if (ok) ok = load_kv(&tm_v, pages, j, pc.head);
          pages = next;
        }
      }
      if (lead && ok && x.w.share > 0) {
        int4 *join = p.chunk_join + 2 * (static_cast<int64_t>(list.cut0[x.at]) + x.local);
        join[0] = join_a;
        join[1] = join_b;
      }
    }
    if (ok) {
      Piece none = {};
      ok = tell(none);
    }
    if (!ok) {
      // give the copies already issued a bounded chance to land
      for (uint32_t s = 0; s < kBufs && s < slot_loads; ++s) {
        const uint32_t n = (slot_loads - s + kBufs - 1) / kBufs;  // loads into s
        drain_wait(bar(kFull + s), (n - 1) & 1u, kDrainLimit);
      }
      if (q_loads) drain_wait(bar(C::kQFull), (q_loads - 1) & 1u, kDrainLimit);
    }
  } else if (warp == 1 || warp == 2) {
    // ================= MMA issuers: warp 1 for tile 0, warp 2 for tile 1 ====
    // Each issuer walks the same pieces and ring slots; it issues its own
    // tile's MMAs in the order S_0 | PV_0 S_1 | PV_1 S_2 ... and frees a slot
    // (or the Q buffer) with one arrival on a two-arrival barrier: a commit
    // once its MMAs reading the slot are done, or a plain arrive where it reads
    // none.  The whole warp runs the issuer, so every operand of an MMA is
    // warp-uniform, and one elected lane issues.
    const int t = warp - 1;
    const bool lead = elect_one();
    uint32_t q_uses = 0, slot_uses = 0, issued = 0, p_waits = 0;
    bool ok = true;
    auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
      const bool w = bounded_wait(b, parity, abort_flag, p.status, kWaitLimit);
      return __all_sync(0xffffffffu, w);
    };
    // next ring slot in consumption order, once its load has landed
    auto wait_slot = [&](uint32_t &s) -> bool {
      s = slot_uses % C::kSlots;
      return wait_all(bar(C::kSlotFull + s), (slot_uses / C::kSlots) & 1u);
    };
    // (descriptors advance by adding the byte offset >> 4 to the start
    // address field; every operand lies below 256 KB, so nothing carries)
    const uint64_t qdesc_one = sdesc_sw128(sQ, 16, 1024);
    const uint64_t qdesc0 = qdesc_one + ((t * C::kTileBytes) >> 4);
    const uint64_t kdesc0 = sdesc_sw128(sRing, 16, 1024);
    const uint64_t vdesc0 = sdesc_sw128(sRing, C::kVLbo, 1024);
    const uint32_t d_s = tmem + C::kColS + t * kTile, d_o = tmem + C::kColO + t * D;
    // S_t = Q_t K^T (both K-major, SBO = 8 rows x 128 B)
    auto issue_s = [&](uint32_t slot, uint64_t qdesc) {
      const uint64_t b0 = kdesc0 + ((slot * C::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kHalfBytes + (kk & 3) * 32) >> 4;
        if (lead) mma_ss(d_s, qdesc + off, b0 + off, C::kIdescS, kk > 0 ? 1u : 0u);
      }
    };
    // O_t += P_t V (P_t is in the first 64 columns of the S buffer)
    auto issue_pv = [&](uint32_t slot, bool fresh) {
      const uint64_t b0 = vdesc0 + ((slot * C::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk) {
        if (lead)
          mma_ts(d_o, d_s + kk * 8, b0 + ((kk * 16 * 128) >> 4), C::kIdescO,
                 (fresh && kk == 0) ? 0u : 1u);
      }
    };
    // The two issuers take turns group by group (S0_0, S1_0, [PV0_0 S0_1],
    // [PV1_0 S1_1], ...); each finishes its waits before taking the turn and
    // commits after passing it on.
    uint32_t turns = 0;
    auto take_turn = [&]() -> bool {
      const uint32_t parity = t == 0 ? ((turns & 1u) ^ 1u) : (turns & 1u);
      return wait_all(bar(C::kTurn + t), parity);
    };
    auto pass_turn = [&]() {
      ++turns;
      if (lead) mbar_arrive(bar(C::kTurn + (1 - t)));
    };
    {
      Piece pc;
      while (ok && next_piece(pc)) {
        const int last_tile = pc.lk > 0 ? (pc.lk - 1) / kTile : 0;   // holds the last key
        if (!wait_all(bar(C::kQFull), q_uses & 1u)) {
          ok = false;
          break;
        }
        ++q_uses;
        if (pc.tokens <= tile_tokens) {
          // One tile of rows: the issuers share its key tiles, tile t of S and O
          // has every second one from t on.  An issuer's PV waits until it has
          // let go of the other's next slots, and comes before its own next S.
          const int n = pc.j1 - pc.j0, mine = (n - t + 1) / 2;
          int done = 0, held = -1;   // S issued; key tile whose PV is still to come
          uint32_t sv = 0;
          auto flush = [&]() -> bool {
            if (held < 0) return true;
            if (!kQuant && held == last_tile) {
              const int valid = pc.lk - held * kTile;
              if (valid < kTile) zero_v_tail<D>(gbase + C::kRingOff + sv * C::kTileBytes, valid, lane);
            }
            if (!wait_all(bar(C::kPReady + t), p_waits & 1u)) return false;
            ++p_waits;
            fence_after_sync();
            issue_pv(sv, held == pc.j0 + t);
            if (lead) {
              mma_commit(bar(C::kSlotEmpty + sv));
              if (done == mine) mma_commit(bar(C::kOFull + t));
            }
            held = -1;
            return true;
          };
          if (mine == 0 && lead) mbar_arrive(bar(C::kQEmpty));
          for (int i = 0; i < n && ok; ++i) {
            uint32_t sk;
            ok = wait_slot(sk);
            if (!ok) break;
            ++slot_uses;
            if ((i & 1) == t) {
              issue_s(sk, qdesc_one);
              issued = 1;
              ++done;
              if (lead) {
                mma_commit(bar(C::kSFull + t));
                mma_commit(bar(C::kSlotEmpty + sk));
                if (done == mine) mma_commit(bar(C::kQEmpty));
              }
              ok = wait_slot(sv);
              ++slot_uses;
              held = pc.j0 + i;
            } else {
              if (lead) mbar_arrive(bar(C::kSlotEmpty + sk));
              ok = wait_slot(sk);
              if (!ok) break;
              ++slot_uses;
              if (lead) mbar_arrive(bar(C::kSlotEmpty + sk));
              ok = flush();
            }
          }
          if (ok) ok = flush();
          continue;
        }
        // release a slot / the Q buffer after this tile's MMAs
        auto release = [&](uint32_t b) {
          if (lead) mma_commit(b);
        };
        // prologue: S of the first key tile
        uint32_t sk;
        if (!wait_slot(sk) || !take_turn()) {
          ok = false;
          break;
        }
        issue_s(sk, qdesc0);
        issued = 1;
        pass_turn();
        if (lead) mma_commit(bar(C::kSFull + t));
        release(bar(C::kSlotEmpty + sk));
        ++slot_uses;
        if (pc.j1 - pc.j0 == 1) release(bar(C::kQEmpty));
        for (int j = pc.j0; j < pc.j1 && ok; ++j) {
          const bool more = j + 1 < pc.j1;
          uint32_t sv, sk2 = 0;
          if (!wait_slot(sv)) {
            ok = false;
            break;
          }
          ++slot_uses;
          // V rows past the sequence's last key: P is 0 there, but 0 * Inf and
          // 0 * NaN are NaN.  Tile 0's issuer issues its PV before tile 1's (the
          // turn order), so it alone clears them.
          // (Widened V tiles come with those rows as zeros.)
          if (!kQuant && t == 0 && j == last_tile) {
            const int valid = pc.lk - j * kTile;
            if (valid < kTile)
              zero_v_tail<D>(gbase + C::kRingOff + sv * C::kTileBytes, valid, lane);
          }
          if (more && !wait_slot(sk2)) {
            ok = false;
            break;
          }
          // the issue turn first (the order is fixed, so holding it early
          // blocks nobody), then P_j written by this tile's softmax
          if (!take_turn()) {
            ok = false;
            break;
          }
          if (!wait_all(bar(C::kPReady + t), p_waits & 1u)) {
            ok = false;
            break;
          }
          ++p_waits;
          fence_after_sync();
          // PV_j, then S_{j+1} (after the PV that reads P from the S buffer)
          issue_pv(sv, j == pc.j0);
          if (more) issue_s(sk2, qdesc0);
          pass_turn();
          if (lead) mma_commit(more ? bar(C::kSFull + t) : bar(C::kOFull + t));
          release(bar(C::kSlotEmpty + sv));
          if (more) {
            release(bar(C::kSlotEmpty + sk2));
            ++slot_uses;
            if (j + 2 == pc.j1) release(bar(C::kQEmpty));
          }
        }
      }
    }
    // every MMA this thread issued has finished before TMEM is released
    if (issued) {
      if (lead) mma_commit(bar(C::kFinal + t));
      drain_wait(bar(C::kFinal + t), 0, kWaitLimit);
    }
    __syncwarp();
  } else if (kQuant && warp >= C::kWidenWarp) {
    // ================= 8-bit rows to bf16 =================
    // Eight warps, 16 rows of a tile each: a lane takes 16 bytes of a row at a
    // time, widens them with the row's scale (lane x holds that of K's row x,
    // lane 16 + x of V's) and stores two 16-byte chunks of the swizzled bf16 tile.  Lanes of the second
    // column half store their odd chunk first, so the eight lanes of a row
    // never meet in a bank.
    if constexpr (kQuant) {
      constexpr int kRowLanes = D / 16, kPass = 32 / kRowLanes;   // rows of a warp-wide load
      constexpr int kRows = kTile / C::kWideners, kPasses = kRows / kPass;
      static_assert(kRows == 16, "a lane holds one exponent");
      const int w = warp - C::kWidenWarp;
      const int sub = lane / kRowLanes, col = lane % kRowLanes;   // 16 columns from col * 16
      const int hf = col >> 2, chunk = (col & 3) * 2;
      uint32_t n = 0;
      bool ok = true;
      auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
        const bool x = bounded_wait(b, parity, abort_flag, p.status, kWaitLimit);
        return __all_sync(0xffffffffu, x);
      };
      {
        Piece pc;
        while (ok && next_piece(pc)) {
          const int32_t *table = p.c.table + static_cast<int64_t>(pc.b) * p.c.table_pages;
          // this lane's row of key tile j: its page, then its exponent byte
          const int my_row = w * kRows + (lane & 15);
          const uint8_t *exps = lane < 16 ? p.c.k_exp : p.c.v_exp;
          auto load_page = [&](int j) -> int32_t {
            const int64_t key = static_cast<int64_t>(j) * kTile + my_row;
            return j < pc.j1 && key < pc.lk ? load_now(table + (key >> p.c.page_shift)) : -1;
          };
          auto load_exp = [&](int j, int32_t page) -> int {
            if (!page_ok(p.c, page)) return -1;   // no such row: scale 0
            const int row = (j * kTile + my_row) & ((1 << p.c.page_shift) - 1);
            return load_now(exps + exp_offset(p.c, page, row, pc.head));
          };
          int32_t page = load_page(pc.j0);
          int byte = load_exp(pc.j0, page);
          page = load_page(pc.j0 + 1);
          for (int j = pc.j0; j < pc.j1 && ok; ++j) {
            const int byte_next = load_exp(j + 1, page);
            page = load_page(j + 2);
            const uint32_t scale = byte < 0 ? 0u : widen_scale(byte) * 0x10001u;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, ++n) {
              const uint32_t r = n % C::kRaws, s = n % C::kSlots;
              if (!wait_all(bar(C::kRawFull + r), (n / C::kRaws) & 1u)) {
                ok = false;
                break;
              }
              // all loads in flight before the first store
              const uint8_t *raw = gbase + C::kRawOff + r * C::kRawBytes + w * kRows * D + lane * 16;
              uint4 y[kPasses];
              uint32_t sc[kPasses];
#pragma unroll
              for (int i = 0; i < kPasses; ++i) y[i] = *reinterpret_cast<const uint4 *>(raw + i * 512);
#pragma unroll
              for (int i = 0; i < kPasses; ++i)
                sc[i] = __shfl_sync(0xffffffffu, scale, kv * 16 + i * kPass + sub);
              if (!wait_all(bar(C::kSlotEmpty + s), ((n / C::kSlots) & 1u) ^ 1u)) {
                ok = false;
                break;
              }
              if (lane == 0) mbar_arrive(bar(C::kRawEmpty + r));   // every lane has its bytes
              uint8_t *tile = gbase + C::kRingOff + s * C::kTileBytes + hf * C::kHalfBytes;
              auto store_rows = [&](auto &&widen) {
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                  const int row = i * kPass + sub;
                  uint4 a, c;
                  a.x = widen(y[i].x, sc[i], 0x4140);
                  a.y = widen(y[i].x, sc[i], 0x4342);
                  a.z = widen(y[i].y, sc[i], 0x4140);
                  a.w = widen(y[i].y, sc[i], 0x4342);
                  c.x = widen(y[i].z, sc[i], 0x4140);
                  c.y = widen(y[i].z, sc[i], 0x4342);
                  c.z = widen(y[i].w, sc[i], 0x4140);
                  c.w = widen(y[i].w, sc[i], 0x4342);
                  uint8_t *dst = tile + (w * kRows + row) * 128;
                  const int even = ((chunk ^ (row & 7)) * 16), odd = (((chunk + 1) ^ (row & 7)) * 16);
                  *reinterpret_cast<uint4 *>(dst + (hf ? odd : even)) = hf ? c : a;
                  *reinterpret_cast<uint4 *>(dst + (hf ? even : odd)) = hf ? a : c;
                }
              };
              uint32_t nan = 0u;
#pragma unroll
              for (int i = 0; i < kPasses; ++i) nan |= holds_nan(y[i]);
              if (__any_sync(0xffffffffu, nan))
                store_rows(widen_pair_nan);
              else
                store_rows(widen_pair);
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::kSlotFull + s));
            }
            byte = byte_next;
          }
        }
      }
    }
  } else if (warp >= C::kSoftmaxWarp) {
    // ================= softmax / correction / epilogue =================
    // four warps to a tile; TMEM lane quadrant = warp % 4
    const int t = (warp - C::kSoftmaxWarp) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int row_token = row / p.G;             // token of the row within its tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t colS = C::kColS + t * kTile;
    const uint32_t colO = C::kColO + t * D;
    const float sl2 = p.scale_log2;
    const bool pos_scale = sl2 > 0.f;
    const float mul = pos_scale ? sl2 : 1.f;
    uint32_t s_waits = 0, o_waits = 0, shares = 0;
    bool ok = true;
    {
      // (a piece is kept where it was told until its rows are stored: its fields
      // would cost registers that the scores need)
      while (ok) {
        const uint32_t told_at = pieces_read % C::kPieces;
        ok = bounded_wait(bar(C::kPieceFull + told_at), (pieces_read / C::kPieces) & 1u, abort_flag,
                          p.status, kWaitLimit);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++pieces_read;
        const volatile Piece &pc = pieces[told_at];
        const int j1 = pc.j1;
        if (j1 == 0) break;
        // one tile of rows: tiles 0 and 1 are its even and its odd key tiles
        const int j_step = pc.tokens <= tile_tokens ? 2 : 1;
        // keys that this row sees
        int lim = pc.lk;
        if (p.causal)
          lim = min(lim, pc.before + pc.tok0 + 1 + row_token + (j_step == 2 ? 0 : t * tile_tokens));
        float m = -INFINITY, l = 0.f;
        for (int j = pc.j0 + (j_step == 2 ? t : 0); j < j1; j += j_step) {
          ok = bounded_wait(bar(C::kSFull + t), s_waits & 1u, abort_flag, p.status, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          ++s_waits;
          fence_after_sync();
          // The row's maximum, then its weights, kCols columns at a time: read
          // once where a thread holds all 128, else twice.
          const int seen = lim - j * kTile;
          const bool masked = __any_sync(0xffffffffu, seen < kTile);
          constexpr int kPairs = C::kCols / 2;
          float2 sc[kPairs];
          auto read_part = [&](int h) {
            uint32_t r[C::kCols];
#pragma unroll
            for (int c = 0; c < C::kCols; c += 32)
              tmem_ld32(lane_base + colS + h * C::kCols + c,
                        *reinterpret_cast<uint32_t(*)[32]>(&r[c]));
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kPairs; ++c)
              sc[c] = make_float2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
            // with a positive scale the scale is folded into the exponent's
            // FFMA, otherwise the scores are scaled first
            if (!pos_scale) {
              const float2 s2 = make_float2(sl2, sl2);
#pragma unroll
              for (int c = 0; c < kPairs; ++c) sc[c] = __fmul2_rn(sc[c], s2);
            }
            if (masked) {
#pragma unroll
              for (int c = 0; c < kPairs; ++c) {
                if (h * C::kCols + 2 * c >= seen) sc[c].x = -INFINITY;
                if (h * C::kCols + 2 * c + 1 >= seen) sc[c].y = -INFINITY;
              }
            }
          };
          // row maximum: four chains of 3-input max, fixed combine
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int h = 0; h < kTile / C::kCols; ++h) {
            read_part(h);
#pragma unroll
            for (int c = 0; c < kPairs; ++c) mx4[c & 3] = fmax3(mx4[c & 3], sc[c].x, sc[c].y);
          }
          // (Rounding steps are written out wherever the compiler could choose: the kernels
          // over bf16 and over 8-bit rows give the same bits.)
          const float mx = __fmul_rn(fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]), mul);
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m + kRescaleThreshold) {   // from -inf: any finite score
            alpha = ex2(m - mx);
            m = mx;
            rescale = l != 0.f;   // without weights so far O is zero, or nothing yet
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 mul2 = make_float2(mul, mul), negm2 = make_float2(-ref, -ref);
          float2 sum4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum4[e] = make_float2(0.f, 0.f);
          // P over the first 64 columns of the S buffer: a part's weights take
          // columns that have been read already
#pragma unroll 1
          for (int h = 0; h < kTile / C::kCols; ++h) {
            if (C::kCols < kTile) read_part(h);
#pragma unroll
            for (int c0 = 0; c0 < kPairs; c0 += 16) {
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float2 tt = __ffma2_rn(sc[c0 + c], mul2, negm2);
                const float2 pp = make_float2(ex2(tt.x), ex2(tt.y));
                sum4[c & 3] = __fadd2_rn(sum4[c & 3], pp);
                pk[c] = pack_bf16x2(pp.x, pp.y);
              }
              tmem_st16(lane_base + colS + h * kPairs + c0, pk);
            }
          }
          const float2 s4 = __fadd2_rn(__fadd2_rn(sum4[0], sum4[1]), __fadd2_rn(sum4[2], sum4[3]));
          l = __fmaf_rn(l, alpha, __fadd_rn(s4.x, s4.y));
          // S_j complete implies the PV issued before it is complete: O is
          // current and can be rescaled in place
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(lane_base + colO + c * 32, r);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st32(lane_base + colO + c * 32, r);
            }
          }
          tmem_wait_st();
          fence_before_sync();
          mbar_arrive(bar(C::kPReady + t));
        }
        if (!ok) break;
        // epilogue: wait for this tile's last PV, then store the valid rows
        const bool shared = j_step == 2, two = shared && j1 - pc.j0 > 1;
        const int row0 = shared ? 0 : t * tile_rows;   // of this tile in the item
        const int token = row_token + (shared ? 0 : t * tile_tokens);
        const bool store = row < tile_rows && token < pc.tokens;
        if (t == 0 || !shared || two) {
          ok = bounded_wait(bar(C::kOFull + t), o_waits & 1u, abort_flag, p.status, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          ++o_waits;
          fence_after_sync();
        }
        // O is f0 O_t (+ f1 O_1 where the tiles share the rows, each of them then
        // storing half of the columns)
        float f0 = 1.f, f1 = 0.f;
        if (shared) {
          float2 *stat = reinterpret_cast<float2 *>(gbase + C::kStatOff);
          stat[t * kTile + row] = make_float2(m, l);
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kBothDone));
          ok = bounded_wait(bar(C::kBothDone), shares & 1u, abort_flag, p.status, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          fence_after_sync();
          const float2 a = stat[row], c = stat[kTile + row];
          m = fmaxf(a.x, c.x);
          const float ref = m == -INFINITY ? 0.f : m;
          f0 = ex2(a.x - ref);
          f1 = ex2(c.x - ref);
          l = __fmaf_rn(f0, a.y, __fmul_rn(f1, c.y));
        }
        const uint32_t src0 = lane_base + (shared ? C::kColO : colO), src1 = lane_base + C::kColO + D;
        const int c_first = shared ? t * (D / 64) : 0, c_end = shared ? c_first + D / 64 : D / 32;
        // a row that sees no key: O and l are 0 (or NaN, if a score was)
        const float inv = m == -INFINITY ? 0.f : 1.f / l;
        const int slot = pc.slot, part_rows = pc.part_rows;
        __nv_bfloat16 *dst = p.out + (static_cast<int64_t>(pc.q0 + pc.tok0 + token) * p.Hq +
                                      pc.head * p.G + (row - row_token * p.G)) * D;
        // a part lies in the workspace column by column, four at a time, so
        // that a warp's stores are runs of 512 bytes
        float4 *part = reinterpret_cast<float4 *>(p.chunk_o + static_cast<int64_t>(slot) * D) +
                       row0 + row;
#pragma unroll 1
        for (int c = c_first; c < c_end; ++c) {
          uint32_t r[32];
          tmem_ld32(src0 + c * 32, r);
          if (two) {
            uint32_t r1[32];
            tmem_ld32(src1 + c * 32, r1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              r[e] = __float_as_uint(
                  __fmaf_rn(f0, __uint_as_float(r[e]), __fmul_rn(f1, __uint_as_float(r1[e]))));
          } else {
            tmem_wait_ld();
            if (shared) {   // f0 is 1, or 0 for a row that sees no key (its O is 0, or NaN)
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(f0 * __uint_as_float(r[e]));
            }
          }
          if (!store) continue;
          if (slot < 0) {
            uint4 *d4 = reinterpret_cast<uint4 *>(dst + c * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(r[8 * v + 2 * e]) * inv,
                                   __uint_as_float(r[8 * v + 2 * e + 1]) * inv);
              d4[v] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              part[static_cast<int64_t>(c * 8 + v) * part_rows] =
                  make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                              __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
          }
        }
        if (slot >= 0 && store && (!shared || t == 0))
          p.chunk_ml[static_cast<int64_t>(slot) + row0 + row] = make_float2(m, l);
        if (shared) {
          // neither tile's O is written again before both have been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kBothRead));
          ok = bounded_wait(bar(C::kBothRead), shares & 1u, abort_flag, p.status, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          ++shares;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kPieceEmpty + told_at));
      }
    }
  }

  // ---- teardown -------------------------------------------------------------
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  // every way out waits: this kernel's end is the end of those launched before it
  griddep_wait();
}

// q as (D, G, Hkv, tokens): a box is 64 columns of the group's heads of the
// tokens of one tile; rows of a page as (D, Hkv, row, page): a box is 64
// columns of one head's rows.  128-byte swizzle.
// Rows of an 8-bit page come whole, unswizzled.
bool make_map(CUtensorMap *map, bool bytes, const void *ptr, const cuuint64_t (&dims)[4],
              const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kQuant>
cudaError_t launch(const PagedAttnParams &p, int num_sms, bool behind, cudaStream_t stream) {
  using C = Cfg<D, kQuant>;
  CUtensorMap mq, mk, mv;
  const cuuint64_t G = p.G, H = p.c.Hkv, d = D;
  const cuuint64_t qdims[4] = {d, G, H, static_cast<cuuint64_t>(p.total_q)};
  const cuuint64_t qstr[3] = {d * 2, G * d * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
  const cuuint32_t qbox[4] = {64, static_cast<cuuint32_t>(G), 1,
                              static_cast<cuuint32_t>(kTile / p.G)};
  const cuuint64_t cdims[4] = {d, H, cuuint64_t{1} << p.c.page_shift,
                               static_cast<cuuint64_t>(p.c.num_pages)};
  const cuuint64_t es = kQuant ? 1 : 2;
  const cuuint64_t cstr[3] = {d * es, H * d * es, static_cast<cuuint64_t>(p.c.page_stride) * es};
  const int page = 1 << p.c.page_shift;
  const cuuint32_t cbox[4] = {kQuant ? D : 64, 1, static_cast<cuuint32_t>(page < kTile ? page : kTile), 1};
  if (!make_map(&mq, false, p.q, qdims, qstr, qbox) ||
      !make_map(&mk, kQuant, p.c.k, cdims, cstr, cbox) ||
      !make_map(&mv, kQuant, p.c.v, cdims, cstr, cbox))
    return cudaErrorInvalidValue;
  static unsigned long long configured = 0;
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(paged_chunk_kernel<D, kQuant>),
                                C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_chunk_kernel<D, kQuant>, mq, mk, mv, p);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnParams &p, bool quant, int num_sms,
                               cudaStream_t stream) {
  if (!quant)
    return p.c.D == 128 ? launch<128, false>(p, num_sms, false, stream)
                        : launch<64, false>(p, num_sms, false, stream);
  PagedAttnParams rest = p;
  if (p.flat_pages > 0) {
    // long sequences over rows widened ahead, then the others, each in its own
    // half of the cuts and behind the kernel before it
    cudaError_t e = launch_paged_widen(p, num_sms, stream);
    if (e != cudaSuccess) return e;
    PagedAttnParams flat = p;
    flat.chunk_set = kSetFlat;
    flat.c.k = p.flat_k;
    flat.c.v = p.flat_v;
    flat.c.page_shift = 7;
    flat.c.page_stride = static_cast<int64_t>(kTile) * p.c.Hkv * p.c.D;
    flat.c.num_pages = p.flat_pages;
    e = p.c.D == 128 ? launch<128, false>(flat, num_sms, true, stream)
                     : launch<64, false>(flat, num_sms, true, stream);
    if (e != cudaSuccess) return e;
    rest.chunk_set = kSetRest;
    rest.chunk_row0 = p.chunk_row0_rest;
    rest.chunk_cut0 = p.chunk_cut0_rest;
  }
  return p.c.D == 128 ? launch<128, true>(rest, num_sms, p.flat_pages > 0, stream)
                      : launch<64, true>(rest, num_sms, p.flat_pages > 0, stream);
}

}  // namespace pa
