// Work items of the packed attention kernels (head dim 64 on single CTAs, head
// dim 128 on CTA pairs): their parameters, the decode of item i of the work list
// into rows and keys, the key-tile order, and the ring through which one warp
// tells the others of the items.
//
// Query head h reads K/V head h / G.  The rows of a 128-row tile are the group's
// heads of 128 / G tokens (row = token * G + head of the group; G = 1: 128
// tokens), so few tokens fill a tile, and causal order cuts all of its rows at
// nearly the same key.  An item is two tiles of one (sequence, K/V head); its
// keys come in kVarlenTile-key tiles in the same order on both kernels, so a
// sequence's rows come out the same whatever the batch around it.
// causal: query i of a sequence sees key j iff j <= lk - lq + i.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "sched.cuh"
#include "tc_ptx.cuh"

namespace pa {

constexpr int kVarlenTile = 128;       // keys of a K/V tile, rows of a Q tile
constexpr int kVarlenItemRows = 256;   // query rows of a work item
constexpr int kItemSlots = 8;          // items told ahead

struct VarlenParams {
  __nv_bfloat16 *out;
  const int32_t *cu_q, *cu_k;
  int batch, H, total_q, total_k, max_q, max_k;
  float scale_log2;
  int32_t *status;
  int G, tokens, causal;   // query heads per K/V head, tokens of a tile, causal order
  int box_tokens;          // of 32 rows of a tile, or 0 where they are no box of out
};

inline VarlenParams varlen_params(const VarlenArgs &a) {
  VarlenParams p;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.batch = a.batch;
  p.H = a.H;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.max_q = a.max_q;
  p.max_k = a.max_k;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  p.G = a.H / a.Hkv;
  p.tokens = kVarlenTile / p.G;
  p.causal = a.causal;
  p.box_tokens = 32 % p.G == 0 ? 32 / p.G : p.G % 32 == 0 ? 1 : 0;
  return p;
}

struct ItemInfo {
  int q_row0;   // global row of the item's first token
  int tokens;   // valid tokens in the item (1..2 * VarlenParams::tokens)
  int k0;       // global row of the sequence's first key
  int lk;       // keys of the sequence
  int nk;       // key tiles
  int head;     // of K and V
  int rot;      // first key tile visited
  int seen;     // token r of the item sees the keys below min(lk, seen + r + 1)
};
static_assert(sizeof(ItemInfo) == 32, "two 16-byte pieces");

// Key tile visited j-th.  Items start at another key tile each (their place in
// the sequence) and wrap around, so the workers of a wave, which hold
// consecutive query blocks of one head, read different K/V tiles at any
// moment.  The order depends only on the sequence's own lengths and the
// item's position in it, so a sequence's result is the same in any batch.
__device__ __forceinline__ int key_tile(const ItemInfo &it, int j) {
  const int kt = it.rot + j;
  return kt >= it.nk ? kt - it.nk : kt;
}

// Item i (0 <= i < prefix[batch]) of the work list; a sequence whose
// boundaries are invalid reads as empty (the list build records why).
__device__ __forceinline__ ItemInfo item_info(const VarlenParams &p, const int32_t *order,
                                              const int32_t *prefix, int i) {
  const int heads = p.H / p.G, item = 2 * p.tokens;
  const WorkItem w = p.causal ? sched_level_item(order, prefix, p.cu_q, p.batch, heads, item, i)
                              : sched_item(order, prefix, p.batch, heads, i);
  int err;
  const SeqBounds sb = seq_bounds(p.cu_q, p.cu_k, w.seq, p.total_q, p.total_k, p.max_q,
                                  p.max_k, err);
  ItemInfo it;
  it.q_row0 = sb.q0 + w.tile * item;
  it.tokens = min(item, sb.lq - w.tile * item);
  it.k0 = sb.k0;
  it.lk = sb.lk;
  it.head = w.head;
  it.seen = sb.lk;
  int keys = sb.lk;   // that any row of the item sees
  if (p.causal) {
    it.seen = sb.lk - sb.lq + w.tile * item;
    keys = max(0, it.seen + it.tokens);   // (at most lk)
  }
  it.nk = (keys + kVarlenTile - 1) / kVarlenTile;
  // A causal item takes its tiles in order: each row that sees any key sees
  // the first one, so its maximum is finite before a tile that hides all.
  it.rot = it.nk > 0 && !p.causal ? w.tile * item / kVarlenItemRows % it.nk : 0;
  return it;
}

// The work list of a kernel, in shared memory (see sched_build).
__device__ __forceinline__ void item_list(const VarlenParams &p, int32_t *order, int32_t *prefix,
                                          int32_t *tmp_lq, int32_t *tmp_lk, bool report) {
  sched_build(order, prefix, tmp_lq, tmp_lk, p.cu_q, p.cu_k, p.batch, p.H / p.G, 2 * p.tokens,
              p.total_q, p.total_k, p.max_q, p.max_k, p.status, report, p.causal != 0);
}

// The worker's n-th item, of `workers`: round robin; in a causal list, whose
// items grow cheaper (of sequences without keys before their queries), every second
// round backwards, which evens out what a
// round's first worker has more than its last.
__device__ __forceinline__ int item_at(const VarlenParams &p, int n, int worker, int workers) {
  return n * workers + (p.causal && (n & 1) ? workers - 1 - worker : worker);
}

// Added to a row's maximum before a causal call's weights are taken relative to it.
// A maximum that grows by more than the rescaling threshold costs a wait and a
// pass over O; with the weights 2^24 smaller it has 2^24 further to go.  They have
// fp32's and bf16's range down to 2^-126, but their products with V reach the end of
// fp32's subnormal numbers 2^24 earlier, so O is off by some 2^-124 in absolute terms
// (V of 2^-112: as exact as any; of 2^-116: 5 % of sum w |v|).  16k keys
// whose sizes differ as a projection's do, 32 heads on 8 of 128: 1345 us without,
// 1130 with it.  (A call without causal order keeps the weights that it has always
// had, bit for bit.)
constexpr float kWeightHead = 24.f;

// A warp's 32 rows of 128 bytes (64 columns), a row to a lane in `words`, out to
// where `dst` of the row's lane says (nullptr: not stored), through 4 KB of shared
// memory: eight lanes write a row, four rows an instruction, where rows stored by
// their own lanes are 32 separate pieces of 16 bytes (head dim 128: the end of an item
// of 64 KB took 3300 cycles so, and 1560 this way; a bulk copy to a row 382 -> 400 us
// on 24 prompts of 90-2700 tokens, 32 heads on 8).  Pieces of a row are permuted
// against bank conflicts, as the 128-byte swizzle has them.
__device__ __forceinline__ void store_rows(uint8_t *buf, const uint32_t (&words)[32],
                                           __nv_bfloat16 *dst) {
  const int lane = threadIdx.x & 31, piece = lane & 7;
#pragma unroll
  for (int v = 0; v < 8; ++v)
    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((v ^ piece) << 4)) =
        make_uint4(words[4 * v], words[4 * v + 1], words[4 * v + 2], words[4 * v + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = i * 4 + (lane >> 3);
    uint4 *to = reinterpret_cast<uint4 *>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
    const uint4 x =
        *reinterpret_cast<const uint4 *>(buf + row * 128 + ((piece ^ (row & 7)) << 4));
    if (to) to[piece] = x;
  }
  __syncwarp();   // the buffer is free again
}

// The same for `token` and `head` of the row's lane (token < 0: not stored), head dim 64.
// Where all 32 rows are stored and are a box of out (whole groups, or
// part of one), one copy takes them, and nobody waits for it (before the kernel ends,
// lane 0 waits for the copies to be written).  The same 24 prompts: 280
// -> 258 us, 64 of 300 tokens 83 -> 70, 16k 1015 -> 1010.  With head dim 128, whose
// key loop has no register to spare, long sequences lost what short ones won (16k
// 1113 -> 1129 us, the 24 prompts 397 -> 382).
__device__ __forceinline__ void send_rows(uint8_t *buf, const uint32_t (&words)[32],
                                          const VarlenParams &p, const CUtensorMap *map, int head,
                                          int token) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) tc::bulk_wait_read();   // the copy before has read the buffer
  __syncwarp();
  if (p.box_tokens > 0 && __all_sync(0xffffffffu, token >= 0)) {
    const int piece = lane & 7;
#pragma unroll
    for (int v = 0; v < 8; ++v)
      *reinterpret_cast<uint4 *>(buf + lane * 128 + ((v ^ piece) << 4)) =
          make_uint4(words[4 * v], words[4 * v + 1], words[4 * v + 2], words[4 * v + 3]);
    tc::fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      tc::tma_store_3d(map, tc::smem_u32(buf), 0, head, token);
      tc::bulk_commit();
    }
  } else {
    store_rows(buf, words,
               token < 0 ? nullptr
                         : p.out + (static_cast<int64_t>(token) * p.H + head) * 64);
  }
}

// The ring of items.  Finding an item takes a search and a chain of loads, some
// thousand cycles, so a warp of its own does it ahead of the others; they read
// what it found.  Full and empty barriers lie one after the other at `full`
// and `empty` (shared-memory addresses); an empty one takes an arrival from
// every warp that reads.  The ring ends with an item of nk < 0.
struct ItemRing {
  ItemInfo *items;   // [kItemSlots]
  uint32_t full, empty;
};

// Whole warp: all items of this worker with keys into the ring.  The rows of
// items without keys are zeroed here; `rank` of `ranks` CTAs that share the
// items, each with the rows of its own tiles.
__device__ __forceinline__ void tell_items(const VarlenParams &p, const int32_t *order,
                                           const int32_t *prefix, int worker, int workers,
                                           const ItemRing &ring, int D, int rank, int ranks,
                                           volatile int32_t *abort_flag, long long limit) {
  const int lane = threadIdx.x & 31, n_items = prefix[p.batch];
  uint32_t told = 0;
  bool more = true;
  for (int n = 0; more; ++n) {
    const int i = item_at(p, n, worker, workers);
    more = i < n_items;
    ItemInfo it = {};
    it.nk = -1;
    if (more) it = item_info(p, order, prefix, i);
    if (it.nk == 0) {
      const int t0 = ranks == 2 ? rank * p.tokens : 0;
      const int t1 = ranks == 2 ? min(it.tokens, t0 + p.tokens) : it.tokens;
      const int vecs = p.G * D / 8;   // of a token's heads
      for (int c = lane; c < (t1 - t0) * vecs; c += 32) {
        const int t = c / vecs;
        reinterpret_cast<uint4 *>(
            p.out + (static_cast<int64_t>(it.q_row0 + t0 + t) * p.H + it.head * p.G) * D)[c - t * vecs] =
            make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const uint32_t s = told % kItemSlots;
    const bool ok = tc::bounded_wait(ring.empty + 8u * s, ((told / kItemSlots) & 1u) ^ 1u, abort_flag,
                                     p.status, limit);
    if (!__all_sync(0xffffffffu, ok)) return;
    if (lane == 0) {
      ring.items[s] = it;
      tc::mbar_arrive(ring.full + 8u * s);
    }
    __syncwarp();
    ++told;
  }
}

// A warp's place in the ring.  next(): the item after, false where the wait for
// it ran out.  last: this is the warp's last reading of its items.
struct ItemReader {
  uint32_t n;
  __device__ __forceinline__ bool next(const ItemRing &ring, ItemInfo &it, bool last,
                                       volatile int32_t *abort_flag, int32_t *status,
                                       long long limit) {
    const uint32_t s = n % kItemSlots;
    bool ok = tc::bounded_wait(ring.full + 8u * s, (n / kItemSlots) & 1u, abort_flag, status, limit);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const volatile int4 *src = reinterpret_cast<const volatile int4 *>(ring.items + s);
    int4 a, b;
    a.x = src[0].x; a.y = src[0].y; a.z = src[0].z; a.w = src[0].w;
    b.x = src[1].x; b.y = src[1].y; b.z = src[1].z; b.w = src[1].w;
    it = ItemInfo{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __syncwarp();
    if (last && (threadIdx.x & 31) == 0) tc::mbar_arrive(ring.empty + 8u * s);
    ++n;
    return true;
  }
};

}  // namespace pa
