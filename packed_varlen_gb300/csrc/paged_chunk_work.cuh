// Work of the tiled paged attention kernel (paged_chunk.cu): how a sequence's
// queries and keys are cut into items, and items into units.
//
// An item is up to 2 * tokens_tile queries of one K/V head with all the query
// heads of its group (two 128-row tiles) against the keys they see, in key
// tiles of 128.  In causal order later items see more keys.  A unit is what
// one CTA takes at a time:
//  - whole items, heaviest first, where a sequence has many of them or few
//    keys;
//  - else an equal share of the sequence's key tiles, items laid end to end
//    (heads in order, then tiles): a share starts and ends in the middle of
//    an item, at most two of its pieces are parts of items, and those go
//    through the workspace.
// The choice looks at the sequence alone, as if it had the GPU (152 CTAs) to
// itself, so its bits do not depend on the batch.
#pragma once

#include <stdint.h>

namespace pa {

constexpr int kChunkTile = 128;      // rows of a query tile, keys of a key tile
constexpr int kChunkShares = 152;    // shares of a lone sequence
constexpr int kChunkMinShare = 6;    // key tiles of the smallest share
constexpr int kChunkManyItems = 6 * kChunkShares;

// sum of floor((a i + b) / m) for i in [0, n), by the Euclidean descent on (a, m)
__host__ __device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const int64_t x = m;
    m = a;
    a = x;
  }
  return sum;
}

struct ChunkWork {
  int lq, lk, causal, item_tokens, items_head;   // items of one K/V head
  int nk_last;                                   // key tiles of the last (heaviest) item
  int64_t head_tiles;                            // key tiles of all items of a head
  int64_t share;                                 // key tiles of a share; 0: whole items
  int units;

  // Key tiles of item i: at least one, so that rows that see nothing are written too.
  __host__ __device__ int tiles_of(int i) const {
    int64_t keys = lk;
    if (causal) {
      const int64_t last = static_cast<int64_t>(lk) - lq + static_cast<int64_t>(i + 1) * item_tokens;
      keys = last < keys ? last : keys;
    }
    return keys <= kChunkTile ? 1 : static_cast<int>((keys + kChunkTile - 1) / kChunkTile);
  }
  // Key tiles of items [0, i) of a head.
  __host__ __device__ int64_t tiles_before(int i) const {
    if (!causal) return static_cast<int64_t>(i) * nk_last;
    if (i <= 0) return 0;
    if (i >= items_head) return tiles_before(items_head - 1) + nk_last;
    const int64_t first = static_cast<int64_t>(lk) - lq;     // keys before the chunk
    int64_t blind = first < 0 ? -first / item_tokens : 0;    // items that see no key count one
    if (blind > i) blind = i;
    return blind + floor_sum(i - blind, kChunkTile, item_tokens,
                             first + (blind + 1) * item_tokens + kChunkTile - 1);
  }
  // Item that holds key tile `pos` of a head.
  __host__ __device__ int item_at(int64_t pos) const {
    if (!causal) return static_cast<int>(pos / nk_last);
    int lo = 0, hi = items_head;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (tiles_before(mid) <= pos) lo = mid; else hi = mid;
    }
    return lo;
  }
};

__host__ __device__ inline ChunkWork chunk_work(int lq, int lk, int causal, int G, int Hkv) {
  ChunkWork w;
  w.lq = lq;
  w.lk = lk;
  w.causal = causal;
  w.item_tokens = 2 * (kChunkTile / G);
  w.items_head = static_cast<int>((static_cast<int64_t>(lq) + w.item_tokens - 1) / w.item_tokens);
  w.nk_last = w.tiles_of(w.items_head - 1);
  w.head_tiles = w.tiles_before(w.items_head);
  const int64_t items = static_cast<int64_t>(w.items_head) * Hkv;
  const int64_t all = w.head_tiles * Hkv;
  int64_t share = (all + kChunkShares - 1) / kChunkShares;
  if (share < kChunkMinShare) share = kChunkMinShare;
  if (items >= kChunkManyItems || w.nk_last <= kChunkMinShare + kChunkMinShare / 2) {
    w.share = 0;
    w.units = static_cast<int>(items);
  } else {
    w.share = share;
    w.units = static_cast<int>((all + share - 1) / share);
  }
  return w;
}

// Rows that a part of an item leaves in the workspace.
__host__ __device__ inline int chunk_part_rows(int lq, int G) {
  const int tokens = 2 * (kChunkTile / G);
  return (lq < tokens ? lq : tokens) * G;
}

// A run of key tiles [j0, j1) of one item.
struct ChunkPiece {
  int head, item, j0, j1, nk;
};

// Walks the pieces of unit `u` of a sequence.
struct ChunkCursor {
  int64_t left;    // key tiles of the unit still to come
  int head, item, j;

  __host__ __device__ void start(const ChunkWork &w, int u, int Hkv) {
    if (w.share == 0) {   // heaviest items first, the heads side by side
      const int i = u / Hkv;
      head = u - i * Hkv;
      item = w.items_head - 1 - i;
      j = 0;
      left = w.tiles_of(item);
    } else {
      const int64_t pos = u * w.share, all = w.head_tiles * Hkv;
      left = all - pos < w.share ? all - pos : w.share;
      head = static_cast<int>(pos / w.head_tiles);
      const int64_t in_head = pos - head * w.head_tiles;
      item = w.item_at(in_head);
      j = static_cast<int>(in_head - w.tiles_before(item));
    }
  }
  __host__ __device__ bool next(const ChunkWork &w, ChunkPiece &p) {
    if (left <= 0) return false;
    p.head = head;
    p.item = item;
    p.nk = w.tiles_of(item);
    p.j0 = j;
    p.j1 = left < p.nk - j ? j + static_cast<int>(left) : p.nk;
    left -= p.j1 - p.j0;
    j = 0;
    if (++item == w.items_head) {
      item = 0;
      ++head;
    }
    return true;
  }
};

}  // namespace pa
