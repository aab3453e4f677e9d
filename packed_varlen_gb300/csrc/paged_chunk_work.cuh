// Work of the tiled paged attention kernel (paged_chunk.cu): how a sequence's
// queries and keys are cut into items, and items into units.
//
// An item is up to 2 * tokens_tile queries of one K/V head with all the query
// heads of its group (two 128-row tiles) against the keys they see, in key
// tiles of 128.  In causal order later items see more keys.  A unit is what
// one CTA takes at a time:
//  - whole items, heaviest first, where a sequence has many of them or few
//    keys;
//  - else an equal share of the sequence's keys, items laid end to end (heads
//    in order, then tiles): a share starts and ends in the middle of an item,
//    at most two of its pieces are parts of items, and those go through the
//    workspace.  Shares are cut in keys rather than in key tiles, which keeps
//    the sum over the items before a place a quadratic, and rounded down to a
//    tile where they meet an item (at most one tile in six or more).
// Smallest share, 6 / 10 / 12 / 16 key tiles, GPU time: 16 tokens of 32 sequences over
// 10-12k keys 372 / 342 / 336 / 334 us, of one 28 / 30 / 31 / 37; a mixed step 93 / 93 /
// 81 / 83; cross attention to 700-1500 states 48 / 42 / 42 / 42; two 8-bit chunks 125 /
// 125 / 124 / 124; a long chunk the same.  10 was taken with a set-up that cost more; 12
// would take 12 us off the mixed step for one off the lone sequence, and other bits.
// The choice looks at the sequence alone, as if it had the GPU (152 CTAs) to
// itself, so its bits do not depend on the batch.
#pragma once

#include <math.h>
#include <stdint.h>

namespace pa {

constexpr int kChunkTile = 128;      // rows of a query tile, keys of a key tile
constexpr int kChunkShares = 152;    // shares of a lone sequence
constexpr int kChunkMinShare = 10;    // key tiles of the smallest share (see below)
constexpr int kChunkManyItems = 6 * kChunkShares;

// x / y for x, y >= 0, in 32 bits where they fit.
__host__ __device__ inline int64_t quotient(int64_t x, int64_t y) {
  if (x < (int64_t{1} << 31) && y < (int64_t{1} << 31))
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// Key tile j of item `item` of head `head`: where a unit starts or ends.
struct ChunkPlace {
  int head, item, j;
};

struct ChunkWork {
  int lq, lk, causal, item_tokens, items_head;   // items of one K/V head
  int few;             // leading items whose queries see at most one tile of keys
  int64_t head_keys;   // keys of all items of a head
  int64_t share;       // keys of a share; 0: whole items
  int units;

  // Keys that item i reads: at least a tile's, so that rows that see nothing are written too.
  __host__ __device__ int keys_of(int i) const {
    int64_t keys = lk;
    if (causal) {
      const int64_t last = static_cast<int64_t>(lk) - lq + static_cast<int64_t>(i + 1) * item_tokens;
      keys = last < keys ? last : keys;
    }
    return keys < kChunkTile ? kChunkTile : static_cast<int>(keys);
  }
  __host__ __device__ int tiles_of(int i) const {
    return (keys_of(i) - 1) / kChunkTile + 1;
  }
  // Keys of items [0, i) of a head, i < items_head.
  __host__ __device__ int64_t keys_before(int i) const {
    if (!causal) return static_cast<int64_t>(i) * keys_of(0);
    if (i <= few) return static_cast<int64_t>(i) * kChunkTile;
    const int64_t n = i - few;   // items few .. i - 1: first, first + item_tokens, ...
    const int64_t first = static_cast<int64_t>(lk) - lq + static_cast<int64_t>(few + 1) * item_tokens;
    return static_cast<int64_t>(few) * kChunkTile + n * first + n * (n - 1) / 2 * item_tokens;
  }
  // Item that holds key `pos` of a head's items laid end to end.
  __host__ __device__ int item_at(int64_t pos) const {
    if (!causal) return static_cast<int>(quotient(pos, keys_of(0)));
    int i;
    const int64_t small = static_cast<int64_t>(few) * kChunkTile;
    if (pos < small) {
      i = static_cast<int>(pos / kChunkTile);
    } else {
      // n first + n^2 / 2 item_tokens (with first at the middle of a step) = pos - small
      const float a = 0.5f * item_tokens, x = static_cast<float>(pos - small);
      const float f = static_cast<float>(lk - lq) + (few + 0.5f) * item_tokens;
      const float root = sqrtf(fmaxf(f * f + 4.f * a * x, 0.f));
      const float n = f + root > 0.f ? 2.f * x / (f + root) : 0.f;
      i = few + static_cast<int>(n < static_cast<float>(items_head) ? n : static_cast<float>(items_head));
    }
    if (i > items_head - 1) i = items_head - 1;
    while (i > 0 && keys_before(i) > pos) --i;                        // the guess is at most
    while (i + 1 < items_head && keys_before(i + 1) <= pos) ++i;      // a rounding away
    return i;
  }
  // Where the share that starts at key `pos` of all heads' items starts.
  __host__ __device__ ChunkPlace place_at(int64_t pos, int Hkv) const {
    ChunkPlace x;
    x.head = static_cast<int>(quotient(pos, head_keys));
    if (x.head >= Hkv) {
      x.item = x.j = 0;
      return x;
    }
    const int64_t in_head = pos - x.head * head_keys;
    x.item = item_at(in_head);
    x.j = static_cast<int>(in_head - keys_before(x.item)) / kChunkTile;
    return x;
  }
  // Shares after share u that go on with an item that it begins.
  __host__ __device__ int shares_after(int u, int head, int item) const {
    const int64_t end = head * head_keys + keys_before(item) + keys_of(item);
    return static_cast<int>(quotient(end - 1, share)) - u;
  }
};

__host__ __device__ inline ChunkWork chunk_work(int lq, int lk, int causal, int G, int Hkv) {
  ChunkWork w;
  w.lq = lq;
  w.lk = lk;
  w.causal = causal;
  w.item_tokens = 2 * (kChunkTile / G);
  w.items_head =
      static_cast<int>(quotient(static_cast<int64_t>(lq) + w.item_tokens - 1, w.item_tokens));
  const int64_t room = kChunkTile - (static_cast<int64_t>(lk) - lq);
  const int64_t few = causal && room > 0 ? quotient(room, w.item_tokens) : 0;
  w.few = static_cast<int>(few < w.items_head ? few : w.items_head);
  w.head_keys = w.keys_before(w.items_head - 1) + w.keys_of(w.items_head - 1);
  const int64_t items = static_cast<int64_t>(w.items_head) * Hkv;
  const int64_t all = w.head_keys * Hkv;
  int64_t share = quotient(all + kChunkShares - 1, kChunkShares);
  if (share < kChunkMinShare * kChunkTile) share = kChunkMinShare * kChunkTile;
  if (items >= kChunkManyItems ||
      w.keys_of(w.items_head - 1) <= (kChunkMinShare + kChunkMinShare / 2) * kChunkTile) {
    w.share = 0;
    w.units = static_cast<int>(items);
  } else {
    w.share = share;
    w.units = static_cast<int>(quotient(all + share - 1, share));
  }
  return w;
}

// Whether an 8-bit cache's rows of a sequence are widened to bf16 once, ahead
// of the products, rather than by every item that reads them: from three items
// to a K/V head on.  Widening a key tile ahead costs about 2.5 us of one SM in
// bytes, and in the tiled kernel 1.8 us for every item.
__host__ __device__ inline bool chunk_widens(int lq, int G) {
  return lq > 2 * (2 * (kChunkTile / G));
}

// Rows that a part of an item leaves in the workspace.
__host__ __device__ inline int chunk_part_rows(int lq, int G) {
  const int tokens = 2 * (kChunkTile / G);
  return (lq < tokens ? lq : tokens) * G;
}

// Places for such parts that a sequence of so many shares and items (of all heads)
// has.  A share leaves two parts at most, so share u's are 2 u (it goes on with an
// item) and 2 u + 1 (it begins one); where items are fewer than shares, piece by
// piece: part of item i in share u at u + i.  Either way the parts of an item are in
// order, the first one at slot s and part n at s + 2 n - 1 or s + n.
__host__ __device__ inline int64_t chunk_slots(int64_t shares, int64_t items) {
  return shares + (items < shares ? items : shares);
}

// A run of key tiles [j0, j1) of one item.
struct ChunkPiece {
  int head, item, j0, j1, nk;
};

// Walks the pieces of a unit: from `at` to before `end`.  Share u runs from
// place_at(u * share) to place_at((u + 1) * share).
struct ChunkCursor {
  ChunkPlace at, end;

  // A whole item: heaviest first, the heads side by side.
  __host__ __device__ void start_whole(const ChunkWork &w, int u, int Hkv) {
    const int i = u / Hkv;
    at.head = u - i * Hkv;
    at.item = w.items_head - 1 - i;
    at.j = 0;
    end = at;
    end.j = w.tiles_of(at.item);
  }
  __host__ __device__ bool next(const ChunkWork &w, ChunkPiece &p) {
    const bool last = at.head == end.head && at.item == end.item;
    if (at.head > end.head || (last && at.j >= end.j)) return false;
    p.head = at.head;
    p.item = at.item;
    p.nk = w.tiles_of(at.item);
    p.j0 = at.j;
    p.j1 = last ? end.j : p.nk;
    at.j = last ? end.j : 0;
    if (!last && ++at.item == w.items_head) {
      at.item = 0;
      ++at.head;
    }
    return true;
  }
};

}  // namespace pa
