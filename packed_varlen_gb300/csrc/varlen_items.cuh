// Work items of the packed varlen attention kernels (head dim 64 on single
// CTAs, head dim 128 on CTA pairs): their parameters, the decode of item i of
// the length-ordered list into rows and keys, and the key-tile order.  Both
// kernels take a work item of kVarlenItemRows query rows of one (sequence,
// head) and walk its keys in kVarlenTile-key tiles in the same order, so a
// sequence's rows come out the same whatever the batch around it.
//
// kPrompt: the form for prompts, with grouped heads (query head h reads K/V
// head h / G) and, where p.causal, causal order: query i of a sequence sees key
// j iff j <= lk - lq + i.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "sched.cuh"

namespace pa {

constexpr int kVarlenTile = 128;       // keys of a K/V tile, rows of a Q tile
constexpr int kVarlenItemRows = 256;   // query rows of a work item

struct VarlenParams {
  __nv_bfloat16 *out;
  const int32_t *cu_q, *cu_k;
  int batch, H, total_q, total_k, max_q, max_k;
  float scale_log2;
  int32_t *status;
  int G, causal;   // prompts: query heads per K/V head, causal order
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
  p.causal = a.causal;
  return p;
}

struct ItemInfo {
  int q_row0;   // global row of the item's first query
  int rows;     // valid query rows in the item (1..kVarlenItemRows)
  int k0;       // global row of the sequence's first key
  int lk;       // keys of the sequence
  int nk;       // key tiles
  int head;
  int rot;      // first key tile visited
  int kv_head;  // head of its K and V rows
  int seen;     // prompts: row r of the item sees the keys below min(lk, seen + r + 1)
};

// Key tile visited j-th.  Items start at key tile (item index in the
// sequence mod nk) and wrap around, so the workers of a wave, which hold
// consecutive query blocks of one head, read different K/V tiles at any
// moment.  The order depends only on the sequence's own lengths and the
// item's position in it, so a sequence's result is the same in any batch.
__device__ __forceinline__ int key_tile(const ItemInfo &it, int j) {
  const int kt = it.rot + j;
  return kt >= it.nk ? kt - it.nk : kt;
}

// Item i (0 <= i < prefix[batch]) of the work list; a sequence whose
// boundaries are invalid reads as empty (the list build records why).
template <bool kPrompt = false>
__device__ __forceinline__ ItemInfo item_info(const VarlenParams &p, const int32_t *order,
                                              const int32_t *prefix, int i) {
  const bool causal = kPrompt && p.causal != 0;
  const WorkItem w = causal ? sched_level_item(order, prefix, p.cu_q, p.batch, p.H,
                                               kVarlenItemRows, i)
                            : sched_item(order, prefix, p.batch, p.H, i);
  int err;
  const SeqBounds sb = seq_bounds(p.cu_q, p.cu_k, w.seq, p.total_q, p.total_k, p.max_q,
                                  p.max_k, err);
  ItemInfo it;
  it.q_row0 = sb.q0 + w.tile * kVarlenItemRows;
  it.rows = min(kVarlenItemRows, sb.lq - w.tile * kVarlenItemRows);
  it.k0 = sb.k0;
  it.lk = sb.lk;
  it.head = w.head;
  it.kv_head = kPrompt ? w.head / p.G : w.head;
  it.seen = sb.lk;
  int keys = sb.lk;   // that any row of the item sees
  if (causal) {
    it.seen = sb.lk - sb.lq + w.tile * kVarlenItemRows;
    keys = max(0, it.seen + it.rows);   // (at most lk)
  }
  it.nk = (keys + kVarlenTile - 1) / kVarlenTile;
  // A causal item takes its tiles in order: each row that sees any key sees
  // the first one, so its maximum is finite before a tile that hides all.
  it.rot = it.nk > 0 && !causal ? w.tile % it.nk : 0;
  return it;
}

// The work list of a kernel, in shared memory (see sched_build).
template <bool kPrompt = false>
__device__ __forceinline__ void item_list(const VarlenParams &p, int32_t *order, int32_t *prefix,
                                          int32_t *tmp_lq, int32_t *tmp_lk, bool report) {
  if (kPrompt && p.causal)
    sched_build<true>(order, prefix, tmp_lq, tmp_lk, p.cu_q, p.cu_k, p.batch, p.H,
                      kVarlenItemRows, p.total_q, p.total_k, p.max_q, p.max_k, p.status, report);
  else
    sched_build(order, prefix, tmp_lq, tmp_lk, p.cu_q, p.cu_k, p.batch, p.H, kVarlenItemRows,
                p.total_q, p.total_k, p.max_q, p.max_k, p.status, report);
}

// The worker's n-th item, of `workers`: round robin; in a causal list, whose
// items grow cheaper, every second round backwards, which evens out what a
// round's first worker has more than its last.
template <bool kPrompt = false>
__device__ __forceinline__ int item_at(const VarlenParams &p, int n, int worker, int workers) {
  if (kPrompt && p.causal && (n & 1)) return n * workers + workers - 1 - worker;
  return n * workers + worker;
}

}  // namespace pa
