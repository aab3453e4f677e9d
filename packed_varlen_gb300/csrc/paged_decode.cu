// Paged attention of sequences with few query rows: single-token steps, and
// steps of a few tokens (up to 32 rows of one K/V head's group, in groups of
// 16 that read the keys once each).
//
// Softmax online, in units of log2: with m the largest score so far and
// s' = s * scale * log2(e), a tile adds 2^(s' - m) v to O and 2^(s' - m) to l,
// after both were multiplied by 2^(m_old - m) where m rose; out = O / l.
//
// Bound by the cache's bytes: each is used for 1 to 16 rows only.  So the
// kernel is built around a stream of copies: a unit is one (sequence, K/V
// head, part of the keys, group of rows) and belongs to one warp, which fetches its tiles
// with TMA into a ring of its own and waits for nobody else.  Twelve warps
// share an SM (eight where 16 rows of D = 128 need the registers); a tile is
// 8 KB of K and V, so some 100 KB are in flight per SM.
// Against fetching into registers (16 loads a lane and their addresses for
// every tile) the copies cost four instructions of one lane.
//
// GPU time, 32 query heads on 8 of 128, bf16: 64 sequences of 900-8000 keys
// 181 us (1143 MB, 6.3 TB/s; 9 us of it the join), one of 131,000 89 us (6.0
// TB/s), four of 370-700 9.5 us (latency: some 1100 cycles a tile, and 4200
// before the first).  64 heads on 8, 8-bit rows, 96 sequences of 2-12k: 273-284 us
// (1484 MB, 5.2-5.4 TB/s; parts add 85 MB of writes, see decode_min_part).
//
// (Tensor cores only save instructions here: 16 rows per key keep these busy 15%
// of the time, so the 5th generation's faster ones would gain nothing.)
// The products run with the keys as the M side of m16n8k16 MMAs, so that 8
// query rows fill a tile (N = 8) that 16 rows of padding would waste:
//   S^T [16 keys, 8 rows] = K [16 keys, D] Q^T
//   O^T [D, 8 rows]      += V^T [D, 16 keys] P^T [16 keys, 8 rows]
// The sum over D may run in any order as long as K and Q agree, so a lane
// takes its four values of a k-step from one 16-byte vector of a row; V^T's
// rows may be numbered in any order too, so a lane's V values come from one
// 16-byte vector of each of its four keys, paired by byte permutes.  P^T's B
// operand is S^T's accumulator transposed in 8x8 blocks (movmatrix).  Keys of
// a run may stand in any order as well: key_of() takes them in one in which
// the lanes that read together (rows 2a and 2a + 1 of K, even or odd rows of
// V) fall on different banks of the 128-byte swizzle.
//
// 8-bit rows become f16, which holds e4m3 exactly, one conversion for two
// values; the rows' scales go to the scores (K) and into the weights (V).  The
// weight that is rounded to f16 is then w 2^e of a V row held in units of 2^e,
// so it is taken against the largest s' + e in place of the largest s': among the
// keys that a row of q sees, the one whose values move the output most has a weight
// near f16's top, whatever the exponents of rows that are hidden or weigh nothing.
// Full precision is kept down to 2^-28 of that, and a step of 2^-38 below.
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "paged_launch.h"
#include "tc_ptx.cuh"
#include "tma_map.h"

namespace pa {
namespace {

constexpr int kWarps = 4;         // of a CTA of the streaming kernel
constexpr int kLocalWarps = 8;    // of a CTA that joins its parts itself
// (sequence, K/V head) pairs that a call may have for that: two for each of 152 SMs.
constexpr int kLocalUnits = 304;
constexpr int kLocalKeys = 1024;  // longest sequence that has at most a part for each warp
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays below 2^8
// 8-bit caches: weights are 2^(s' - m) 2^(e + kExpMid), m the largest s' + e + kExpMid
// less kWeightTop at its last rise, so at most 2^(kWeightTop + kWeightRoom), within f16.
// With e + kExpMid in [-54, 53] the sum of the 2^(s' - m) stays within 2^-39 and
// 2^69 for each key.  A rise costs the output's rescaling: room for one binade.
// Beyond kLargeScore a score's own steps would swallow the exponents: from the first
// such rise on, a part's weights are 2^(s' - m - c) 2^(e + kExpMid), with m the
// largest s' and c the largest s' - m + e + kExpMid less kWeightTop.  (That from the
// start costs 14% of four tokens each of 96 sequences, and 1 us of 9.6 where the
// contexts are few and short.)
constexpr int kExpMid = 46;
constexpr float kWeightTop = 14.f, kWeightRoom = 1.f;
constexpr float kLargeScore = 1 << 20;   // log2 units; steps of 2^-4

constexpr long long kWaitLimit = 4000000000LL;   // clock cycles (~2 s)
constexpr long long kDrainLimit = 400000000LL;

// 16 bytes (aligned) to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load16(uint32_t dst, const void *src, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];\n" ::"r"(
          dst),
      "l"(src), "r"(bar)
      : "memory");
}

// Key of a run of 8 that stands in row x of an MMA (see the head of the file):
// 0 4 3 7 5 1 6 2.
__device__ __forceinline__ int key_of(int x) { return (0x26157340 >> (4 * x)) & 7; }

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The low (high) two e4m3 bytes of w as f16, exactly.
__device__ __forceinline__ uint32_t f16_low(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
__device__ __forceinline__ uint32_t f16_high(uint32_t w) { return f16_low(w >> 16); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
template <int D, bool kQuant, int NT, bool kLocal>
struct Cfg {
  static constexpr int kCtaWarps = kLocal ? kLocalWarps : kWarps;
  static constexpr int kRowBytes = D * (kQuant ? 1 : 2);
  static constexpr int kKVecs = kRowBytes / 32;             // a lane's 16-byte K vectors of 16 keys
  static constexpr int kVBytes = kRowBytes >= 128 ? 16 : 8; // a lane's V vector
  static constexpr int kVSets = kRowBytes / (8 * kVBytes);  // vectors of one key
  static constexpr int kVWords = kVBytes / 4;
  static constexpr int kHalves = kRowBytes == 256 ? 1 : 2;  // 16-key runs of a tile
  static constexpr int kTileKeys = 16 * kHalves;
  // A run in shared memory: 16 rows of 128 swizzled bytes, two such blocks for
  // rows of 256 bytes; rows of 64 bytes as they are.
  static constexpr int kBlocks = kRowBytes == 256 ? 2 : 1;
  static constexpr int kLine = kRowBytes / kBlocks;
  static constexpr int kRunBytes = 16 * kRowBytes;
  // a stage: K runs, V runs, then (8-bit) 16 exponent bytes of each
  static constexpr int kExpOff = 2 * kHalves * kRunBytes;
  static constexpr int kStageBytes = kExpOff + (kQuant ? 1024 : 0);   // 1024: the swizzle's period
  static constexpr int kStageTx = kExpOff + (kQuant ? 2 * kHalves * 16 : 0);
  static constexpr int kCtas = kLocal ? 1 : NT == 1 || D == 64 ? 3 : 2;   // CTAs that share an SM
  static constexpr int kPartBytes = kLocal ? kLocalWarps * 8 * NT * (D + 2) * 4 : 0;
  static constexpr int kRoom = 233472 / kCtas - 1024 - 1024 - kPartBytes;
  static constexpr int kFit = kRoom / (kCtaWarps * kStageBytes);
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kPartOff = kCtaWarps * kStages * kStageBytes;
  static constexpr int kBarOff = kPartOff + kPartBytes;
  static constexpr int kSmem = kBarOff + kCtaWarps * (kStages + 1) * 8;   // a flag's place for each warp
  static_assert(kStages >= 2, "no ring");
};

// Walks the units of the call, (sequence, part of its keys, group of 16 rows,
// K/V head), heads running fastest: a warp holds 32 sequences at a time, one per lane, with the
// units before each.  Units are asked for in rising order.
struct Walk {
  int group, base, total;       // 32 sequences from group * 32, their first unit, their units
  int q0, lq, lk, first, units; // this lane's sequence
  // the unit found
  int b, part, rows0, hk, s_q0, s_lq, s_lk;

  __device__ __forceinline__ void load(const PagedAttnParams &p, bool report) {
    const int lane = threadIdx.x & 31, x = group * 32 + lane;
    q0 = lq = lk = units = 0;
    if (x < p.batch) {
      int err;
      const PagedSeq s = paged_seq(p, x, err);
      if (err && report) record_error(p.status, err);
      q0 = s.q0;
      lq = s.lq;
      lk = s.lk;
      if (lq > 0 && decode_takes(lq, p.G)) {
        const int groups = row_groups(lq, p.G);   // no keys: a unit writes zeros
        units = max(decode_split(lk, groups, p.dec_most).parts, 1) * groups * p.c.Hkv;
      }
    }
    int incl = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    first = incl - units;
    total = __shfl_sync(0xffffffffu, incl, 31);
  }
  __device__ __forceinline__ void open(const PagedAttnParams &p, bool report) {
    group = base = 0;
    load(p, report);
  }
  __device__ __forceinline__ bool seek(const PagedAttnParams &p, int u, bool report) {
    while (u >= base + total) {
      base += total;
      ++group;
      if (group * 32 >= p.batch) {
        total = 0;
        --group;
        return false;
      }
      load(p, report);
    }
    const int local = u - base;
    const uint32_t at = __ballot_sync(0xffffffffu, units > 0 && first <= local);
    const int src = 31 - __clz(at);
    const int rest = local - __shfl_sync(0xffffffffu, first, src);
    b = group * 32 + src;
    s_q0 = __shfl_sync(0xffffffffu, q0, src);
    s_lq = __shfl_sync(0xffffffffu, lq, src);
    part = rest / p.c.Hkv;
    hk = rest - part * p.c.Hkv;
    rows0 = 0;
    const int groups = row_groups(s_lq, p.G);
    if (groups > 1) {
      rows0 = part % groups * kGroupRows;
      part /= groups;
    }
    s_lk = __shfl_sync(0xffffffffu, lk, src);
    return true;
  }
};

// Every warp walks units of its own: its number, its number + all warps, ...
// kLocal: a CTA has one (sequence, K/V head), each of its warps a part, and
// joins them in shared memory: one launch and no workspace, for calls of few
// short contexts, whose time is latency.
template <int D, bool kQuant, int NT, bool kLocal>
__global__ void __launch_bounds__(Cfg<D, kQuant, NT, kLocal>::kCtaWarps * 32,
                                  Cfg<D, kQuant, NT, kLocal>::kCtas)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedAttnParams p) {
  using C = Cfg<D, kQuant, NT, kLocal>;
  constexpr int kTile = C::kTileKeys;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int page_mask = (1 << p.c.page_shift) - 1;
  if (tc::smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) record_error(p.status, PA_DEVICE_ERR_SMEM_ALIGN);
    tc::griddep_wait();
    return;
  }
  uint8_t *ring = smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_u = tc::smem_u32(ring);
  const uint32_t bars = tc::smem_u32(smem + C::kBarOff) + warp * (C::kStages + 1) * 8;
  volatile int32_t *gave_up = reinterpret_cast<volatile int32_t *>(
      smem + C::kBarOff + (warp * (C::kStages + 1) + C::kStages) * 8);
  if (lane == 0) {
    for (int x = 0; x < C::kStages; ++x) tc::mbar_init(bars + 8 * x, 1);
    *gave_up = 0;
    tc::fence_mbar_init();
  }
  __syncwarp();
  const bool lead = tc::elect_one();
  if (warp == 0 && lead) {
    tc::tma_prefetch_desc(&tm_k);
    tc::tma_prefetch_desc(&tm_v);
  }
  // this lane's places in a run: K rows g and g + 8, V rows of four keys
  const int kkey = key_of(g);
  const int vkey[2] = {key_of(2 * t), key_of(2 * t + 1)};
  float *part_o = reinterpret_cast<float *>(smem + C::kPartOff);   // kLocal: [part][row][D]
  float2 *part_ml = reinterpret_cast<float2 *>(part_o + kLocalWarps * 8 * NT * D);
  uint32_t issued = 0, used = 0;   // tiles of this warp so far
  uint32_t bad = 0;                // bit (stage * halves + run): no such page, or past the part
  bool ok = true;
  Walk w;
  const bool report = blockIdx.x == 0 && warp == 0;
  int32_t early = 0;   // kLocal: pages of this warp's part, read before its length is known
  if constexpr (kLocal) {
    w.b = blockIdx.x / p.c.Hkv;
    w.hk = blockIdx.x - w.b * p.c.Hkv;
    // runs of parts of 64 keys in lanes 0 to 3, of 128 keys in lanes 8 to 15
    const int entry = (lane < 4 ? warp * 64 + lane * 16 : warp * 128 + (lane & 7) * 16) >> p.c.page_shift;
    if ((lane < 4 || (lane & 24) == 8) && entry < p.c.table_pages)
      early = __ldg(p.c.table + static_cast<int64_t>(w.b) * p.c.table_pages + entry);
    int err;
    const PagedSeq s = paged_seq(p, w.b, err);
    if (err && w.hk == 0 && threadIdx.x == 0) record_error(p.status, err);
    if (s.lq == 0 || !decode_takes(s.lq, p.G)) {
      tc::griddep_wait();
      return;
    }
    w.s_q0 = s.q0;
    w.s_lq = s.lq;
    w.s_lk = s.lk;
    w.rows0 = 0;
    w.total = max(decode_split(s.lk, 1, p.dec_most).parts, 1);
  } else {
    w.open(p, report);
  }
  // the next unit; a warp of a local CTA has one part
  auto more_units = [&](int u) -> bool {
    if constexpr (kLocal) {
      w.part = u;
      return u < w.total;
    } else {
      return w.seek(p, u, report);
    }
  };
  const int u_first = kLocal ? warp : blockIdx.x * kWarps + warp;
  const int u_step = kLocal ? kLocalWarps : gridDim.x * kWarps;
  // ---- copies: the part that is being fetched and its next tile
  const int32_t *table = p.c.table;
  int src_k0 = 0, src_runs = 0, src_tiles = 0, src_n = 0;
  // pages of 32 runs of 16 keys at a time, one per lane (a run lies in one page)
  int32_t pages = 0, pages_next = 0;
  auto load_pages = [&](int n0) -> int32_t {
    const int n = n0 + lane;
    return n < src_runs ? __ldg(table + ((src_k0 + n * 16) >> p.c.page_shift)) : 0;
  };
  auto open_source = [&](int part) {
    const int keys_part = decode_split(w.s_lk, row_groups(w.s_lq, p.G), p.dec_most).part;
    src_k0 = part * keys_part;
    const int keys = min(w.s_lk - src_k0, keys_part);
    src_runs = keys > 0 ? (keys + 15) / 16 : 0;
    src_tiles = (src_runs + C::kHalves - 1) / C::kHalves;
    src_n = 0;
    if (kLocal && (keys_part == 64 || keys_part == 128)) {
      pages = __shfl_sync(0xffffffffu, early, keys_part == 64 ? lane : 8 + (lane & 7));
    } else {
      pages = load_pages(0);
      pages_next = load_pages(32);
    }
  };
  // copies of the next tile, if there is one, into the ring's next stage
  auto issue = [&]() {
    if (src_n == src_tiles) return;
    const int n = src_n++;
    const uint32_t st = issued % C::kStages, dst = ring_u + st * C::kStageBytes;
    const uint32_t bar = bars + 8 * st;
    if (n > 0 && (n * C::kHalves & 31) == 0) {
      pages = pages_next;
      pages_next = load_pages(n * C::kHalves + 32);
    }
    if (lead) tc::mbar_arrive_expect_tx(bar, C::kStageTx);
#pragma unroll
    for (int h = 0; h < C::kHalves; ++h) {
      const int run = n * C::kHalves + h;
      int32_t page = __shfl_sync(0xffffffffu, pages, run & 31);
      const bool there = run < src_runs, good = there && page_ok(p.c, page);
      const uint32_t bit = 1u << (st * C::kHalves + h);
      bad = good ? bad & ~bit : bad | bit;
      if (there && !good && lead) record_error(p.status, PA_DEVICE_ERR_PAGE);
      if (!good) page = -1;   // lands as zeros
      const int row0 = (src_k0 + run * 16) & page_mask;
      if (lead) {
#pragma unroll
        for (int x = 0; x < C::kBlocks; ++x) {
          tc::tma_load_4d(dst + h * C::kRunBytes + x * 2048, &tm_k, bar, x * 64, w.hk, row0, page);
          tc::tma_load_4d(dst + (C::kHalves + h) * C::kRunBytes + x * 2048, &tm_v, bar, x * 64, w.hk,
                          row0, page);
        }
        if (kQuant) {
          const int64_t ex = exp_offset(p.c, good ? page : 0, row0, w.hk);
          bulk_load16(dst + C::kExpOff + h * 16, p.c.k_exp + ex, bar);
          bulk_load16(dst + C::kExpOff + (C::kHalves + h) * 16, p.c.v_exp + ex, bar);
        }
      }
    }
    ++issued;
  };

  auto token_of = [&](int r) { return r * p.g_inv >> 16; };   // of a row of the sequence
  for (int u = u_first; ok && more_units(u); u += u_step) {
    const int lq = w.s_lq, lk = w.s_lk, hk = w.hk;
    const int r0 = w.rows0, R = min(lq * p.G - r0, kGroupRows);   // this unit's rows
    const DecodeSplit split = decode_split(lk, row_groups(lq, p.G), p.dec_most);
    const int parts = split.parts, k0 = w.part * split.part, keys = min(lk - k0, split.part);
    const int n_tiles = (keys + kTile - 1) / kTile;
    table = p.c.table + static_cast<int64_t>(w.b) * p.c.table_pages;
    open_source(w.part);
    // Q^T, the B operand of every S^T product.  Over an 8-bit cache it is f16,
    // each row scaled by a power of two to the top of f16's range (what that
    // loses lies 2^-40 below the row's largest); the scores' factor takes it back.
    uint32_t qf[NT][D / 16][2];
    float factor[NT][2];   // of this lane's two columns (rows of q)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const bool live = r < R;
      const int i = live ? token_of(r0 + r) : 0, gg = live ? r0 + r - i * p.G : 0;
      const __nv_bfloat16 *row =
          p.q + (w.s_q0 + i) * p.q_stride + static_cast<int64_t>(hk * p.G + gg) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint2 x = make_uint2(0u, 0u);
        // four values: of vector t + 4 (ks / 2) (bf16) or t + 4 (ks / 4) (e4m3)
        const int d = kQuant ? (t + 4 * (ks >> 2)) * 16 + (ks & 3) * 4
                             : (t + 4 * (ks >> 1)) * 8 + (ks & 1) * 4;
        if (live) x = __ldg(reinterpret_cast<const uint2 *>(row + d));
        qf[nt][ks][0] = x.x;
        qf[nt][ks][1] = x.y;
      }
    }
#pragma unroll
    for (int n = 0; n < C::kStages - 1; ++n) issue();   // while q is on its way
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float back = p.scale_log2;
      if constexpr (kQuant) {
        uint32_t top = 0;   // largest exponent field of the row, in place
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = qf[nt][ks][e] & 0x7f807f80u;
            top = max(top, max(x & 0xffffu, x >> 16));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // |q| < 2^(field - 126): times 2^up it stays below 2^15
        const int up = min(141 - static_cast<int>(top >> 7), 126);
        const float f = pow2f(up);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[nt][ks][e] = pack_f16x2(__uint_as_float(qf[nt][ks][e] << 16) * f,
                                       __uint_as_float(qf[nt][ks][e] & 0xffff0000u) * f);
        back = p.scale_log2 * pow2f(-up);
      }
      factor[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      factor[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }
    // last key + 1 that each of this lane's columns (rows of q) sees
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
        lim[nt][e] = r >= R ? 0 : p.causal ? lk - lq + 1 + token_of(r0 + r) : lk;
      }
    const int all_see = p.causal ? lk - lq + 1 + token_of(r0) : lk;   // keys before it need no mask

    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    [[maybe_unused]] float c[NT][2];   // with large scores over an 8-bit cache
    bool large = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // Tiles from n on, until the first large score (not kLarge).
    int n = 0;
    auto walk = [&](auto columns, auto with_large) {
      constexpr int NC = decltype(columns)::value;
      constexpr bool kLarge = decltype(with_large)::value;
      const int n_here = kLarge ? n : -1;   // this tile's copies are waited for already
      for (; n < n_tiles; ++n) {
        const int key = k0 + n * kTile;
        if (n != n_here) {
          // every lane has read the stage that is filled next (the tile before this one)
          __syncwarp();
          issue();
        }
        const uint32_t stage = used % C::kStages;
        ok = tc::bounded_wait(bars + 8 * stage, (used / C::kStages) & 1u, gave_up, p.status, kWaitLimit);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const uint8_t *st = ring + stage * C::kStageBytes;
        [[maybe_unused]] const uint32_t bad_runs = bad >> (stage * C::kHalves);
        // byte address of 16-byte vector `vec` of row `row` of a run
        auto vector = [&](const uint8_t *run, int row, int vec) -> const uint8_t * {
          if constexpr (C::kLine == 128)
            return run + (vec >> 3) * 2048 + row * 128 + (((vec & 7) ^ (row & 7)) << 4);
          else
            return run + row * C::kLine + (vec << 4);
        };

        // S^T = K Q^T, in two chains
        float sc[C::kHalves][NC][4];
        float kf[C::kHalves][2], vf[C::kHalves][2];
        [[maybe_unused]] float ve[C::kHalves][2] = {};   // log2 of vf: keys key_of(g) and 8 later
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
          float s2[NC][4];
#pragma unroll
          for (int nt = 0; nt < NC; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[h][nt][e] = s2[nt][e] = 0.f;
#pragma unroll
          for (int i = 0; i < C::kKVecs / 2; ++i) {
            const uint8_t *run = st + h * C::kRunBytes;
            const uint4 a = *reinterpret_cast<const uint4 *>(vector(run, kkey, t + 4 * i));
            const uint4 c = *reinterpret_cast<const uint4 *>(vector(run, kkey + 8, t + 4 * i));
            if constexpr (!kQuant) {
#pragma unroll
              for (int nt = 0; nt < NC; ++nt) {
                mma16816(sc[h][nt], a.x, c.x, a.y, c.y, qf[nt][2 * i][0], qf[nt][2 * i][1]);
                mma16816(s2[nt], a.z, c.z, a.w, c.w, qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
              }
            } else {
              const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t a0 = f16_low(aw[x]), a2 = f16_high(aw[x]);
                const uint32_t a1 = f16_low(cw[x]), a3 = f16_high(cw[x]);
#pragma unroll
                for (int nt = 0; nt < NC; ++nt)
                  mma16816_f16(x & 1 ? s2[nt] : sc[h][nt], a0, a1, a2, a3, qf[nt][4 * i + x][0],
                               qf[nt][4 * i + x][1]);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NC; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[h][nt][e] += s2[nt][e];
          if constexpr (kQuant) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // bytes of rows that are not the sequence's may be anything
              const bool mine = key + 16 * h + 8 * e + kkey < lk && !(bad_runs >> h & 1u);
              const uint8_t *ex = st + C::kExpOff + h * 16 + 8 * e + kkey;
              kf[h][e] = mine ? row_scale(ex[0]) : 0.f;
              const int byte = mine ? ex[C::kHalves * 16] : kExpNan;
              const bool has = byte != kExpNan;   // an exponent
              ve[h][e] = static_cast<float>((has ? byte : kExpBias + kExpMin) - (kExpBias - kExpMid));
              vf[h][e] = has ? pow2f(byte - (kExpBias - kExpMid))
                             : mine ? __int_as_float(0x7fffffff) : 0.f;
            }
          }
        }

        // online softmax over the tile's keys, all lanes of a column in step
        bool above = false, up[NC][2];
        float mx[NC][2];
        // highest score of this lane's keys in a column; `graded`: with V's exponents
        auto highest = [&](auto graded, int nt, int e, float ref) {
          auto level = [&](int h, int x) {
            const float y = kLarge ? sc[h][nt][e + 2 * x] - ref : sc[h][nt][e + 2 * x];
            if constexpr (decltype(graded)::value) return y + ve[h][x];
            return y;
          };
          float y = fmaxf(level(0, 0), level(0, 1));
#pragma unroll
          for (int h = 1; h < C::kHalves; ++h) y = tc::fmax3(y, level(h, 0), level(h, 1));
          return y;
        };
        constexpr std::bool_constant<kQuant> by_level;
        auto of_column = [](float x) {   // largest of the eight lanes of a column
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        };
#pragma unroll
        for (int nt = 0; nt < NC; ++nt) {
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (kQuant) sc[h][nt][e] *= kf[h][e >> 1];
              sc[h][nt][e] = __fmul_rn(sc[h][nt][e], factor[nt][e & 1]);   // (no FFMA with a maximum)
            }
            if (key + kTile > all_see) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key + 16 * h + kkey + 8 * (e >> 1) >= lim[nt][e & 1]) sc[h][nt][e] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[nt][e] = highest(by_level, nt, e, m[nt][e] == -INFINITY ? 0.f : m[nt][e]);
            // from -inf: any finite score
            up[nt][e] = mx[nt][e] > (kLarge ? c[nt][e] : m[nt][e]) +
                                        (kQuant ? kWeightTop + kWeightRoom : kRescaleThreshold);
            above |= up[nt][e];
          }
        }
        // The columns' maxima are joined only where one has risen (a vote in place of
        // six shuffles: 100 cycles of a tile's 1150).
        if (__any_sync(0xffffffffu, above)) {
          if constexpr (kQuant && !kLarge) {
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NC; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                mx[nt][e] = of_column(mx[nt][e]);
                far |= fabsf(mx[nt][e]) > kLargeScore && mx[nt][e] > -INFINITY;
              }
            if (__any_sync(0xffffffffu, far)) {
              large = true;
              break;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NC; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              alpha[e] = 1.f;
              if constexpr (kLarge) {
                const float top =
                    fmaxf(of_column(highest(std::false_type{}, nt, e, 0.f)), m[nt][e]);
                const float x = of_column(highest(by_level, nt, e, top == -INFINITY ? 0.f : top));
                if (__ballot_sync(0xffffffffu, up[nt][e]) & (0x11111111u << t)) {
                  alpha[e] = tc::ex2((m[nt][e] - top) + (c[nt][e] - (x - kWeightTop)));
                  m[nt][e] = top;
                  c[nt][e] = x - kWeightTop;
                }
              } else {
                float x = kQuant ? mx[nt][e] : of_column(mx[nt][e]);
                if (x > m[nt][e] + (kQuant ? kWeightTop + kWeightRoom : kRescaleThreshold)) {
                  if (kQuant) x -= kWeightTop;
                  alpha[e] = tc::ex2(m[nt][e] - x);
                  m[nt][e] = x;
                }
              }
              l[nt][e] *= alpha[e];
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][mt][e] *= alpha[e & 1];
          }
        }
        uint32_t pf[C::kHalves][NC][2];
#pragma unroll
        for (int nt = 0; nt < NC; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool none = m[nt][e] == -INFINITY;
            const float ref = none ? 0.f : m[nt][e];
            auto weight = [&](float x) {
              if constexpr (kLarge) return tc::ex2(x - ref - (none ? 0.f : c[nt][e]));
              return tc::ex2(x - ref);
            };
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
              const float p0 = weight(sc[h][nt][e]), p1 = weight(sc[h][nt][e + 2]);
              l[nt][e] += p0 + p1;
              sc[h][nt][e] = kQuant ? p0 * vf[h][0] : p0;
              sc[h][nt][e + 2] = kQuant ? p1 * vf[h][1] : p1;
            }
          }
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
            pf[h][nt][0] = transpose8x8(kQuant ? pack_f16x2(sc[h][nt][0], sc[h][nt][1])
                                               : tc::pack_bf16x2(sc[h][nt][0], sc[h][nt][1]));
            pf[h][nt][1] = transpose8x8(kQuant ? pack_f16x2(sc[h][nt][2], sc[h][nt][3])
                                               : tc::pack_bf16x2(sc[h][nt][2], sc[h][nt][3]));
          }
        }

        // O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
#pragma unroll
          for (int cs = 0; cs < C::kVSets; ++cs) {
            uint32_t va[4][C::kVWords];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const int row = vkey[kk & 1] + 8 * (kk >> 1);
              const uint8_t *run = st + (C::kHalves + h) * C::kRunBytes;
              if constexpr (C::kVBytes == 16) {
                const uint4 x = *reinterpret_cast<const uint4 *>(vector(run, row, g + 8 * cs));
                va[kk][0] = x.x;
                va[kk][1] = x.y;
                va[kk][2] = x.z;
                va[kk][3] = x.w;
              } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(run + row * C::kLine + g * 8);
                va[kk][0] = x.x;
                va[kk][1] = x.y;
              }
            }
            if (key + kTile > lk) {   // rows past the last key: weight 0, whatever they hold
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (key + 16 * h + vkey[kk & 1] + 8 * (kk >> 1) >= lk)
#pragma unroll
                  for (int x = 0; x < C::kVWords; ++x) va[kk][x] = 0u;
            }
#pragma unroll
            for (int x = 0; x < C::kVWords; ++x) {
              // bf16: values 0 and 1 of the word, of two keys each; e4m3: 0, 1 and 2, 3
              const uint32_t ab0 = __byte_perm(va[0][x], va[1][x], kQuant ? 0x5140 : 0x5410);
              const uint32_t ab1 = __byte_perm(va[0][x], va[1][x], kQuant ? 0x7362 : 0x7632);
              const uint32_t cd0 = __byte_perm(va[2][x], va[3][x], kQuant ? 0x5140 : 0x5410);
              const uint32_t cd1 = __byte_perm(va[2][x], va[3][x], kQuant ? 0x7362 : 0x7632);
#pragma unroll
              for (int nt = 0; nt < NC; ++nt) {
                if constexpr (!kQuant) {
                  mma16816(o[nt][cs * 4 + x], ab0, ab1, cd0, cd1, pf[h][nt][0], pf[h][nt][1]);
                } else {
                  mma16816_f16(o[nt][2 * x], f16_low(ab0), f16_high(ab0), f16_low(cd0),
                               f16_high(cd0), pf[h][nt][0], pf[h][nt][1]);
                  mma16816_f16(o[nt][2 * x + 1], f16_low(ab1), f16_high(ab1), f16_low(cd1),
                               f16_high(cd1), pf[h][nt][0], pf[h][nt][1]);
                }
              }
            }
          }
        }
        ++used;
      }
    };
    // A sequence of at most eight rows takes one group of columns, whatever the call's
    // others need: 96 8-bit sequences of one token in a call that allows for 32 rows 324
    // / 300 us.  (Not the second half of more rows: its warps would run ahead of those
    // that read the same keys, 246 / 275 us with five tokens of four heads each.)
    auto walk_all = [&](auto columns) {
      walk(columns, std::false_type{});
      if constexpr (kQuant) {
        if (large) {   // from here on with m and c
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) c[nt][e] = m[nt][e] == -INFINITY ? -INFINITY : 0.f;
          walk(columns, std::true_type{});
        }
      }
    };
    if (NT == 1 || lq * p.G <= 8)
      walk_all(std::integral_constant<int, 1>{});
    else
      walk_all(std::integral_constant<int, NT>{});

    // ---- this lane's columns: D / 8 dims each of rows 2 t and 2 t + 1, in runs
    // of 2 KR consecutive ones
    constexpr int KR = !kQuant && D == 128 ? 4 : D / 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
        const int r = nt * 8 + 2 * t + e;
        if (r >= R) continue;
        const int i = token_of(r0 + r), h = hk * p.G + r0 + r - i * p.G;
        if (parts <= 1) {
          constexpr float grade = kQuant ? 1.f / (1ll << kExpMid) : 1.f;
          const float inv = m[nt][e] == -INFINITY ? 0.f : 1.f / l[nt][e];
          __nv_bfloat16 *dst = p.out + (static_cast<int64_t>(w.s_q0 + i) * p.Hq + h) * D;
#pragma unroll
          for (int mt = 0; mt < D / 16; mt += 4) {
            const int d = g * 2 * KR + 16 * KR * (mt / KR) + 2 * (mt % KR);
            uint32_t x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              x[y] = tc::pack_bf16x2(o[nt][mt + y][e] * grade * inv, o[nt][mt + y][e + 2] * grade * inv);
            *reinterpret_cast<uint4 *>(dst + d) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else {
          const int64_t slot =
              w.b * p.dec_slots + static_cast<int64_t>(w.part * lq + i) * p.Hq + h;
          float *dst = kLocal ? part_o + (w.part * 8 * NT + r) * D : p.dec_o + slot * D;
          // both against m alone, as the join takes them
          const float from_c = kQuant && large && m[nt][e] != -INFINITY ? tc::ex2(c[nt][e]) : 1.f;
          const float grade = kQuant ? from_c * pow2f(-kExpMid) : 1.f;
#pragma unroll
          for (int mt = 0; mt < D / 16; mt += 2) {
            const int d = g * 2 * KR + 16 * KR * (mt / KR) + 2 * (mt % KR);
            *reinterpret_cast<float4 *>(dst + d) =
                make_float4(o[nt][mt][e] * grade, o[nt][mt][e + 2] * grade, o[nt][mt + 1][e] * grade,
                            o[nt][mt + 1][e + 2] * grade);
          }
          float2 *ml = kLocal ? part_ml + w.part * 8 * NT + r : p.dec_ml + slot;
          if (g == 0) *ml = make_float2(m[nt][e], l[nt][e] * from_c);
        }
      }
    }
  }
  if constexpr (kLocal) {
    // the join of paged_join_kernel, step for step: each of its eight sums has
    // at most one part here
    static_assert(kLocalWarps == kJoinSums, "one part to a sum");
    if (w.total > 1) {
      __syncthreads();
      const int R = w.s_lq * p.G;
      for (int x = threadIdx.x; x < R * (D / 4); x += kLocalWarps * 32) {
        const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
        float2 v[kJoinSums];
        float4 o[kJoinSums];
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kJoinSums; ++n) {
          v[n] = make_float2(-INFINITY, 0.f);
          o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n < w.total) {
            v[n] = part_ml[n * 8 * NT + r];
            o[n] = *reinterpret_cast<const float4 *>(part_o + (n * 8 * NT + r) * D + d);
          }
          top = fmaxf(top, v[n].x);
        }
        const float ref = top == -INFINITY ? 0.f : top;
        float total = 0.f;
        float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int n = 0; n < kJoinSums; ++n) {
          const float f = tc::ex2(v[n].x - ref);
          total = __fadd_rn(total, __fmul_rn(f, v[n].y));
          out.x = __fadd_rn(out.x, __fmul_rn(f, o[n].x));
          out.y = __fadd_rn(out.y, __fmul_rn(f, o[n].y));
          out.z = __fadd_rn(out.z, __fmul_rn(f, o[n].z));
          out.w = __fadd_rn(out.w, __fmul_rn(f, o[n].w));
        }
        const float inv = top == -INFINITY ? 0.f : 1.f / total;   // NaN stays NaN
        const int i = r / p.G, h = w.hk * p.G + r - i * p.G;
        *reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(w.s_q0 + i) * p.Hq + h) * D + d) =
            make_uint2(tc::pack_bf16x2(out.x * inv, out.y * inv),
                       tc::pack_bf16x2(out.z * inv, out.w * inv));
      }
    }
  }
  if (!ok) {   // give the copies already issued a bounded chance to land
    for (; used < issued; ++used)
      tc::drain_wait(bars + 8 * (used % C::kStages), (used / C::kStages) & 1u, kDrainLimit);
  }
  // every way out waits: this kernel's end is the end of the tiled one before it
  tc::griddep_wait();
}

// Rows of a page as (D, Hkv, row, page): a box is one head's rows of a run.
bool make_map(CUtensorMap *map, const void *ptr, const PagedCache &c, bool quant) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t es = quant ? 1 : 2, D = c.D, H = c.Hkv;
  const cuuint64_t dims[4] = {D, H, cuuint64_t{1} << c.page_shift,
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {D * es, H * D * es, static_cast<cuuint64_t>(c.page_stride) * es};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(quant ? D : 64), 1, 16, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             quant && D == 64 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kQuant, int NT, bool kLocal>
cudaError_t launch(const PagedAttnParams &p, int num_sms, bool after_chunk, cudaStream_t stream) {
  using C = Cfg<D, kQuant, NT, kLocal>;
  CUtensorMap mk, mv;
  if (!make_map(&mk, p.c.k, p.c, kQuant) || !make_map(&mv, p.c.v, p.c, kQuant))
    return cudaErrorInvalidValue;
  static unsigned long long configured = 0;
  cudaError_t e =
      set_smem_once(reinterpret_cast<const void *>(paged_decode_kernel<D, kQuant, NT, kLocal>),
                    C::kSmem, configured);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(p.batch) * p.c.Hkv *
                        (kLocal ? 1 : p.dec_parts * (p.dec_rows / p.Hq * p.G + 15) / 16);
  const int64_t most = kLocal ? units : (units + kWarps - 1) / kWarps;
  const int64_t ctas = kLocal ? units : static_cast<int64_t>(num_sms) * C::kCtas;
  // After the tiled kernel of the same call this one may start as that one's
  // CTAs leave their SMs (it waits for its end at its own end).
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < ctas ? most : ctas));
  cfg.blockDim = dim3(C::kCtaWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = after_chunk ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_decode_kernel<D, kQuant, NT, kLocal>, mk, mv, p);
}

}  // namespace

bool paged_decode_is_local(int batch, int tokens, int max_k, int G, int Hkv) {
  return tokens > 0 && tokens * G <= 8 && max_k <= kLocalKeys &&
         static_cast<int64_t>(batch) * Hkv <= kLocalUnits;
}

template <int D, bool kQuant>
static cudaError_t launch_for(const PagedAttnParams &p, int num_sms, bool after_chunk,
                       cudaStream_t stream) {
  // 8 columns where no sequence of the call can have more rows: a column's
  // results do not depend on the others, so this changes no bits
  const int tokens = p.dec_rows / p.Hq;   // the bound that the workspace was planned for
  if (paged_decode_is_local(p.batch, tokens, p.max_k, p.G, p.c.Hkv))
    return launch<D, kQuant, 1, true>(p, num_sms, after_chunk, stream);
  return tokens * p.G > 8 ? launch<D, kQuant, 2, false>(p, num_sms, after_chunk, stream)
                          : launch<D, kQuant, 1, false>(p, num_sms, after_chunk, stream);
}

cudaError_t launch_paged_decode(const PagedAttnParams &p, bool quant, int num_sms,
                                bool after_chunk, cudaStream_t stream) {
  if (p.c.D == 128)
    return quant ? launch_for<128, true>(p, num_sms, after_chunk, stream)
                 : launch_for<128, false>(p, num_sms, after_chunk, stream);
  return quant ? launch_for<64, true>(p, num_sms, after_chunk, stream)
               : launch_for<64, false>(p, num_sms, after_chunk, stream);
}

}  // namespace pa
