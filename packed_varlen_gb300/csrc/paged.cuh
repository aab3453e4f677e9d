// Paged K/V cache: what its kernels share -- the cache's layout, the checks
// of one sequence's lengths against it, and the 8-bit rows' arithmetic.
//
// Pages are token-major like every other tensor: row (page g, row r, head h)
// of D elements starts at g * page_stride + (r * Hkv + h) * D.  Position p of
// sequence b is row p % page_size of page table[b, p / page_size].
//
// 8-bit rows.  A row x[0..D) of one token and head is stored as e4m3 values
// y_i and one exponent e, x_i ~ y_i * 2^e, with 2^e the smallest power of two
// that brings max |x_i| to 448 (e4m3's largest value) or less.  A power of two
// leaves a floating format's relative step as it is, so against a scale of
// max / 448 it gives up nothing but the lowest of e4m3's 18 binades; in
// return x * 2^-e and y * 2^e are exact, the one rounding is that to e4m3,
// and a stored value (4 significant bits) is exact in bf16: attention over
// an 8-bit cache is attention over the bf16 rows that reading it back gives.
// e is kept as a byte e + 127 in [num_pages, Hkv, page_size], so a head's
// exponents of one page are one run of page_size bytes.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "packedattn.h"
#include "sched.cuh"

namespace pa {

constexpr int kExpMin = -100;   // rows below 448 * 2^-100 lose low bits, then values
constexpr int kExpMax = 7;      // magnitudes above 448 * 2^7 = 57344 saturate
constexpr int kExpBias = 127;
constexpr int kExpNan = 255;    // a row that held a NaN: all of it reads as NaN

// Everything that locates a cached row.
struct PagedCache {
  void *k, *v;             // pages, bf16 or e4m3
  uint8_t *k_exp, *v_exp;  // exponent bytes (8-bit caches)
  const int32_t *table;    // [batch, table_pages]
  int64_t page_stride;     // elements from one page to the next
  int32_t num_pages, page_shift, table_pages, Hkv, D;
};

__device__ __forceinline__ bool page_ok(const PagedCache &c, int32_t page) {
  return static_cast<uint32_t>(page) < static_cast<uint32_t>(c.num_pages);
}

// Element offset of row (page, row in page, head) and of its exponent byte.
__device__ __forceinline__ int64_t row_offset(const PagedCache &c, int32_t page, int row,
                                              int head) {
  return page * c.page_stride + static_cast<int64_t>(row * c.Hkv + head) * c.D;
}
__device__ __forceinline__ int64_t exp_offset(const PagedCache &c, int32_t page, int row,
                                              int head) {
  return ((static_cast<int64_t>(page) * c.Hkv + head) << c.page_shift) + row;
}

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of a row whose largest magnitude is `a` (no NaN).
__device__ __forceinline__ int row_exponent(float a) {
  const int bits = __float_as_int(a);   // a = (1 + m) 2^n, n from the exponent field
  const int n = (bits >> 23) - 127;
  const int e = n - 8 + ((bits & 0x7fffff) > 0x600000);   // a 2^-e in (224, 448]
  return min(max(e, kExpMin), kExpMax);
}

// Scale of a stored row: 2^e, or NaN for a row that held one.
__device__ __forceinline__ float row_scale(int byte) {
  return byte == kExpNan ? __int_as_float(0x7fffffff) : pow2f(byte - kExpBias);
}

// Four fp32 values -> four e4m3 bytes, rounded to nearest even, saturating.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 2^(120 + e) in bf16 bits for an exponent byte e + 127; NaN for a NaN row.
__device__ __forceinline__ uint32_t widen_scale(uint32_t byte) {
  return byte == kExpNan ? 0x7fffu : (byte + 120u) << 7;
}

// ---------------------------------------------------------------- splits
// Keys of one (sequence, K/V head) are split over CTAs, and the parts joined
// by paged_join_kernel (paged_join.cu).  The rule looks at the sequence's own lengths and the
// head counts only, never at the batch, so a sequence's bits are its own.

// Sequences of few (query, head of the group) rows take the streaming kernel
// (paged_decode.cu), which reads the keys once for every 16 rows, the others
// the tiled one (paged_chunk.cu), which has 256 rows for a key tile and a
// pipeline to fill first.  32 rows, GPU time of the two: 32 sequences over
// 10-12k keys 352 against 410 us, four 62 against 82, 16 over 700-1500 of D = 64
// 44 against 56; 64 rows: 681 against 421, 62 against 62, 69 against 56.
constexpr int kGroupRows = 16;
constexpr int kFewRows = 32;
__host__ __device__ __forceinline__ bool decode_takes(int lq, int G) {
  return lq <= kFewRows && lq * G <= kFewRows;
}
__host__ __device__ __forceinline__ int row_groups(int lq, int G) {   // lq <= kFewRows / G
  return (lq * G + kGroupRows - 1) / kGroupRows;
}

constexpr int kDecodeUnits = 1824;   // parts of a lone sequence: twelve warps for each of 152 SMs

// Smallest part: short contexts are bound by latency and want eight parts at
// most, one for each warp of a CTA that joins them itself; long ones by bytes,
// and want few partial results but enough parts for an even load.  256 keys
// against others, GPU time: one context of 8000 tokens 17.8 us (512: 25.0), 64
// of 900-8000 185 us (512: 192), 96 8-bit ones of 2-12k 281 us (512: 274,
// 1024: 267); 128 up to 4096 keys: one of 4000 16.7 -> 13.7, 24 of 1500 31.5 ->
// 34.4, the 64 185 -> 189.
__host__ __device__ __forceinline__ int decode_min_part(int lk) {
  return lk <= 512 ? 64 : lk <= 1024 ? 128 : 256;
}
__host__ __device__ __forceinline__ int decode_most_parts(int Hkv) {
  return Hkv >= kDecodeUnits ? 1 : kDecodeUnits / Hkv;
}
// Keys of each part (a multiple of 64) of a sequence of lk keys, and its parts.
struct DecodeSplit {
  int part, parts;
};
__host__ __device__ __forceinline__ DecodeSplit decode_split(int lk, int groups, int most) {
  if (groups > 1) most = most > groups ? most / groups : 1;   // more rows, fewer parts
  const int least = decode_min_part(lk);   // a power of two
  DecodeSplit x{least, 0};
  if (lk <= 0) return x;
  if (static_cast<int64_t>(least) * most >= lk) {   // no division for most sequences
    x.parts = (lk - 1) / (lk <= 512 ? 64 : lk <= 1024 ? 128 : 256) + 1;   // least, by shifts
  } else {
    const uint32_t even = (static_cast<uint32_t>(lk) + most - 1) / static_cast<uint32_t>(most);
    x.part = even > (1u << 30) ? static_cast<int>(even) : static_cast<int>((even + 63u) & ~63u);
    x.parts = static_cast<int>((static_cast<uint32_t>(lk) - 1) / static_cast<uint32_t>(x.part)) + 1;
  }
  return x;
}
// The most parts that a sequence of at most max_k keys and so many groups of rows has.
inline int decode_parts_bound(int max_k, int groups, int Hkv) {
  if (max_k <= 0) return 1;
  int64_t n = (static_cast<int64_t>(max_k) + decode_min_part(max_k) - 1) / decode_min_part(max_k);
  if (max_k > 512 && n < 8) n = 8;   // shorter sequences have smaller parts
  int most = decode_most_parts(Hkv);
  if (groups > 1) most = most > groups ? most / groups : 1;
  return static_cast<int>(n < most ? n : most);
}

// The parts of a row are added up in this many sums in turn, these in order.
constexpr int kJoinSums = 8;

// A paged attention call as its kernels see it.
struct PagedAttnParams {
  PagedCache c;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  const int32_t *cu_q, *seq_lens;
  int64_t q_stride;
  int64_t capacity;    // positions that the page table has room for
  int batch0;          // sequences of the call before this launch's (cu_q, seq_lens and
                       // c.table begin at its first)
  int batch, total_q, max_q, max_k, Hq, G;
  int g_inv;           // 2^16 / G + 1: r * g_inv >> 16 is r / G for rows r < 32, G <= 32
  int causal;
  float scale_log2;
  int32_t *status;
  // partial results of the streaming kernel: part s of row (token i, head h)
  // of sequence b, of lq tokens, at slot b * dec_slots + (s * lq + i) * Hq + h
  float *dec_o;        // [slot][D], not normalised
  float2 *dec_ml;      // [slot] (maximum in log2 units, sum)
  int64_t dec_slots;
  int dec_parts, dec_rows;   // bounds of a sequence's parts and rows
  int dec_most;        // decode_most_parts(Hkv)
  // partial results of the tiled kernel
  float *chunk_o;      // [chunk_rows][D], not normalised
  float2 *chunk_ml;    // [chunk_rows]
  int4 *chunk_join;    // two to a share: what to join at its end
  int32_t *chunk_n_cuts;   // shares of the call
  int64_t chunk_rows;
  int chunk_cuts;      // bound on the shares of the call
  int64_t chunk_row0, chunk_row0_rest;   // where part rows and cuts of this launch, and
  int chunk_cut0, chunk_cut0_rest;       // of the one for kSetRest, begin
  // 8-bit rows of long sequences widened once (chunk_widens): bf16 rows in
  // pages of 128, a sequence's pages in a row from flat_page[b] on
  __nv_bfloat16 *flat_k, *flat_v;
  int32_t *flat_page;
  int flat_pages;      // room for so many; 0: the call widens nothing ahead
  int flat_seqs;       // the most sequences that are widened
  int chunk_set;       // the sequences that a launch of the tiled kernel takes
};
enum { kSetAll = 0, kSetFlat = 1, kSetRest = 2 };

// Sequence b of the launch: query rows [q0, q0 + lq), lk keys.  Read like
// seq_bounds: a sequence that breaks the rules is returned without queries and
// `err` says why.
struct PagedSeq {
  int32_t q0, lq, lk;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedAttnParams &p, int b, int &err) {
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), lk = __ldg(p.seq_lens + b);
  PagedSeq s{0, 0, 0};
  err = 0;
  if (!(q0 >= 0 && q0 <= q1 && q1 <= p.total_q && (b + p.batch0 > 0 || q0 == 0))) {
    err = PA_DEVICE_ERR_CU_SEQLENS;
  } else if (lk < 0) {
    err = PA_DEVICE_ERR_LENGTH;
  } else if (q1 - q0 > p.max_q || lk > p.max_k || lk > p.capacity) {
    err = PA_DEVICE_ERR_MAX_LEN;
  } else {
    s.q0 = q0;
    s.lq = q1 - q0;
    s.lk = lk;
  }
  return s;
}

}  // namespace pa
