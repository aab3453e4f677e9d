// Packed rows into a paged K/V cache (quantised to 8 bits as they are
// written, where the cache holds 8-bit rows) and back out of it.
//
// Token j of packed sequence b sits at position pos_offset[b] + j, as in the
// rotary embedding of the same rows; paged.cuh has the layout and the 8-bit
// rows' arithmetic.  Both directions are bound by HBM: every byte is read and
// written once, 16 bytes of cache row to a thread (8 bf16 or 16 e4m3
// elements).  A row's D elements lie in D / 8 (or D / 16) neighbouring lanes,
// so its largest magnitude is a butterfly of 2 to 3 shuffles and the row
// never leaves registers between its load and its store.  Where each token of a
// tile goes is found first, a token to a thread, so that a vector's address is
// a lookup in shared memory.  GPU time, 8 heads of 128: 32k tokens into 8-bit
// pages 35.6 us (196 MB, 5.5 TB/s), 106k tokens out of them 103 us (651 MB, 6.3
// TB/s), 2.4k tokens out of bf16 pages 5.5 us.
#include "internal.h"
#include "paged.cuh"
#include "paged_chunk_work.cuh"
#include "paged_launch.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kTileTokens = 64;   // tokens of a tile, at most
// Cache vectors of a tile: one per thread, and twice or four times as many where
// that leaves three tiles per SM.  256 / 512 / 1024, GPU time: 96 tokens into 8-bit
// pages 4.3 / 4.6 / 5.4 us, 2424 out of bf16 pages 7.4 / 5.5 / 5.5, 106k out of
// 8-bit pages - / 109 / 103 (2048: 104).
constexpr int kLeastVecs = kThreads, kMostVecs = 1024, kTilesPerSm = 3;

struct CopyParams {
  PagedCache c;
  uint8_t *k_rows, *v_rows;      // packed rows, bf16
  int64_t k_stride, v_stride;    // bytes from one token to the next
  const int32_t *cu, *pos_offset;
  int batch, total;
  int row_vecs;                  // cache vectors of one token: Hkv * D / elements per vector
  uint32_t row_inv;              // ceil(2^32 / row_vecs); row_vecs > 1
  int tile_tokens;
  int32_t *status;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Larger magnitudes of two pairs, with signs that mean nothing; NaN wins.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// kLanes = lanes that share a row; all lanes of the warp call it.
template <int kLanes>
__device__ __forceinline__ uint4 quantise16(const uint4 &a, const uint4 &b, int &byte) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max_bf16x2(top, w[i]);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) top = max_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, o));
  top &= 0x7fff7fffu;
  // magnitudes as integers: they order like the values, and a NaN is above all
  const uint32_t m = max(top << 16, top & 0xffff0000u);
  if (m > 0x7f800000u) {
    byte = kExpNan;
    return make_uint4(0u, 0u, 0u, 0u);
  }
  const int e = row_exponent(__uint_as_float(m));
  byte = e + kExpBias;
  // 2^-e twice over in bf16: the products are exact, but for values so small that
  // they end as zero all the same (e = 7 alone makes any smaller)
  const uint32_t s = static_cast<uint32_t>(kExpBias - e) * 0x800080u;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = mul_bf16x2(w[2 * i], s), b = mul_bf16x2(w[2 * i + 1], s);
    r[i] = pack_e4m3x4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Four e4m3 bytes -> four bf16 (two registers), times the row's scale.  Every
// step is exact: e4m3 fits f16, and the product fits bf16.
__device__ __forceinline__ uint2 dequantise4(uint32_t w, float scale) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h0) : "h"(static_cast<uint16_t>(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
  float f[4];
  asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;}\n"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(h0));
  asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;}\n"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(h1));
  return make_uint2(tc::pack_bf16x2(f[0] * scale, f[1] * scale), tc::pack_bf16x2(f[2] * scale, f[3] * scale));
}

// A tile: consecutive packed rows, their places found a token to a thread.
struct Tile {
  int32_t seq[kTileTokens];     // sequence of each row, or -1
  int64_t pos[kTileTokens];     // its position there
  int64_t at[kTileTokens];      // element offset in the cache, or one of the two below
  int64_t exp_at[kTileTokens];  // offset of its first head's exponent byte
};
constexpr int64_t kNoRow = -1, kNoPage = -2;

// Rows [row0, row0 + tokens) whose seq and pos are known: their places, then
// the copies, a thread over the tile's cache vectors.  All threads call it,
// after a __syncthreads().
template <bool kWrite, bool kQuant, int D>
__device__ __forceinline__ void copy_tile(const CopyParams &p, Tile &tile, bool is_v, int64_t row0,
                                          int tokens) {
  constexpr int kElems = kQuant ? 16 : 8;     // elements of a cache vector
  constexpr int kLanes = D / kElems;          // vectors (lanes) of a row
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  uint8_t *rows = (is_v ? p.v_rows : p.k_rows) + row0 * stride;
  uint8_t *pages = static_cast<uint8_t *>(is_v ? p.c.v : p.c.k);
  uint8_t *exps = is_v ? p.c.v_exp : p.c.k_exp;
  for (int x = threadIdx.x; x < tokens; x += kThreads) {
    int64_t at = kNoRow, exp_at = 0;
    if (tile.seq[x] >= 0) {
      const int64_t pos = tile.pos[x];
      const int32_t page = __ldg(p.c.table + static_cast<int64_t>(tile.seq[x]) * p.c.table_pages +
                                 (pos >> p.c.page_shift));
      const int row = static_cast<int>(pos) & ((1 << p.c.page_shift) - 1);
      at = kNoPage;
      if (page_ok(p.c, page)) {
        at = row_offset(p.c, page, row, 0);
        exp_at = exp_offset(p.c, page, row, 0);
      } else {
        record_error(p.status, PA_DEVICE_ERR_PAGE);
      }
    }
    tile.at[x] = at;
    tile.exp_at[x] = exp_at;
  }
  __syncthreads();
  const int vecs = tokens * p.row_vecs;
  // the whole warp goes round together (a row's lanes shuffle)
  for (int i0 = threadIdx.x & ~31; i0 < vecs; i0 += kThreads) {
    const int i = i0 + (threadIdx.x & 31);
    // i / row_vecs: i below 2^16 (a tile's vectors), so the rounded-up inverse is exact
    const int jt = i < vecs ? static_cast<int>(__umulhi(i, p.row_inv)) : 0;
    const int vec = i - jt * p.row_vecs;
    const int64_t place = i < vecs ? tile.at[jt] : kNoRow, at = place + vec * kElems;
    const bool live = place >= 0;
    uint4 *r = reinterpret_cast<uint4 *>(rows + jt * stride + vec * (kElems * 2));
    if constexpr (!kQuant) {
      uint4 *cached = reinterpret_cast<uint4 *>(pages + at * 2);
      if (kWrite) {
        if (live) *cached = __ldg(r);
      } else if (place != kNoRow) {
        *r = live ? *cached : make_uint4(0u, 0u, 0u, 0u);
      }
    } else {
      uint4 *cached = reinterpret_cast<uint4 *>(pages + at);
      uint8_t *exp = exps + (live ? tile.exp_at[jt] + ((vec / kLanes) << p.c.page_shift) : 0);
      if (kWrite) {
        uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a;
        if (live) {
          a = __ldg(r);
          c = __ldg(r + 1);
        }
        int byte;
        const uint4 y = quantise16<kLanes>(a, c, byte);
        if (live) {
          *cached = y;
          if (vec % kLanes == 0) *exp = static_cast<uint8_t>(byte);
        }
      } else if (place != kNoRow) {
        uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (live) {
          const uint4 y = *cached;
          const float s = row_scale(*exp);
          const uint2 d0 = dequantise4(y.x, s), d1 = dequantise4(y.y, s), d2 = dequantise4(y.z, s),
                      d3 = dequantise4(y.w, s);
          o[0] = make_uint4(d0.x, d0.y, d1.x, d1.y);
          o[1] = make_uint4(d2.x, d2.y, d3.x, d3.y);
        }
        r[0] = o[0];
        r[1] = o[1];
      }
    }
  }
}

// grid (tiles of the packed rows, K or V).  Every thread looks at its share of
// the sequences for those that the tile cuts; tiles are of the packed rows, not
// of a sequence's, so that one long sequence among many short ones has as many
// CTAs as its rows ask for.
template <bool kWrite, bool kQuant, int D>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const CopyParams p) {
  __shared__ Tile tile;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.tile_tokens;
  const int tokens = min(static_cast<int64_t>(p.tile_tokens), p.total - row0);
  const bool is_v = blockIdx.y == 1, report = blockIdx.x == 0 && !is_v;
  for (int x = threadIdx.x; x < tokens; x += kThreads) tile.seq[x] = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < p.batch; b += kThreads) {
    const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
    const int64_t off = p.pos_offset ? __ldg(p.pos_offset + b) : 0;
    if (c0 < 0 || c0 > c1 || c1 > p.total || (b == 0 && c0 != 0)) {
      if (report) record_error(p.status, PA_DEVICE_ERR_CU_SEQLENS);
    } else if (c0 < c1 &&
               (off < 0 || off + (c1 - c0) > static_cast<int64_t>(p.c.table_pages) << p.c.page_shift)) {
      if (report) record_error(p.status, PA_DEVICE_ERR_MAX_LEN);
    } else {
      const int from = static_cast<int>(max(c0 - row0, int64_t{0}));
      const int to = static_cast<int>(min(c1 - row0, static_cast<int64_t>(tokens)));
      for (int x = from; x < to; ++x) {
        tile.seq[x] = b;
        tile.pos[x] = off + (row0 + x - c0);
      }
    }
  }
  __syncthreads();
  copy_tile<kWrite, kQuant, D>(p, tile, is_v, row0, tokens);
}

// The keys of the long sequences of an attention call over an 8-bit cache as
// bf16 rows, a sequence from a multiple of 128 rows on (flat_page: which).
// grid (CTAs of a sequence, long sequences, K or V).
// The keys of two sequences of 7000, 4 heads of 128: 12 us.
template <int D>
__global__ void __launch_bounds__(kThreads) widen_kernel(const PagedAttnParams a, const CopyParams p) {
  __shared__ Tile tile;
  __shared__ int32_t warp_seqs[kThreads / 32], warp_pages[kThreads / 32], found[3];
  tc::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.y;
  if (threadIdx.x == 0) found[0] = -1;
  // the long sequence of that rank, and the pages of those before it
  int seqs = 0, pages = 0;
  for (int b0 = 0; b0 < a.batch && seqs <= rank; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    PagedSeq s{0, 0, 0};
    int err;
    if (b < a.batch)
      s = paged_seq(a, b, err);
    const bool in = !decode_takes(s.lq, a.G) && chunk_widens(s.lq, a.G);
    const uint32_t all = __ballot_sync(0xffffffffu, in);
    const int mine = in ? (s.lk - 1) / kChunkTile + (s.lk > 0) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) {
      warp_seqs[warp] = __popc(all);
      warp_pages[warp] = incl;
    }
    __syncthreads();
    int at = seqs + __popc(all & ((1u << lane) - 1u)), page = pages + incl - mine;
    for (int x = 0; x < kThreads / 32; ++x) {
      if (x < warp) {
        at += warp_seqs[x];
        page += warp_pages[x];
      }
      seqs += warp_seqs[x];
      pages += warp_pages[x];
    }
    if (in && at == rank) {
      found[0] = b;
      found[1] = page;
      found[2] = s.lk;
      if (blockIdx.x == 0 && blockIdx.z == 0) a.flat_page[b] = page;
    }
    __syncthreads();
  }
  const int b = found[0], page = found[1], lk = found[2];
  if (b < 0 || page + (static_cast<int64_t>(lk) + kChunkTile - 1) / kChunkTile > a.flat_pages) return;
  for (int64_t j0 = static_cast<int64_t>(blockIdx.x) * p.tile_tokens; j0 < lk;
       j0 += static_cast<int64_t>(gridDim.x) * p.tile_tokens) {
    const int tokens = min(static_cast<int64_t>(p.tile_tokens), lk - j0);
    __syncthreads();   // the last tile's places have been read
    for (int x = threadIdx.x; x < tokens; x += kThreads) {
      tile.seq[x] = b;
      tile.pos[x] = j0 + x;
    }
    __syncthreads();
    copy_tile<false, true, D>(p, tile, blockIdx.z == 1, static_cast<int64_t>(page) * kChunkTile + j0,
                              tokens);
  }
}

// K and V of so many tokens as tiles.
void plan_tiles(CopyParams &p, int row_vecs, int64_t tokens, int sms) {
  p.row_vecs = row_vecs;
  p.row_inv = 0xffffffffu / static_cast<uint32_t>(row_vecs) + 1;
  int vecs = kLeastVecs;
  while (vecs < kMostVecs &&
         2 * tokens * row_vecs >= static_cast<int64_t>(2 * vecs) * kTilesPerSm * sms)
    vecs *= 2;
  const int rows = row_vecs >= vecs ? 1 : vecs / row_vecs;
  p.tile_tokens = rows < kTileTokens ? rows : kTileTokens;
}

template <bool kWrite>
pa_status cache_copy(void *k_rows, void *v_rows, const PagedCacheArgs &a, const int32_t *cu,
                     const int32_t *pos_offset, int32_t batch, int32_t total, int64_t k_stride,
                     int64_t v_stride, pa_stream_t stream) {
  if (batch < 1 || total < 0 || !cu) return PA_ERR_INVALID_ARG;
  if (total > 0 && (!k_rows || !v_rows)) return PA_ERR_INVALID_ARG;
  PagedCache c;
  pa_status st = check_cache(a, c);
  if (st != PA_OK) return st;
  const int64_t row = static_cast<int64_t>(a.Hkv) * a.D;
  if (k_stride < row || v_stride < row) return PA_ERR_INVALID_ARG;
  if (batch > 65535) return PA_ERR_UNSUPPORTED;
  if (!aligned_to(k_rows, 16) || !aligned_to(v_rows, 16) || !aligned_to(cu, 4) ||
      !aligned_to(pos_offset, 4) || (k_stride & 7) != 0 || (v_stride & 7) != 0)
    return PA_ERR_MISALIGNED;
  if (total == 0) return PA_OK;
  CopyParams p;
  int sms;
  cudaError_t e = device_context(&p.status, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  const bool quant = a.format == PA_CACHE_E4M3;
  p.c = c;
  p.k_rows = static_cast<uint8_t *>(k_rows);
  p.v_rows = static_cast<uint8_t *>(v_rows);
  p.k_stride = k_stride * 2;
  p.v_stride = v_stride * 2;
  p.cu = cu;
  p.pos_offset = pos_offset;
  p.total = total;
  p.batch = batch;
  plan_tiles(p, static_cast<int>(row / (quant ? 16 : 8)), total, sms);
  const int64_t tiles = (static_cast<int64_t>(total) + p.tile_tokens - 1) / p.tile_tokens;
  const dim3 grid(static_cast<unsigned>(tiles), 2);
  auto s = reinterpret_cast<cudaStream_t>(stream);
  if (quant) {
    if (a.D == 128)
      cache_copy_kernel<kWrite, true, 128><<<grid, kThreads, 0, s>>>(p);
    else
      cache_copy_kernel<kWrite, true, 64><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (a.D == 128)
      cache_copy_kernel<kWrite, false, 128><<<grid, kThreads, 0, s>>>(p);
    else
      cache_copy_kernel<kWrite, false, 64><<<grid, kThreads, 0, s>>>(p);
  }
  return from_cuda(cudaGetLastError());
}

}  // namespace

cudaError_t launch_paged_widen(const PagedAttnParams &a, int num_sms, cudaStream_t stream) {
  CopyParams p;
  p.c = a.c;
  p.k_rows = reinterpret_cast<uint8_t *>(a.flat_k);
  p.v_rows = reinterpret_cast<uint8_t *>(a.flat_v);
  p.k_stride = p.v_stride = static_cast<int64_t>(a.c.Hkv) * a.c.D * 2;
  p.cu = nullptr;
  p.pos_offset = nullptr;
  p.batch = p.total = 0;
  plan_tiles(p, a.c.Hkv * a.c.D / 16, static_cast<int64_t>(a.flat_pages) * kChunkTile, num_sms);
  p.status = a.status;
  int64_t per_seq = (static_cast<int64_t>(num_sms) * 16 + a.flat_seqs - 1) / a.flat_seqs;
  const int64_t most = (static_cast<int64_t>(a.max_k) + p.tile_tokens - 1) / p.tile_tokens;
  if (per_seq > most) per_seq = most;
  const dim3 grid(static_cast<unsigned>(per_seq), a.flat_seqs, 2);
  if (a.c.D == 128)
    widen_kernel<128><<<grid, kThreads, 0, stream>>>(a, p);
  else
    widen_kernel<64><<<grid, kThreads, 0, stream>>>(a, p);
  return cudaGetLastError();
}

pa_status check_cache(const PagedCacheArgs &a, PagedCache &c) {
  if (!a.k || !a.v || !a.table) return PA_ERR_INVALID_ARG;
  if (a.num_pages < 1 || a.page_size < 1 || a.table_pages < 1 || a.Hkv < 1 || a.D < 1)
    return PA_ERR_INVALID_ARG;
  if (a.format != PA_CACHE_BF16 && a.format != PA_CACHE_E4M3) return PA_ERR_INVALID_ARG;
  const bool quant = a.format == PA_CACHE_E4M3;
  if (quant && (!a.k_exp || !a.v_exp)) return PA_ERR_INVALID_ARG;
  if (a.page_size < 16 || a.page_size > 256 || (a.page_size & (a.page_size - 1)) != 0 ||
      (a.D != 64 && a.D != 128) || a.Hkv > 4096)
    return PA_ERR_UNSUPPORTED;
  const int64_t page = static_cast<int64_t>(a.page_size) * a.Hkv * a.D;
  const int64_t elem = quant ? 1 : 2;
  if (a.page_stride < page) return PA_ERR_INVALID_ARG;
  if (a.page_stride > (int64_t{1} << 38)) return PA_ERR_UNSUPPORTED;
  if ((a.page_stride * elem & 15) != 0 || !aligned_to(a.k, 16) || !aligned_to(a.v, 16) ||
      !aligned_to(a.table, 4) || (quant && (!aligned_to(a.k_exp, 16) || !aligned_to(a.v_exp, 16))))
    return PA_ERR_MISALIGNED;
  c.k = a.k;
  c.v = a.v;
  c.k_exp = quant ? a.k_exp : nullptr;
  c.v_exp = quant ? a.v_exp : nullptr;
  c.table = a.table;
  c.page_stride = a.page_stride;
  c.num_pages = a.num_pages;
  c.page_shift = 0;
  while ((1 << c.page_shift) < a.page_size) ++c.page_shift;
  c.table_pages = a.table_pages;
  c.Hkv = a.Hkv;
  c.D = a.D;
  return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_kv_cache_write(const void *k, const void *v, void *k_cache,
                                       void *v_cache, uint8_t *k_exp, uint8_t *v_exp,
                                       const int32_t *cu_seqlens, const int32_t *pos_offset,
                                       const int32_t *page_table, int32_t batch, int32_t total,
                                       int64_t k_stride, int64_t v_stride, int32_t num_pages,
                                       int32_t page_size, int32_t table_pages,
                                       int64_t page_stride, int32_t Hkv, int32_t D,
                                       int32_t format, pa_stream_t stream) {
  const PagedCacheArgs a{k_cache, v_cache, k_exp, v_exp, page_table, num_pages, page_size,
                         table_pages, page_stride, Hkv, D, format};
  return cache_copy<true>(const_cast<void *>(k), const_cast<void *>(v), a, cu_seqlens,
                          pos_offset, batch, total, k_stride, v_stride, stream);
}

extern "C" pa_status pa_kv_cache_read(const void *k_cache, const void *v_cache,
                                      const uint8_t *k_exp, const uint8_t *v_exp, void *k,
                                      void *v, const int32_t *cu_seqlens,
                                      const int32_t *pos_offset, const int32_t *page_table,
                                      int32_t batch, int32_t total, int32_t num_pages,
                                      int32_t page_size, int32_t table_pages,
                                      int64_t page_stride, int32_t Hkv, int32_t D,
                                      int32_t format, pa_stream_t stream) {
  const PagedCacheArgs a{const_cast<void *>(k_cache), const_cast<void *>(v_cache),
                         const_cast<uint8_t *>(k_exp), const_cast<uint8_t *>(v_exp),
                         page_table, num_pages, page_size, table_pages, page_stride, Hkv, D,
                         format};
  const int64_t row = static_cast<int64_t>(Hkv) * D;
  return cache_copy<false>(k, v, a, cu_seqlens, pos_offset, batch, total, row, row, stream);
}
