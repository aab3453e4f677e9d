// Packed rows into a paged K/V cache (quantised to 8 bits as they are
// written, where the cache holds 8-bit rows) and back out of it.
//
// Token j of packed sequence b sits at position pos_offset[b] + j, as in the
// rotary embedding of the same rows; paged.cuh has the layout and the 8-bit
// rows' arithmetic.  Both directions are bound by HBM: every byte is read and
// written once, 16 bytes of cache row to a thread (8 bf16 or 16 e4m3
// elements).  A row's D elements lie in D / 8 (or D / 16) neighbouring lanes,
// so its largest magnitude is a butterfly of 2 to 3 shuffles and the row
// never leaves registers between its load and its store.  GPU time, 8 heads of
// 128: 32k tokens into 8-bit pages 37.6 us (196 MB, 5.2 TB/s: 184 instructions
// for 16 elements keep the schedulers two thirds busy), 106k tokens out of them
// 114 us (651 MB, 5.7 TB/s), 2.4k tokens out of bf16 pages 6.6 us.
#include "internal.h"
#include "paged.cuh"
#include "paged_chunk_work.cuh"
#include "paged_launch.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kTileVecs = 1024;   // cache vectors of a tile: four per thread

struct CopyParams {
  PagedCache c;
  uint8_t *k_rows, *v_rows;      // packed rows, bf16
  int64_t k_stride, v_stride;    // bytes from one token to the next
  const int32_t *cu, *pos_offset;
  int total;
  int row_vecs;                  // cache vectors of one token: Hkv * D / elements per vector
  uint32_t row_inv;              // ceil(2^32 / row_vecs); row_vecs > 1
  int tile_tokens;
  int32_t *status;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

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
  return make_uint2(pack_bf16(f[0] * scale, f[1] * scale), pack_bf16(f[2] * scale, f[3] * scale));
}

// Positions [off, off + n) of sequence b, packed rows from row0 on: the CTAs of
// blockIdx.x stride over tiles of tile_tokens tokens, a thread over a tile's
// cache vectors.
template <bool kWrite, bool kQuant, int D>
__device__ __forceinline__ void copy_rows(const CopyParams &p, int b, bool is_v, int64_t row0,
                                          int64_t off, int n) {
  constexpr int kElems = kQuant ? 16 : 8;     // elements of a cache vector
  constexpr int kLanes = D / kElems;          // vectors (lanes) of a row
  const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.table_pages;
  uint8_t *rows = is_v ? p.v_rows : p.k_rows;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  uint8_t *pages = static_cast<uint8_t *>(is_v ? p.c.v : p.c.k);
  uint8_t *exps = is_v ? p.c.v_exp : p.c.k_exp;
  const int page_mask = (1 << p.c.page_shift) - 1;
  for (int64_t j0 = static_cast<int64_t>(blockIdx.x) * p.tile_tokens; j0 < n;
       j0 += static_cast<int64_t>(gridDim.x) * p.tile_tokens) {
    const int vecs = min(static_cast<int64_t>(p.tile_tokens), n - j0) * p.row_vecs;
    uint8_t *tile_rows = rows + (row0 + j0) * stride;
    const int64_t pos0 = off + j0;
    // the whole warp goes round together (a row's lanes shuffle)
    for (int i0 = threadIdx.x & ~31; i0 < vecs; i0 += kThreads) {
      const int i = i0 + (threadIdx.x & 31);
      const bool on = i < vecs;
      // i / row_vecs: i below 2^16 (a tile's vectors), so the rounded-up inverse is exact
      const int jt = on ? static_cast<int>(__umulhi(i, p.row_inv)) : 0;
      const int vec = on ? i - jt * p.row_vecs : 0;
      const int64_t pos = pos0 + jt;
      const int32_t page = __ldg(table + (pos >> p.c.page_shift));
      const int row = static_cast<int>(pos) & page_mask, head = vec / kLanes;
      const bool good = page_ok(p.c, page);
      if (on && !good) record_error(p.status, PA_DEVICE_ERR_PAGE);
      uint8_t *packed = tile_rows + static_cast<uint32_t>(jt) * stride + vec * (kElems * 2);
      // (a page has at most 256 x 4096 x 128 elements)
      const int64_t at = page * p.c.page_stride + (row * (p.c.Hkv * D) + vec * kElems);
      const bool live = on && good;
      if constexpr (!kQuant) {
        uint4 *cached = reinterpret_cast<uint4 *>(pages + at * 2);
        uint4 *r = reinterpret_cast<uint4 *>(packed);
        if (kWrite) {
          uint4 a = make_uint4(0u, 0u, 0u, 0u);
          if (on) a = __ldg(r);   // while the page is looked up
          if (live) *cached = a;
        } else if (on) {
          *r = good ? *cached : make_uint4(0u, 0u, 0u, 0u);
        }
      } else {
        uint4 *cached = reinterpret_cast<uint4 *>(pages + at);
        uint4 *r = reinterpret_cast<uint4 *>(packed);
        if (kWrite) {
          uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a;
          if (on) {   // while the page is looked up
            a = __ldg(r);
            c = __ldg(r + 1);
          }
          int byte;
          const uint4 y = quantise16<kLanes>(a, c, byte);
          if (live) {
            *cached = y;
            if (vec % kLanes == 0)
              exps[exp_offset(p.c, page, row, head)] = static_cast<uint8_t>(byte);
          }
        } else if (on) {
          uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
          if (good) {
            const uint4 y = *cached;
            const float s = row_scale(exps[exp_offset(p.c, page, row, head)]);
            const uint2 d0 = dequantise4(y.x, s), d1 = dequantise4(y.y, s),
                        d2 = dequantise4(y.z, s), d3 = dequantise4(y.w, s);
            o[0] = make_uint4(d0.x, d0.y, d1.x, d1.y);
            o[1] = make_uint4(d2.x, d2.y, d3.x, d3.y);
          }
          r[0] = o[0];
          r[1] = o[1];
        }
      }
    }
  }
}

// grid (CTAs of a sequence, batch, K or V)
template <bool kWrite, bool kQuant, int D>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const CopyParams p) {
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z == 1;
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  const int64_t off = p.pos_offset ? __ldg(p.pos_offset + b) : 0;
  const bool lead = blockIdx.x == 0 && threadIdx.x == 0 && !is_v;
  if (c0 < 0 || c0 > c1 || c1 > p.total || (b == 0 && c0 != 0)) {
    if (lead) record_error(p.status, PA_DEVICE_ERR_CU_SEQLENS);
    return;
  }
  const int n = c1 - c0;
  if (n == 0) return;
  if (off < 0 || off + n > static_cast<int64_t>(p.c.table_pages) << p.c.page_shift) {
    if (lead) record_error(p.status, PA_DEVICE_ERR_MAX_LEN);
    return;
  }
  copy_rows<kWrite, kQuant, D>(p, b, is_v, c0, off, n);
}

// The keys of the long sequences of an attention call over an 8-bit cache as
// bf16 rows, a sequence from a multiple of 128 rows on (flat_page: which).
// The keys of two sequences of 7000, 4 heads of 128: 12 us.
template <int D>
__global__ void __launch_bounds__(kThreads) widen_kernel(const PagedAttnParams a, const CopyParams p) {
  __shared__ int32_t sums[kThreads / 32];
  tc::griddep_launch_dependents();
  const int b = blockIdx.y;
  int err;
  const PagedSeq s = paged_seq(a.cu_q, a.seq_lens, b, a.total_q, a.max_q, a.max_k, a.capacity, err);
  if (decode_takes(s.lq, a.G) || !chunk_widens(s.lq, a.G)) return;
  int before = 0;   // pages of the long sequences before this one
  for (int x = threadIdx.x; x < b; x += kThreads) {
    const PagedSeq o = paged_seq(a.cu_q, a.seq_lens, x, a.total_q, a.max_q, a.max_k, a.capacity, err);
    if (!decode_takes(o.lq, a.G) && chunk_widens(o.lq, a.G))
      before += (o.lk + kChunkTile - 1) / kChunkTile;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = before;
  __syncthreads();
  int page = 0;
#pragma unroll
  for (int x = 0; x < kThreads / 32; ++x) page += sums[x];
  if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) a.flat_page[b] = page;
  if (page + static_cast<int64_t>(s.lk + kChunkTile - 1) / kChunkTile > a.flat_pages) return;
  copy_rows<false, true, D>(p, b, blockIdx.z == 1, static_cast<int64_t>(page) * kChunkTile, 0, s.lk);
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
  p.row_vecs = static_cast<int>(row / (quant ? 16 : 8));
  p.row_inv = 0xffffffffu / static_cast<uint32_t>(p.row_vecs) + 1;
  p.tile_tokens = p.row_vecs >= kTileVecs ? 1 : kTileVecs / p.row_vecs;
  // as many tiles as the longest sequence can have, at most eight CTAs per SM over the call
  int64_t per_seq = (static_cast<int64_t>(sms) * 8 + batch - 1) / batch;
  const int64_t most = (static_cast<int64_t>(total) + p.tile_tokens - 1) / p.tile_tokens;
  if (per_seq > most) per_seq = most;
  const dim3 grid(static_cast<unsigned>(per_seq), batch, 2);
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
  p.total = 0;
  p.row_vecs = a.c.Hkv * a.c.D / 16;
  p.row_inv = 0xffffffffu / static_cast<uint32_t>(p.row_vecs) + 1;
  p.tile_tokens = p.row_vecs >= kTileVecs ? 1 : kTileVecs / p.row_vecs;
  p.status = a.status;
  int64_t per_seq = (static_cast<int64_t>(num_sms) * 8 + a.batch - 1) / a.batch;
  const int64_t most = (static_cast<int64_t>(a.max_k) + p.tile_tokens - 1) / p.tile_tokens;
  if (per_seq > most) per_seq = most;
  const dim3 grid(static_cast<unsigned>(per_seq), a.batch, 2);
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
