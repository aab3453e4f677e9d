// Joins what the paged attention kernels left in parts: rows whose keys were
// split over several warps (paged_decode.cu) and items that shares of the
// tiled kernel cut (paged_chunk.cu).  A part is an unnormalised output, the
// maximum it was taken against and the sum of its weights:
//   out = sum_n 2^(m_n - m) o_n / sum_n 2^(m_n - m) l_n,   m = max_n m_n.
// Bound by latency, then by L2: 2048 rows of 17 parts take some 8 us, 6144 rows
// of 27 (85 MB) 12, 32 rows of 228 parts 9.
#include <math.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_chunk_work.cuh"
#include "paged_launch.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

// Warps of a CTA: one for each sum of a row, or few, for short CTAs in numbers.
template <bool kWide>
constexpr int kWarps = kWide ? kJoinSums : 4;

// A lane's D / 32 values of a part's row.
template <int E>
__device__ __forceinline__ void load_row(float (&o)[E], const float *src) {
  if constexpr (E == 4) {
    const float4 y = *reinterpret_cast<const float4 *>(src);
    o[0] = y.x;
    o[1] = y.y;
    o[2] = y.z;
    o[3] = y.w;
  } else {
    const float2 y = *reinterpret_cast<const float2 *>(src);
    o[0] = y.x;
    o[1] = y.y;
  }
}
template <int E>
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, const float (&o)[E], float inv) {
  uint32_t *d = reinterpret_cast<uint32_t *>(dst);
#pragma unroll
  for (int e = 0; e < E; e += 2) d[e / 2] = tc::pack_bf16x2(o[e] * inv, o[e + 1] * inv);
}

// Row `row` (token * Hq + head) of sequence b of the streaming kernel.  The
// parts go to eight sums in turn, and these are added in order: by eight warps
// that have a sum each (kWide: few rows with many parts; one sequence with 228
// parts and 32 rows takes 92 us in all, 102 with four warps to a row), or by
// one warp that has them all (many rows with few parts).  The same bits
// either way.
template <int D, bool kWide>
__device__ __forceinline__ void join_row(const PagedAttnParams &p, int b, int row) {
  constexpr int E = D / 32;
  __shared__ float acc_s[kWide ? kJoinSums : 1][D];
  __shared__ float sum_s[kJoinSums];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int err;
  const PagedSeq s = paged_seq(p, b, err);
  if (!decode_takes(s.lq, p.G) || row >= s.lq * p.Hq) return;
  const int parts = decode_split(s.lk, row_groups(s.lq, p.G), p.dec_most).parts;
  if (parts <= 1) return;
  const int64_t slot0 = b * p.dec_slots + row;
  auto slot_of = [&](int n) { return slot0 + static_cast<int64_t>(n) * (s.lq * p.Hq); };
  float top = -INFINITY;
  for (int n = lane; n < parts; n += 32) top = fmaxf(top, p.dec_ml[slot_of(n)].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float ref = top == -INFINITY ? 0.f : top;

  // eight parts in flight: of this warp's sum, or one of each sum
  constexpr int kOwn = kWide ? 1 : kJoinSums;
  float acc[kOwn][E], sum[kOwn];
#pragma unroll
  for (int y = 0; y < kOwn; ++y) {
    sum[y] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[y][e] = 0.f;
  }
  constexpr int kStep = kWide ? kJoinSums : 1;
  for (int n0 = kWide ? warp : 0; n0 < parts; n0 += 8 * kStep) {
    float2 v[8];
    float o[8][E];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int n = n0 + x * kStep;
      v[x] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[x][e] = 0.f;
      if (n < parts) {
        v[x] = p.dec_ml[slot_of(n)];
        load_row<E>(o[x], p.dec_o + slot_of(n) * D + lane * E);
      }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float f = tc::ex2(v[x].x - ref);
      sum[x % kOwn] += f * v[x].y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[x % kOwn][e] += f * o[x][e];
    }
  }
  float total = 0.f, out[E];
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = 0.f;
  if constexpr (kWide) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc_s[warp][lane * E + e] = acc[0][e];
    if (lane == 0) sum_s[warp] = sum[0];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int y = 0; y < kJoinSums; ++y) {
      total += sum_s[y];
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] += acc_s[y][lane * E + e];
    }
  } else {
#pragma unroll
    for (int y = 0; y < kJoinSums; ++y) {
      total += sum[y];
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] += acc[y][e];
    }
  }
  // a maximum of -inf: no key seen (0), or a NaN score (stays NaN)
  store_row<E>(p.out + (static_cast<int64_t>(s.q0) * p.Hq + row) * D + lane * E, out,
               top == -INFINITY ? 0.f : 1.f / total);
}

// 32 columns of 32 rows, a row to a lane, of the item that cut `cut` begins
// (parts lie column by column there, four at a time).  What the tiled kernel
// noted is checked against the call before it is used, so that a call that
// gave up (a wait that ran out) reads nothing out of place.
template <int D>
__device__ __forceinline__ void join_item_block(const PagedAttnParams &p, int cut, int block) {
  constexpr int kCols = 8;   // of four
  const int r = block / (D / 32) * 32 + (threadIdx.x & 31), c0 = block % (D / 32) * kCols;
  const int4 a = p.chunk_join[2 * static_cast<int64_t>(cut)];
  const int4 c = p.chunk_join[2 * static_cast<int64_t>(cut) + 1];
  // part 0 at row a.y of the workspace, part 1 one part further, then every second or
  // the next (chunk_slots)
  const int parts = a.x, rows = c.x, part_rows = a.z;
  auto first_row = [&](int n) -> int64_t {
    return a.y + static_cast<int64_t>(a.w || n == 0 ? n : 2 * n - 1) * part_rows;
  };
  if (parts < 2 || parts > kChunkShares + 1 || rows < 1 || part_rows < rows ||
      part_rows > 2 * kChunkTile || a.y < 0 ||
      first_row(parts - 1) + part_rows > p.chunk_rows || c.y < 0 ||
      rows % p.G != 0 ||
      c.y + static_cast<int64_t>(rows) / p.G > p.total_q || c.z < 0 || c.z >= p.c.Hkv || r >= rows)
    return;
  float top = -INFINITY;
  for (int n = 0; n < parts; ++n) top = fmaxf(top, p.chunk_ml[first_row(n) + r].x);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  float4 acc[kCols];
#pragma unroll
  for (int x = 0; x < kCols; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int n = 0; n < parts; ++n) {
    const float2 v = p.chunk_ml[first_row(n) + r];
    const float4 *src =
        reinterpret_cast<const float4 *>(p.chunk_o + first_row(n) * D) + c0 * part_rows + r;
    const float f = tc::ex2(v.x - ref);
    sum += f * v.y;
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
      const float4 o = src[x * part_rows];
      acc[x].x += f * o.x;
      acc[x].y += f * o.y;
      acc[x].z += f * o.z;
      acc[x].w += f * o.w;
    }
  }
  const float inv = top == -INFINITY ? 0.f : 1.f / sum;
  const int tok = r / p.G;
  uint4 *dst = reinterpret_cast<uint4 *>(
      p.out + (static_cast<int64_t>(c.y + tok) * p.Hq + c.z * p.G + (r - tok * p.G)) * D + c0 * 4);
#pragma unroll
  for (int x = 0; x < kCols; x += 2)
    dst[x / 2] = make_uint4(tc::pack_bf16x2(acc[x].x * inv, acc[x].y * inv),
                            tc::pack_bf16x2(acc[x].z * inv, acc[x].w * inv),
                            tc::pack_bf16x2(acc[x + 1].x * inv, acc[x + 1].y * inv),
                            tc::pack_bf16x2(acc[x + 1].z * inv, acc[x + 1].w * inv));
}

// CTAs [0, dec_ctas) join rows of the streaming kernel, dec_per_seq of them to
// a sequence; the others go round the rows of all cut items.
template <int D, bool kWide>
__global__ void __launch_bounds__(kWarps<kWide> * 32)
    paged_join_kernel(const PagedAttnParams p, int dec_per_seq, int dec_ctas) {
  tc::griddep_wait();
  const int warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < dec_ctas) {
    const int b = blockIdx.x / dec_per_seq, x = blockIdx.x - b * dec_per_seq;
    join_row<D, kWide>(p, b, kWide ? x : x * kWarps<kWide> + warp);
    return;
  }
  // the cuts of one launch of the tiled kernel, or of two
  const int sets = p.flat_pages > 0 ? 2 : 1;
  for (int set = 0; set < sets; ++set) {
    const int from = set ? p.chunk_cut0_rest : 0, to = min(p.chunk_n_cuts[set], p.chunk_cuts);
    constexpr int kBlocks = 2 * kChunkTile / 32 * (D / 32);   // of an item
    for (int x = (blockIdx.x - dec_ctas) * kWarps<kWide> + warp; x < (to - from) * kBlocks;
         x += (gridDim.x - dec_ctas) * kWarps<kWide>)
      join_item_block<D>(p, from + x / kBlocks, x % kBlocks);
  }
}

template <int D, bool kWide>
cudaError_t launch(const PagedAttnParams &p, int num_sms, cudaStream_t stream) {
  const int per_seq = p.dec_parts <= 1 ? 0
                      : kWide          ? p.dec_rows
                                       : (p.dec_rows + kWarps<kWide> - 1) / kWarps<kWide>;
  const int dec_ctas = per_seq * p.batch;
  const int64_t cut_ctas =
      static_cast<int64_t>(p.chunk_cuts) * (2 * kChunkTile / 32 * (D / 32) / kWarps<kWide>);
  const int most = num_sms * (kWide ? 6 : 12);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(dec_ctas + static_cast<int>(cut_ctas < most ? cut_ctas : most));
  cfg.blockDim = dim3(kWarps<kWide> * 32);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kWide>, p, per_seq, dec_ctas);
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnParams &p, int num_sms, cudaStream_t stream) {
  // Many parts are worth eight warps to a row where the rows are few; where they are
  // many a warp each fills the GPU, and the bound on the parts may be far above
  // what the sequences have (64 of 900-8000 keys, bounds of 131,072: 191 us with
  // eight warps to a row, 184 with one).
  const bool wide = p.dec_parts > 64 && static_cast<int64_t>(p.batch) * p.dec_rows <= 1024;
  if (p.c.D == 128)
    return wide ? launch<128, true>(p, num_sms, stream) : launch<128, false>(p, num_sms, stream);
  return wide ? launch<64, true>(p, num_sms, stream) : launch<64, false>(p, num_sms, stream);
}

}  // namespace pa
