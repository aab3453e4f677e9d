// Paged attention of sequences with few query rows: single-token steps, and
// steps of a few tokens (up to 16 rows of one K/V head's group).
//
// Bound by the cache's bytes: each is used for 2 to 16 rows only.  So the
// kernel is built around a stream of loads that never waits for anything: a
// unit is one (sequence, K/V head, part of the keys), its four warps take
// 16-key tiles in turn, and every lane fetches, with 16-byte cp.async into
// slots of its own, exactly the bytes that it later feeds to the tensor core
// from registers.  Nothing in the loop waits for another warp, no
// swizzle or transposing load is needed, and a tile needs no staging beyond
// the slots, three to four tiles deep.
//
// The products run with the keys as the M side of m16n8k16 MMAs, so that 8
// query rows fill a tile (N = 8) that 16 rows of padding would waste:
//   S^T [16 keys, 8 rows] = K [16 keys, D] Q^T
//   O^T [D, 8 rows]      += V^T [D, 16 keys] P^T [16 keys, 8 rows]
// The sum over D may run in any order as long as K and Q agree, so a lane
// takes its four (e4m3: four) values of a k-step from one 16-byte vector of a
// row; V^T's rows may be numbered in any order too, so a lane's V values come
// from one 16-byte vector of each of its four keys, paired by byte permutes.
// P^T's B operand is S^T's accumulator transposed in 8x8 blocks (movmatrix).
//
// 8-bit rows are widened in registers (paged.cuh).
#include <math.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_launch.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTileKeys = 16;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays below 2^8

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
template <int D, bool kQuant, int NT>
struct Cfg {
  static constexpr int kRowBytes = D * (kQuant ? 1 : 2);
  static constexpr int kKVecs = kRowBytes / 32;             // a lane's 16-byte K vectors of a tile
  static constexpr int kVBytes = kRowBytes >= 128 ? 16 : 8; // a lane's V vector
  static constexpr int kVSets = kRowBytes / (8 * kVBytes);  // vectors of one key
  static constexpr int kTileBytes = 16 * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes + (kQuant ? 128 : 0);
  static constexpr int kStages = kQuant ? 4 : 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kPitch = D + 4;                      // floats of a merged row
  static constexpr int kMergeBytes = kWarps * kRows * (kPitch + 2) * 4;
  static constexpr int kSmem = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
};

template <int D, bool kQuant, int NT>
__global__ void __launch_bounds__(kThreads) paged_decode_kernel(const PagedAttnParams p) {
  using C = Cfg<D, kQuant, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.y, hk = blockIdx.x % p.c.Hkv, part = blockIdx.x / p.c.Hkv;
  const int64_t cap = static_cast<int64_t>(p.c.table_pages) << p.c.page_shift;
  int err;
  const PagedSeq s = paged_seq(p.cu_q, p.seq_lens, b, p.total_q, p.max_q, p.max_k, cap, err);
  if (err && blockIdx.x == 0 && tid == 0) record_error(p.status, err);
  const int R = s.lq * p.G;
  if (s.lq == 0 || s.lq > kDecodeRows / p.G) return;
  const int keys_part = decode_part(s.lk, p.c.Hkv);
  const int parts = decode_parts(s.lk, p.c.Hkv);
  if (part > 0 && part >= parts) return;   // part 0 of a sequence without keys writes its zeros
  const int k0 = part * keys_part, k1 = k0 + min(s.lk - k0, keys_part);

  // ---- Q^T, the B operand of every S^T product
  uint32_t qf[NT][D / 16][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
    const bool live = r < R;
    const int i = live ? r / p.G : 0, gg = live ? r - i * p.G : 0;
    const __nv_bfloat16 *row =
        p.q + (s.q0 + i) * p.q_stride + static_cast<int64_t>(hk * p.G + gg) * D;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint2 w = make_uint2(0u, 0u);
      // four values: of vector t + 4 (ks / 2) (bf16) or t + 4 (ks / 4) (e4m3)
      const int d = kQuant ? (t + 4 * (ks >> 2)) * 16 + (ks & 3) * 4
                           : (t + 4 * (ks >> 1)) * 8 + (ks & 1) * 4;
      if (live) w = __ldg(reinterpret_cast<const uint2 *>(row + d));
      if (kQuant) {   // the widened bytes come as values 0, 2 and 1, 3
        qf[nt][ks][0] = __byte_perm(w.x, w.y, 0x5410);
        qf[nt][ks][1] = __byte_perm(w.x, w.y, 0x7632);
      } else {
        qf[nt][ks][0] = w.x;
        qf[nt][ks][1] = w.y;
      }
    }
  }
  // last key + 1 that each of this lane's columns (rows of q) sees
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * t + e;
      lim[nt][e] = r >= R ? 0 : p.causal ? s.lk - s.lq + 1 + r / p.G : s.lk;
    }
  const int all_see = p.causal ? s.lk - s.lq + 1 : s.lk;   // keys before it need no mask

  float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  // ---- this warp's tiles: warp, warp + 4, ... of the part
  const int part_tiles = k1 > k0 ? (k1 - k0 + kTileKeys - 1) / kTileKeys : 0;
  const int n_tiles = part_tiles > warp ? (part_tiles - warp + kWarps - 1) / kWarps : 0;
  const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.table_pages;
  const int page_mask = (1 << p.c.page_shift) - 1;
  const int64_t row_stride = static_cast<int64_t>(p.c.Hkv) * C::kRowBytes;
  const uint8_t *kbase = static_cast<const uint8_t *>(p.c.k) + hk * C::kRowBytes;
  const uint8_t *vbase = static_cast<const uint8_t *>(p.c.v) + hk * C::kRowBytes;
  uint8_t *ring = smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_u = tc::smem_u32(ring);

  // pages of 32 tiles at a time, one per lane (a tile lies inside one page)
  auto tile_key = [&](int n) { return k0 + (n * kWarps + warp) * kTileKeys; };
  auto load_pages = [&](int n0) -> int32_t {
    const int n = n0 + lane;
    return n < n_tiles ? __ldg(table + (tile_key(n) >> p.c.page_shift)) : 0;
  };
  int32_t pages = load_pages(0), pages_next = load_pages(32);

  auto issue = [&](int n) {
    if (n < n_tiles) {
      if (n > 0 && (n & 31) == 0) {
        pages = pages_next;
        pages_next = load_pages(n + 32);
      }
      int32_t page = __shfl_sync(0xffffffffu, pages, n & 31);
      bool good = page_ok(p.c, page);
      if (!good) {
        if (lane == 0) record_error(p.status, PA_DEVICE_ERR_PAGE);
        page = 0;
      }
      const int key = tile_key(n);
      const int have = good ? s.lk - key : 0;   // rows of the tile that are the sequence's
      const int row0 = key & page_mask;
      const int64_t at = (page * p.c.page_stride) * (kQuant ? 1 : 2) + row0 * row_stride;
      const uint32_t dst = ring_u + (n % C::kStages) * C::kStageBytes;
#pragma unroll
      for (int v = 0; v < C::kKVecs; ++v) {
        const int row = (v & 1) * 8 + g, chunk = t + 4 * (v >> 1);
        cp_async16(dst + v * 512 + lane * 16, kbase + at + row * row_stride + chunk * 16,
                   row < have ? 16 : 0);
      }
#pragma unroll
      for (int v = 0; v < 4 * C::kVSets; ++v) {
        const int row = 2 * t + (v & 1) + 8 * ((v >> 1) & 1), chunk = g + 8 * (v >> 2);
        const uint8_t *src = vbase + at + row * row_stride + chunk * C::kVBytes;
        const uint32_t to = dst + C::kTileBytes + v * (32 * C::kVBytes) + lane * C::kVBytes;
        if (C::kVBytes == 16)
          cp_async16(to, src, row < have ? 16 : 0);
        else
          cp_async8(to, src, row < have ? 8 : 0);
      }
      if (kQuant && lane < 2) {
        const uint8_t *e = lane == 0 ? p.c.k_exp : p.c.v_exp;
        cp_async16(dst + 2 * C::kTileBytes + lane * 16, e + exp_offset(p.c, page, row0, hk),
                   good ? 16 : 0);
      }
    }
    cp_async_commit();
  };

#pragma unroll
  for (int n = 0; n < C::kStages - 1; ++n) issue(n);

  for (int n = 0; n < n_tiles; ++n) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();                       // the exponents come from other lanes' copies
    issue(n + C::kStages - 1);          // into the slots that tile n - 1 has left
    const uint8_t *st = ring + (n % C::kStages) * C::kStageBytes;
    const int key = tile_key(n);

    // S^T = K Q^T
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
    if constexpr (!kQuant) {
#pragma unroll
      for (int i = 0; i < C::kKVecs / 2; ++i) {
        const uint4 a = *reinterpret_cast<const uint4 *>(st + (2 * i) * 512 + lane * 16);
        const uint4 c = *reinterpret_cast<const uint4 *>(st + (2 * i + 1) * 512 + lane * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(sc[nt], a.x, c.x, a.y, c.y, qf[nt][2 * i][0], qf[nt][2 * i][1]);
          mma16816(sc[nt], a.z, c.z, a.w, c.w, qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
        }
      }
    } else {
      const uint8_t *ex = st + 2 * C::kTileBytes;
      const uint32_t s0 = widen_scale(ex[g]) * 0x10001u, s8 = widen_scale(ex[g + 8]) * 0x10001u;
#pragma unroll
      for (int i = 0; i < C::kKVecs / 2; ++i) {
        const uint4 a = *reinterpret_cast<const uint4 *>(st + (2 * i) * 512 + lane * 16);
        const uint4 c = *reinterpret_cast<const uint4 *>(st + (2 * i + 1) * 512 + lane * 16);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = mul_bf16x2(even_bytes(aw[w]), s0), a2 = mul_bf16x2(odd_bytes(aw[w]), s0);
          const uint32_t a1 = mul_bf16x2(even_bytes(cw[w]), s8), a3 = mul_bf16x2(odd_bytes(cw[w]), s8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(sc[nt], a0, a1, a2, a3, qf[nt][4 * i + w][0], qf[nt][4 * i + w][1]);
        }
      }
    }

    // online softmax over the tile's keys, all lanes of a column in step
    uint32_t pf[NT][2];
    bool moved = false;
    float alpha[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] *= p.scale_log2;
      if (key + kTileKeys > all_see) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key + g + 8 * (e >> 1) >= lim[nt][e & 1]) sc[nt][e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(sc[nt][e], sc[nt][e + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        alpha[nt][e] = 1.f;
        if (mx > m[nt][e] + kRescaleThreshold) {   // from -inf: any finite score
          alpha[nt][e] = tc::ex2(m[nt][e] - mx);
          m[nt][e] = mx;
          moved = true;
        }
        const float base = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
        const float p0 = tc::ex2(sc[nt][e] - base), p1 = tc::ex2(sc[nt][e + 2] - base);
        l[nt][e] = l[nt][e] * alpha[nt][e] + (p0 + p1);
        sc[nt][e] = p0;
        sc[nt][e + 2] = p1;
      }
      pf[nt][0] = transpose8x8(tc::pack_bf16x2(sc[nt][0], sc[nt][1]));
      pf[nt][1] = transpose8x8(tc::pack_bf16x2(sc[nt][2], sc[nt][3]));
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][mt][e] *= alpha[nt][e & 1];
    }

    // O^T += V^T P^T
    const uint8_t *sv = st + C::kTileBytes;
    if constexpr (!kQuant) {
#pragma unroll
      for (int cs = 0; cs < C::kVSets; ++cs) {
        uint4 v[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          v[kk] = *reinterpret_cast<const uint4 *>(sv + (cs * 4 + kk) * 512 + lane * 16);
        const uint32_t va[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w},
                                   {v[1].x, v[1].y, v[1].z, v[1].w},
                                   {v[2].x, v[2].y, v[2].z, v[2].w},
                                   {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = __byte_perm(va[0][w], va[1][w], 0x5410);
          const uint32_t a1 = __byte_perm(va[0][w], va[1][w], 0x7632);
          const uint32_t a2 = __byte_perm(va[2][w], va[3][w], 0x5410);
          const uint32_t a3 = __byte_perm(va[2][w], va[3][w], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[nt][cs * 4 + w], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
      }
    } else {
      const uint8_t *ex = st + 2 * C::kTileBytes + 16;
      uint32_t sc4[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int row = 2 * t + (kk & 1) + 8 * (kk >> 1);
        // a NaN byte of a row past the end must not meet its zeros
        sc4[kk] = key + row < s.lk ? widen_scale(ex[row]) : 0u;
      }
      const uint32_t s0 = sc4[0] | (sc4[1] << 16), s8 = sc4[2] | (sc4[3] << 16);
      uint32_t va[4][C::kVBytes / 4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if constexpr (C::kVBytes == 16) {
          const uint4 v = *reinterpret_cast<const uint4 *>(sv + kk * 512 + lane * 16);
          va[kk][0] = v.x;
          va[kk][1] = v.y;
          va[kk][2] = v.z;
          va[kk][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(sv + kk * 256 + lane * 8);
          va[kk][0] = v.x;
          va[kk][1] = v.y;
        }
      }
#pragma unroll
      for (int w = 0; w < C::kVBytes / 4; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // values 0, 1, then 2, 3 of the word
          const uint32_t ab = __byte_perm(va[0][w], va[1][w], half ? 0x7632 : 0x5410);
          const uint32_t cd = __byte_perm(va[2][w], va[3][w], half ? 0x7632 : 0x5410);
          const uint32_t a0 = mul_bf16x2(even_bytes(ab), s0), a1 = mul_bf16x2(odd_bytes(ab), s0);
          const uint32_t a2 = mul_bf16x2(even_bytes(cd), s8), a3 = mul_bf16x2(odd_bytes(cd), s8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[nt][2 * w + half], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
      }
    }
  }
  tc::griddep_launch_dependents();

  // ---- join the four warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
  cp_async_wait<0>();
  __syncthreads();
  float *mo = reinterpret_cast<float *>(smem);                       // [warp][row][pitch]
  float2 *ml = reinterpret_cast<float2 *>(mo + kWarps * C::kRows * C::kPitch);   // [warp][row]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * t + e;
      float *dst = mo + (warp * C::kRows + r) * C::kPitch;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        const int d = !kQuant && D == 128 ? g * 8 + 64 * (mt >> 2) + 2 * (mt & 3)
                                          : g * (D / 8) + 2 * mt;
        *reinterpret_cast<float2 *>(dst + d) = make_float2(o[nt][mt][e], o[nt][mt][e + 2]);
      }
      if (g == 0) ml[warp * C::kRows + r] = make_float2(m[nt][e], l[nt][e]);
    }
  }
  __syncthreads();
  for (int x = tid; x < R * (D / 4); x += kThreads) {
    const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + r].x);
    const float base = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = ml[w * C::kRows + r];
      const float f = tc::ex2(v.x - base);
      const float4 a = *reinterpret_cast<const float4 *>(mo + (w * C::kRows + r) * C::kPitch + d);
      sum += f * v.y;
      acc.x += f * a.x;
      acc.y += f * a.y;
      acc.z += f * a.z;
      acc.w += f * a.w;
    }
    const int i = r / p.G, h = hk * p.G + r - i * p.G;
    if (parts <= 1) {
      const float inv = top == -INFINITY ? 0.f : 1.f / sum;
      const uint2 w = make_uint2(tc::pack_bf16x2(acc.x * inv, acc.y * inv),
                                 tc::pack_bf16x2(acc.z * inv, acc.w * inv));
      *reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(s.q0 + i) * p.Hq + h) * D + d) = w;
    } else {
      const int64_t slot = (static_cast<int64_t>(b) * p.dec_parts + part) * p.dec_rows +
                           static_cast<int64_t>(i) * p.Hq + h;
      *reinterpret_cast<float4 *>(p.dec_o + slot * D + d) = acc;
      if (d == 0) p.dec_ml[slot] = make_float2(top, sum);
    }
  }
}

// Joins the parts of every row that has more than one: a CTA per row, its four
// warps over the parts, a lane over D / 32 dims.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_combine_kernel(const PagedAttnParams p) {
  constexpr int E = D / 32;
  __shared__ float acc_s[kWarps][D];
  __shared__ float sum_s[kWarps];
  tc::griddep_wait();
  const int b = blockIdx.y, row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cap = static_cast<int64_t>(p.c.table_pages) << p.c.page_shift;
  int err;
  const PagedSeq s = paged_seq(p.cu_q, p.seq_lens, b, p.total_q, p.max_q, p.max_k, cap, err);
  if (s.lq > kDecodeRows / p.G || row >= s.lq * p.Hq) return;
  const int parts = decode_parts(s.lk, p.c.Hkv);
  if (parts <= 1) return;
  const int64_t slot0 = static_cast<int64_t>(b) * p.dec_parts * p.dec_rows + row;
  float top = -INFINITY;
  for (int n = lane; n < parts; n += 32)
    top = fmaxf(top, p.dec_ml[slot0 + static_cast<int64_t>(n) * p.dec_rows].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float base = top == -INFINITY ? 0.f : top;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int n = warp; n < parts; n += kWarps) {
    const int64_t slot = slot0 + static_cast<int64_t>(n) * p.dec_rows;
    const float2 v = p.dec_ml[slot];
    const float f = tc::ex2(v.x - base);
    sum += f * v.y;
    const float *src = p.dec_o + slot * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * src[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc_s[warp][lane * E + e] = acc[e];
  if (lane == 0) sum_s[warp] = sum;
  __syncthreads();
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    const float total = sum_s[0] + sum_s[1] + sum_s[2] + sum_s[3];
    const float v = acc_s[0][d] + acc_s[1][d] + acc_s[2][d] + acc_s[3][d];
    p.out[(static_cast<int64_t>(s.q0) * p.Hq + row) * D + d] =
        __float2bfloat16(v * (top == -INFINITY ? 0.f : 1.f / total));   // NaN stays NaN
  }
}

template <int D, bool kQuant, int NT>
cudaError_t launch(const PagedAttnParams &p, cudaStream_t stream) {
  constexpr int smem = Cfg<D, kQuant, NT>::kSmem;
  static unsigned long long configured = 0;
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(paged_decode_kernel<D, kQuant, NT>),
                                smem, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.dec_parts) * p.c.Hkv, p.batch);
  paged_decode_kernel<D, kQuant, NT><<<grid, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.dec_parts == 1) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.dec_rows, p.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D>, p);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedAttnParams &p, bool quant, cudaStream_t stream) {
  // 8 columns where no sequence of the call can have more rows: a column's
  // results do not depend on the others, so this changes no bits
  const int most = p.max_q < kDecodeRows / p.G ? p.max_q * p.G : kDecodeRows / p.G * p.G;
  const bool wide = most > 8;
  if (p.c.D == 128) {
    if (quant) return wide ? launch<128, true, 2>(p, stream) : launch<128, true, 1>(p, stream);
    return wide ? launch<128, false, 2>(p, stream) : launch<128, false, 1>(p, stream);
  }
  if (quant) return wide ? launch<64, true, 2>(p, stream) : launch<64, true, 1>(p, stream);
  return wide ? launch<64, false, 2>(p, stream) : launch<64, false, 1>(p, stream);
}

}  // namespace pa
