// Rotary positions with several axes, on packed q and k.
//
// An image or video token has a position per axis (time, height, width), and
// every axis turns pairs of its own: pair i of the rotated width R (the sum of
// the axes' widths) belongs to axis a, and
//   (x, y) -> (x cos z - y sin z, x sin z + y cos z),   z = positions[a, t] theta_i
// for its two elements, 2i and 2i + 1 or (halves) i and i + R/2.  theta_i is
// base^(-2 j / dim_a), j the pair's place on its axis, or (shared) base^(-2 i / R).
//
// Angles: theta_i / (2 pi) is kept as a 64-bit fraction of a turn (computed in
// double on the host), so position * fraction modulo 2^64 is the fraction of a
// turn that is left, with no error but the fraction's own (theta's 2^-52 at most,
// times the position) and no double-precision arithmetic on the GPU.  sincospif then
// has an argument in [-1, 1).
//
// HBM bound: q and k are read and written once.  A warp's task is a token and
// its heads, or a share of them where the tokens are too few to fill the SMs.  A
// lane has a fixed place in its head, a vector of eight elements (with halves,
// the two vectors of its pairs), so its fractions stay in registers and its cos
// and sin, computed while the task's first loads are in flight, serve all of
// the task's heads; lanes at one place of several heads compute a part each.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "sched.cuh"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;      // 8 warps, a task each
constexpr int kMaxPairs = 128;     // D <= 256: the lanes of a warp cover a head
constexpr int kMaxAxes = 8;

struct RopeParams {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  const int32_t *positions;     // [axes, total]
  const int32_t *num_tokens;    // rows from here on are left alone, or nullptr
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int total, Hq, Hkv, D;
  int width;                    // R
  int units;                    // lanes of a head
  int heads_per_step;
  int chunks, steps;            // tasks of a token, and the steps of one
  uint64_t turn[kMaxPairs];     // theta_i / (2 pi), in 2^-64
  uint8_t axis[kMaxPairs];
};

template <int kElems>
struct Vec;
template <>
struct Vec<8> {
  using type = uint4;
};
template <>
struct Vec<4> {
  using type = uint2;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// cos and sin of position * theta.
__device__ __forceinline__ float2 turned(int32_t position, uint64_t turn) {
  const uint64_t left = static_cast<uint64_t>(static_cast<int64_t>(position)) * turn;
  // [-1/2, 1/2) of a turn, as half turns
  const float half_turns = __ll2float_rn(static_cast<int64_t>(left)) * 0x1p-63f;
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

// A call of many tokens has tasks of whole tokens, or nearly, for all SMs; where there
// are few it is the latency of a task that counts.  With 24 warps an SM:
//   heads of a lane at a time: 6, or with halves 3 where tokens are many (9801 of 32
//   heads of 80: 16.7 us, by two 18.2; 20000 of 40 heads of 128 65.3 and 67.8) and 2
//   where they are few (48 of 40 heads of 128: 2.2 us, by three 3.2);
//   cos and sin computed once for all heads of a step, but for many tokens without
//   halves (48 tokens of 48 heads of 128: 2.5 us, each lane its own 2.8; 3000 14.3
//   and 12.2).
// (One call in a row of them in a graph, over rows in L2.)  30269 tokens of 48 heads
// of 128: 115 us out of HBM, 6.4 TB/s.  9801 tokens of 32 heads of 80, halves: 20 us of 15
// that the bytes take; 8 blocks an SM are launched, of which 3 are resident, so nearly
// every warp has one task, and blocks turn over with nothing in flight between them.
constexpr int batch_of(bool halves, bool many) { return !halves ? 6 : many ? 3 : 2; }

// kHalves: pairs (i, i + R/2), else (2i, 2i + 1).  kElems: elements of a vector.
// kOwn: pairs of a lane whose cos and sin it computes itself; the lanes at the same
// place of the step's other heads have the rest.  kBatch: heads of a lane at a time.
template <bool kHalves, int kElems, int kOwn, int kBatch>
__global__ void __launch_bounds__(kThreads, 3) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  using V = typename Vec<kElems>::type;
  constexpr int kPairs = kHalves ? kElems : kElems / 2;   // of a lane
  const int lane = threadIdx.x & 31;
  const int in_step = lane / p.units, u = lane - in_step * p.units;   // head of the step, place in it
  if (in_step >= p.heads_per_step) return;
  const uint32_t lanes = 0xffffffffu >> (32 - p.heads_per_step * p.units);
  uint64_t turn[kOwn];
  int64_t at[kOwn];   // of its axis' positions
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    const int pair = u * kPairs + in_step % (kPairs / kOwn) * kOwn + j;
    turn[j] = p.turn[pair];
    at[j] = static_cast<int64_t>(p.axis[pair]) * p.total;
  }
  // (launch_beside: everything above ran beside the kernel before)
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const int total = p.num_tokens ? min(p.total, max(0, __ldg(p.num_tokens))) : p.total;
  const int heads = p.Hq + p.Hkv;
  const int a0 = u * kElems, b0 = a0 + p.width / 2;
  const int tasks = total * p.chunks;   // (at most 2^30)
  for (int task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks;
       task += gridDim.x * (kThreads / 32)) {
    const int t = task / p.chunks, chunk = task - t * p.chunks;
    const __nv_bfloat16 *q = p.q + t * p.q_stride, *k = p.k + t * p.k_stride;
    __nv_bfloat16 *q_out = p.q_out + t * p.q_out_stride, *k_out = p.k_out + t * p.k_out_stride;
    const int first = chunk * p.steps * p.heads_per_step;
    const int end = min(heads, (chunk + 1) * p.steps * p.heads_per_step);
    float2 cs[kPairs];
    for (int h0 = first; h0 < end; h0 += kBatch * p.heads_per_step) {
      V a[kBatch], b[kHalves ? kBatch : 1];
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const int h = h0 + in_step + s * p.heads_per_step;
        if (h >= end) break;
        const __nv_bfloat16 *src = h < p.Hq ? q + static_cast<int64_t>(h) * p.D
                                            : k + static_cast<int64_t>(h - p.Hq) * p.D;
        a[s] = *reinterpret_cast<const V *>(src + a0);
        if (kHalves) b[s] = *reinterpret_cast<const V *>(src + b0);
      }
      if (h0 == first) {
        float2 own[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) own[j] = turned(__ldg(p.positions + at[j] + t), turn[j]);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const int from = i / kOwn * p.units + u;
          cs[i] = own[i % kOwn];
          if (kOwn < kPairs) {
            cs[i].x = __shfl_sync(lanes, cs[i].x, from);
            cs[i].y = __shfl_sync(lanes, cs[i].y, from);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const int h = h0 + in_step + s * p.heads_per_step;
        if (h >= end) break;
        uint32_t *aw = reinterpret_cast<uint32_t *>(&a[s]);
        uint32_t *bw = reinterpret_cast<uint32_t *>(&b[kHalves ? s : 0]);
#pragma unroll
        for (int w = 0; w < kElems / 2; ++w) {
          const float2 c0 = cs[kHalves ? 2 * w : w], c1 = cs[kHalves ? 2 * w + 1 : w];
          const float x0 = lo_of(aw[w]), x1 = hi_of(aw[w]);
          if (kHalves) {
            const float y0 = lo_of(bw[w]), y1 = hi_of(bw[w]);
            aw[w] = pack2(x0 * c0.x - y0 * c0.y, x1 * c1.x - y1 * c1.y);
            bw[w] = pack2(x0 * c0.y + y0 * c0.x, x1 * c1.y + y1 * c1.x);
          } else {
            aw[w] = pack2(x0 * c0.x - x1 * c0.y, x0 * c0.y + x1 * c0.x);
          }
        }
        __nv_bfloat16 *dst = h < p.Hq ? q_out + static_cast<int64_t>(h) * p.D
                                      : k_out + static_cast<int64_t>(h - p.Hq) * p.D;
        *reinterpret_cast<V *>(dst + a0) = a[s];
        if (kHalves) *reinterpret_cast<V *>(dst + b0) = b[kHalves ? s : 0];
        if (p.width < p.D) {   // elements past the rotated width
          const __nv_bfloat16 *src = h < p.Hq ? q + static_cast<int64_t>(h) * p.D
                                              : k + static_cast<int64_t>(h - p.Hq) * p.D;
          if (src != dst)
            for (int at = p.width + a0; at < p.D; at += p.units * kElems)
              *reinterpret_cast<V *>(dst + at) = *reinterpret_cast<const V *>(src + at);
        }
      }
    }
  }
}

template <bool kHalves, int kElems, bool kMany>
void (*pick(int own))(RopeParams) {
  constexpr int kBatch = batch_of(kHalves, kMany);
  return own == 1   ? rope_axes_kernel<kHalves, kElems, 1, kBatch>
         : own == 2 ? rope_axes_kernel<kHalves, kElems, 2, kBatch>
                    : rope_axes_kernel<kHalves, kElems, 4, kBatch>;
}

// What a call's numbers say about every pair: theta / (2 pi) in 2^-64 of a turn, and
// its axis.  64 powers take some 2 us, so each thread keeps the last call's.
struct Spectrum {
  int32_t axes = 0, shared = 0, dims[kMaxAxes] = {};
  float base = 0.f;
  uint64_t turn[kMaxPairs] = {};
  uint8_t axis[kMaxPairs] = {};

  bool of(const int32_t *d, int32_t n, int32_t s, float b) const {
    if (n != axes || s != shared || b != base) return false;
    for (int a = 0; a < n; ++a)
      if (d[a] != dims[a]) return false;
    return true;
  }
  void set(const int32_t *d, int32_t n, int32_t s, float b) {
    axes = n;
    shared = s;
    base = b;
    int width = 0, pair = 0;
    for (int a = 0; a < n; ++a) width += dims[a] = d[a];
    const double log2_base = log2(static_cast<double>(b));
    for (int a = 0; a < n; ++a)
      for (int j = 0; j < d[a] / 2; ++j, ++pair) {
        const double power = s ? 2.0 * pair / width : 2.0 * j / d[a];
        double turns = exp2(-power * log2_base) * 0.15915494309189533577;
        turns -= floor(turns);   // (whole turns, with a base below 1)
        turn[pair] = turns < 1.0 ? static_cast<uint64_t>(turns * 0x1p64) : 0;
        axis[pair] = static_cast<uint8_t>(a);
      }
  }
};

}  // namespace
}  // namespace pa

extern "C" pa_status pa_rope_axes(const void *q, const void *k, void *q_out, void *k_out,
                                  const int32_t *positions, const int32_t *num_tokens,
                                  const int32_t *axis_dims, int32_t axes, int32_t total,
                                  int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                                  int64_t k_out_stride, int32_t Hq, int32_t Hkv, int32_t D,
                                  int32_t halves, int32_t shared, float base,
                                  pa_stream_t stream) {
  using namespace pa;
  if (!axis_dims || axes < 1 || total < 0 || Hq < 1 || Hkv < 0 || D < 2 || !isfinite(base) ||
      !(base > 0.f))
    return PA_ERR_INVALID_ARG;
  if (total > 0 && (!positions || !q || !q_out || (Hkv > 0 && (!k || !k_out))))
    return PA_ERR_INVALID_ARG;
  if (axes > kMaxAxes || D > 2 * kMaxPairs || (D & 7) || Hq > (1 << 20) || Hkv > (1 << 20))
    return PA_ERR_UNSUPPORTED;
  int64_t width = 0;
  for (int a = 0; a < axes; ++a) {
    if (axis_dims[a] < 2 || (axis_dims[a] & 1)) return PA_ERR_INVALID_ARG;
    width += axis_dims[a];
  }
  if (width > D) return PA_ERR_INVALID_ARG;
  if (width & 7) return PA_ERR_UNSUPPORTED;
  const int64_t row_q = int64_t{Hq} * D, row_k = int64_t{Hkv} * D;
  if (q_stride < row_q || q_out_stride < row_q || k_stride < row_k || k_out_stride < row_k ||
      (q == q_out && q_stride != q_out_stride) ||
      (Hkv > 0 && k == k_out && k_stride != k_out_stride))
    return PA_ERR_INVALID_ARG;
  constexpr int64_t kMostStride = int64_t{1} << 38;
  if (q_stride > kMostStride || k_stride > kMostStride || q_out_stride > kMostStride ||
      k_out_stride > kMostStride)
    return PA_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(q_out, 16) ||
      !aligned_to(k_out, 16) || !aligned_to(positions, 4) || !aligned_to(num_tokens, 4) ||
      ((q_stride | k_stride | q_out_stride | k_out_stride) & 7) != 0)
    return PA_ERR_MISALIGNED;
  if (int64_t{total} * (Hq + Hkv) > (int64_t{1} << 30)) return PA_ERR_UNSUPPORTED;
  if (total == 0) return PA_OK;
  RopeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k = static_cast<const __nv_bfloat16 *>(k);
  p.q_out = static_cast<__nv_bfloat16 *>(q_out);
  p.k_out = static_cast<__nv_bfloat16 *>(k_out);
  p.positions = positions;
  p.num_tokens = num_tokens;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.total = total;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.width = static_cast<int>(width);
  static thread_local Spectrum spectrum;
  if (!spectrum.of(axis_dims, axes, shared != 0, base))
    spectrum.set(axis_dims, axes, shared != 0, base);
  memcpy(p.turn, spectrum.turn, sizeof(uint64_t) * (width / 2));
  memcpy(p.axis, spectrum.axis, width / 2);
  // with halves a vector must not cross from one half into the other
  const int elems = halves && (width & 15) ? 4 : 8;
  p.units = static_cast<int>(width) / (halves ? 2 * elems : elems);   // (at most 32)
  p.heads_per_step = 32 / p.units;
  int32_t *status;
  int sms;
  const cudaError_t e = device_context(&status, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  // A token is shared out where whole ones leave the SMs short of 32 warps each,
  // as far as a batch of loads a lane: cos and sin are then computed for each.
  const int64_t want = (int64_t{sms} * 32 + total - 1) / total;
  const bool many = want <= 4;
  const int batch = batch_of(halves != 0, many);
  const int all_steps = (Hq + Hkv - 1) / p.heads_per_step + 1;
  const int most = (all_steps + batch - 1) / batch;
  p.chunks = want < most ? static_cast<int>(want) : most;
  p.steps = ((all_steps + p.chunks - 1) / p.chunks + batch - 1) / batch * batch;
  p.chunks = (all_steps + p.steps - 1) / p.steps;
  const int64_t tasks = int64_t{total} * p.chunks;
  const int64_t blocks = (tasks + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = static_cast<int>(blocks < int64_t{sms} * 8 ? blocks : int64_t{sms} * 8);
  // pairs of a lane's own: those it has, over the heads of a step (as a power of two)
  int own = halves ? elems : elems / 2;
  for (int others = 2; others <= p.heads_per_step && own > 1; others *= 2) own /= 2;
  const auto kernel = !halves      ? pick<false, 8, false>(many ? 4 : own)
                      : elems == 8 ? many ? pick<true, 8, true>(own) : pick<true, 8, false>(own)
                      : many       ? pick<true, 4, true>(own) : pick<true, 4, false>(own);
  return from_cuda(launch_beside(kernel, dim3(grid), kThreads, 0,
                                 reinterpret_cast<cudaStream_t>(stream), p));
}
