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
// turn that is left, with no error but the fraction's own (2^-53 of it, times
// the position) and no double-precision arithmetic on the GPU.  sincospif then
// has an argument in [-1, 1).
//
// HBM bound: q and k are read and written once.  A warp's task is a token and
// some of its heads.  A lane has a fixed place in its head, a vector of eight
// elements (with halves, the two vectors of its pairs), so its fractions stay in
// registers and its cos and sin, computed while the task's loads are in
// flight, serve all of the task's heads.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "sched.cuh"

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
  int heads_per_step, chunks;   // chunks: tasks of a token
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

// Heads a lane takes per task: 128 bytes of loads in flight.
constexpr int steps_of(bool halves) { return halves ? 4 : 8; }

// kHalves: pairs (i, i + R/2), else (2i, 2i + 1).  kElems: elements of a vector.
template <bool kHalves, int kElems>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  using V = typename Vec<kElems>::type;
  constexpr int kPairs = kHalves ? kElems : kElems / 2;   // of a lane
  constexpr int kSteps = steps_of(kHalves);
  const int lane = threadIdx.x & 31;
  const int in_step = lane / p.units, u = lane - in_step * p.units;   // head of the step, place in it
  if (in_step >= p.heads_per_step) return;
  uint64_t turn[kPairs];
  const int32_t *pos[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    turn[i] = p.turn[u * kPairs + i];
    pos[i] = p.positions + static_cast<int64_t>(p.axis[u * kPairs + i]) * p.total;
  }
  const int total = p.num_tokens ? min(p.total, max(0, __ldg(p.num_tokens))) : p.total;
  const int heads = p.Hq + p.Hkv;
  const int a0 = u * kElems, b0 = a0 + p.width / 2;
  const int tasks = total * p.chunks;   // (at most 2^30)
  for (int task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks;
       task += gridDim.x * (kThreads / 32)) {
    const int t = task / p.chunks, chunk = task - t * p.chunks;
    const int h0 = chunk * kSteps * p.heads_per_step + in_step;
    const __nv_bfloat16 *q = p.q + t * p.q_stride, *k = p.k + t * p.k_stride;
    __nv_bfloat16 *q_out = p.q_out + t * p.q_out_stride, *k_out = p.k_out + t * p.k_out_stride;
    V a[kSteps], b[kHalves ? kSteps : 1];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = h0 + s * p.heads_per_step;
      if (h >= heads) break;
      const __nv_bfloat16 *src = h < p.Hq ? q + static_cast<int64_t>(h) * p.D
                                          : k + static_cast<int64_t>(h - p.Hq) * p.D;
      a[s] = *reinterpret_cast<const V *>(src + a0);
      if (kHalves) b[s] = *reinterpret_cast<const V *>(src + b0);
    }
    float2 cs[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) cs[i] = turned(__ldg(pos[i] + t), turn[i]);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = h0 + s * p.heads_per_step;
      if (h >= heads) break;
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
  const double log2_base = log2(static_cast<double>(base));
  int pair = 0;
  for (int a = 0; a < axes; ++a)
    for (int j = 0; j < axis_dims[a] / 2; ++j, ++pair) {
      const double power = shared ? 2.0 * pair / static_cast<double>(width)
                                  : 2.0 * j / axis_dims[a];
      // theta / (2 pi) of a turn; whole turns are dropped (a base below 1)
      double turns = exp2(-power * log2_base) * 0.15915494309189533577;
      turns -= floor(turns);
      p.turn[pair] = turns < 1.0 ? static_cast<uint64_t>(turns * 0x1p64) : 0;
      p.axis[pair] = static_cast<uint8_t>(a);
    }
  // with halves a vector must not cross from one half into the other
  const int elems = halves && (width & 15) ? 4 : 8;
  p.units = static_cast<int>(width) / (halves ? 2 * elems : elems);   // (at most 32)
  p.heads_per_step = 32 / p.units;
  const int heads_per_task = steps_of(halves != 0) * p.heads_per_step;
  p.chunks = (Hq + Hkv + heads_per_task - 1) / heads_per_task;
  const int64_t tasks = int64_t{total} * p.chunks;
  if (tasks > (int64_t{1} << 30)) return PA_ERR_UNSUPPORTED;
  int32_t *status;
  int sms;
  const cudaError_t e = device_context(&status, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  const int64_t blocks = (tasks + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = static_cast<int>(blocks < int64_t{sms} * 8 ? blocks : int64_t{sms} * 8);
  auto s = reinterpret_cast<cudaStream_t>(stream);
  if (halves && elems == 8)
    rope_axes_kernel<true, 8><<<grid, kThreads, 0, s>>>(p);
  else if (halves)
    rope_axes_kernel<true, 4><<<grid, kThreads, 0, s>>>(p);
  else
    rope_axes_kernel<false, 8><<<grid, kThreads, 0, s>>>(p);
  return from_cuda(cudaGetLastError());
}
