// The linear layers with an epilogue (gemm_tc.cu) for few rows: a step of single
// tokens, a short prompt.
//
// Few rows are bound by w's bytes (2 N K of them for 2 M N K operations), so the
// work is split over the features, finely enough that every SM streams a part
// of w: a CTA computes F features (a multiple of 8, at most 128) of R rows of x
// (a multiple of 16, at most 256; few_plan).  The product is turned around: w is the MMA's A operand, its rows
// the accumulator's TMEM lanes, and x is B, its rows the columns, so
// a call of 13 rows pays for 16 columns and not for a tile of 128 rows.  An MMA
// has 64 or 128 rows; where F is less, those past F are whatever follows in shared
// memory, and what they give in the lanes past F is never read.  (With room for all
// rows in the ring less of w was on its way: gated 24 x 4096 x 11264 36.2 us, now 32.6.)
//
// An element's products are added in the same order as in the large kernel (K
// in steps of 16, one accumulator, no split over K), and the epilogue is the
// same arithmetic, so rows come out with the same bits by either.
//
//   warp 0      TMA producer: groups of K-blocks of w and x into a ring
//   warp 1      allocates TMEM, issues the MMAs (what bounds short calls: an MMA of
//               few columns takes its issuer some 45 cycles and the tensor core
//               less, so the loop has one branch a K-block and no divisions)
//   warps 2-5   epilogue, a lane a feature: bias, activation, residual (read ahead of
//               the accumulator's end), columns of y as runs of 32 features
// Every wait is bounded; a timeout records PA_DEVICE_ERR_TIMEOUT.
#include <cuda_bf16.h>
#include <stdint.h>

#include "activation.cuh"
#include "internal.h"
#include "linear.cuh"
#include "sched.cuh"
#include "tc_ptx.cuh"
#include "tma_map.h"

namespace pa {
namespace {

using namespace tc;

constexpr int kThreads = 192;
constexpr int kMaxStages = 16;
constexpr int kRingBytes = 212 * 1024;          // stages, at most
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (~2 s)
constexpr long long kDrainLimit = 400000000LL;  // teardown after an abort (~0.2 s)
constexpr int kRowBytes = kLinearBK * 2;        // of a K-block: 128
constexpr int kChunk = 16;                      // columns the epilogue takes at once

// Shared memory: full and empty barriers, the accumulator's, TMEM address and
// abort flag; then the ring on 1024 bytes.
constexpr int kBarBytes = (2 * kMaxStages + 1) * 8;
constexpr int kMiscOff = kBarBytes;
constexpr int kRingOff = 1024;
// An MMA reads the rows of kM features, of which a K-block has F: those past its
// last one are the next one's bytes, and past the ring's end these.
constexpr int kPadBytes = 56 * kRowBytes;
constexpr int kSmemBytes = kRingOff + kRingBytes + kPadBytes;
static_assert(kMiscOff + 8 <= kRingOff && kSmemBytes <= 232448, "shared memory plan");

struct FewParams {
  const __nv_bfloat16 *bias;       // [N] or nullptr
  const __nv_bfloat16 *residual;   // or nullptr
  __nv_bfloat16 *y;
  int64_t y_stride, residual_stride;
  int act;
  int M, N, K;
  int features, rows;              // of a CTA: F, and columns of its accumulator
  int k_blocks, group, stages;     // K-blocks, those of a stage
  int stage_bytes, block_bytes;    // of a stage, of a K-block
  uint32_t idesc, tmem_cols;
  int32_t *status;
};

// kM: rows of an MMA, at least the features of a CTA.
template <int kMode, int kM>
__global__ void __launch_bounds__(kThreads, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_w2, const FewParams p) {
  constexpr int kParts = kMode == kGated ? 2 : 1;   // weights, accumulators
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {   // swizzle atoms need a 1024-byte aligned base
    if (threadIdx.x == 0) record_error(p.status, PA_DEVICE_ERR_SMEM_ALIGN);
    return;
  }
  auto full = [&](uint32_t s) -> uint32_t { return base + 8u * s; };
  auto empty = [&](uint32_t s) -> uint32_t { return base + 8u * (kMaxStages + s); };
  const uint32_t acc_full = base + 8u * (2 * kMaxStages);
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem_raw + kMiscOff);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(smem_raw + kMiscOff + 4);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int n0 = blockIdx.x * p.features, m0 = blockIdx.y * p.rows;
  const int a_bytes = p.features * kRowBytes, b_bytes = p.rows * kRowBytes;   // of a K-block
  const int n_stages = (p.k_blocks + p.group - 1) / p.group;   // filled in all

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(base + kMiscOff, p.tmem_cols);
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
    if (kMode == kGated) tma_prefetch_desc(&tm_w2);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_ptr;
  // w on its way from HBM to L2 for the first stages, before the kernel before
  // has ended (the copies below come after it)
  if (warp == 0 && blockIdx.y == 0 && elect_one()) {
    const int ahead = min(p.k_blocks, p.stages * p.group);
    for (int b = 0; b < ahead; ++b) {
      tma_prefetch_2d(&tm_w, b * kLinearBK, n0);
      if (kMode == kGated) tma_prefetch_2d(&tm_w2, b * kLinearBK, n0);
    }
  }
  __syncwarp();
  // (launch_beside: everything above ran beside the kernel before)
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    const bool lead = elect_one();
    bool ok = true;
    int i = 0;
    for (; i < n_stages; ++i) {
      const uint32_t s = i % p.stages;
      ok = bounded_wait(empty(s), ((i / p.stages) & 1u) ^ 1u, abort_flag, p.status, kWaitLimit);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int kb0 = i * p.group, blocks = min(p.group, p.k_blocks - kb0);
      const uint32_t dst = base + kRingOff + s * p.stage_bytes;
      if (lead) {
        mbar_arrive_expect_tx(full(s), blocks * (kParts * a_bytes + b_bytes));
        for (int b = 0; b < blocks; ++b) {
          const uint32_t a = dst + b * p.block_bytes;
          const int k = (kb0 + b) * kLinearBK;
          tma_load_2d(a, &tm_w, full(s), k, n0);
          if (kMode == kGated) tma_load_2d(a + a_bytes, &tm_w2, full(s), k, n0);
          tma_load_2d(a + kParts * a_bytes, &tm_x, full(s), k, m0);
        }
      }
    }
    if (!ok) {   // give the copies already issued a bounded chance to land
      for (int s = 0; s < p.stages && s < i; ++s)
        drain_wait(full(s), ((i - s + p.stages - 1) / p.stages - 1) & 1u, kDrainLimit);
    }
  } else if (warp == 1) {
    const bool lead = elect_one();
    const uint64_t desc0 = sdesc_sw128(base + kRingOff, 16, 1024);
    const uint64_t w2_off = a_bytes >> 4, x_off = kParts * a_bytes >> 4;
    bool ok = true;
    int i = 0;
    uint32_t s = 0, parity = 0, more = 0;
    for (; i < n_stages; ++i) {
      ok = bounded_wait(full(s), parity, abort_flag, p.status, kWaitLimit);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int blocks = min(p.group, p.k_blocks - i * p.group);
      uint64_t a = desc0 + ((s * p.stage_bytes) >> 4);
#pragma unroll 1
      for (int b = 0; b < blocks; ++b) {
        const uint64_t x = a + x_off;
        if (lead) {
          mma_ss(tmem, a, x, p.idesc, more);
          if (kMode == kGated) mma_ss(tmem + p.rows, a + w2_off, x, p.idesc, more);
#pragma unroll
          for (int kk = 1; kk < kLinearBK / 16; ++kk) {
            mma_ss(tmem, a + kk * 2, x + kk * 2, p.idesc, 1u);
            if (kMode == kGated)
              mma_ss(tmem + p.rows, a + w2_off + kk * 2, x + kk * 2, p.idesc, 1u);
          }
        }
        more = 1;
        a += p.block_bytes >> 4;
      }
      if (lead) mma_commit(empty(s));
      if (++s == static_cast<uint32_t>(p.stages)) {
        s = 0;
        parity ^= 1u;
      }
    }
    if (lead) mma_commit(acc_full);   // every MMA issued so far is done
    if (!ok) drain_wait(acc_full, 0, kWaitLimit);
    __syncwarp();
  } else {
    const int quad = warp & 3;
    // accumulator rows: 32 a quadrant, or (an MMA of 64 rows) its first 16 lanes
    const int f = kM == 128 ? quad * 32 + lane : quad * 16 + lane;
    const int n = n0 + f;
    const bool mine = (kM == 128 || lane < 16) && f < p.features && f < p.N - n0;
    const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int rows = min(p.rows, p.M - m0);
    float bias = 0.f;
    if (kMode == kAct && p.bias && mine) bias = __bfloat162float(p.bias[n]);
    __nv_bfloat16 *y = p.y + m0 * p.y_stride + n;
    const bool add = kMode == kAct && p.residual != nullptr && mine;
    const __nv_bfloat16 *res = p.residual + m0 * p.residual_stride + n;
    __nv_bfloat16 r[kChunk];
    auto read_ahead = [&](int c) {
      if (!add) return;
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (c + e < rows) r[e] = res[(c + e) * p.residual_stride];
    };
    read_ahead(0);
    const bool ok = bounded_wait(acc_full, 0, abort_flag, p.status, kWaitLimit);
    if (__all_sync(0xffffffffu, ok) && *abort_flag == 0) {
      fence_after_sync();
      for (int c = 0; c < rows; c += kChunk) {
        uint32_t a[kChunk], u[kChunk];
        tmem_ld8(acc + c, a);
        tmem_ld8(acc + c + 8, a + 8);
        if (kMode == kGated) {
          tmem_ld8(acc + p.rows + c, u);
          tmem_ld8(acc + p.rows + c + 8, u + 8);
        }
        tmem_wait_ld();
        float v[kChunk];
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[e] = __uint_as_float(a[e]) + (kMode == kAct ? bias : 0.f);
        activate(v, p.act);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
          if (kMode == kGated) v[e] *= __uint_as_float(u[e]);
          if (add && c + e < rows) v[e] += __bfloat162float(r[e]);
        }
        if (c + kChunk < rows) read_ahead(c + kChunk);
        if (mine) {
#pragma unroll
          for (int e = 0; e < kChunk; ++e)
            if (c + e < rows) y[(c + e) * p.y_stride] = __float2bfloat16_rn(v[e]);
        }
      }
    }
  }

  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

int round_up(int x, int to) { return (x + to - 1) / to * to; }

template <int kMode, int kM>
pa_status launch(const GemmArgs &a, FewParams &p, cudaStream_t stream) {
  CUtensorMap mx, mw, mw2;
  if (!make_map_2d(&mx, a.x, a.M, a.K, a.x_stride, p.rows) ||
      !make_map_2d(&mw, a.w, a.N, a.K, a.K, p.features) ||
      !make_map_2d(&mw2, kMode == kGated ? a.w2 : a.w, a.N, a.K, a.K, p.features))
    return from_cuda(cudaErrorInvalidValue);
  p.block_bytes = ((kMode == kGated ? 2 : 1) * p.features + p.rows) * kRowBytes;
  p.idesc = idesc_bf16_f32(kM, p.rows, false);
  // Stages of a quarter of the ring: large, as a barrier's cost to the issuer is
  // spread over a stage's MMAs, and not larger, as a stage is waited for whole (13
  // rows, K = 16384, 4096 features: a half 26.6 us, a third 24.9, a quarter 24.5).
  // All of an SM's shared memory is on its way from HBM; rings of half of it, with
  // the next call's CTAs beside this one's, took 9.9 us for 4096 x 4096 in place of 7.8.
  p.group = kRingBytes / 4 / p.block_bytes > 1 ? kRingBytes / 4 / p.block_bytes : 1;
  if (p.group > p.k_blocks) p.group = p.k_blocks;
  p.stage_bytes = p.group * p.block_bytes;
  p.stages = kRingBytes / p.stage_bytes < kMaxStages ? kRingBytes / p.stage_bytes : kMaxStages;
  static unsigned long long configured = 0;
  const auto kernel = linear_few_kernel<kMode, kM>;
  const cudaError_t e =
      set_smem_once(reinterpret_cast<const void *>(kernel), kSmemBytes, configured);
  if (e != cudaSuccess) return from_cuda(e);
  const dim3 grid((a.N - 1) / p.features + 1, (a.M - 1) / p.rows + 1);   // (N up to 2^31 - 8)
  return from_cuda(launch_beside(kernel, grid, kThreads, kSmemBytes, stream, mx, mw,
                                 mw2, p));
}

// How a call is cut: CTAs of F features x R rows, and its time in ns.
struct FewPlan {
  int features, rows;
  int64_t ns;
};

// A CTA's K-block takes 75 + 1.33 R ns with an MMA of 64 rows (F <= 64) and
// 95 + 1.5 R with 128, 1.75 times that where there are two weights; all CTAs
// together get 9.7 TB/s out of L2 and 6.7 of w out of HBM; and a call costs 3 us
// besides.  Up to 16 rows and for wide pairs of weights this is within some 20 % of
// what was measured; from some 30 rows on the L2 term is far too slow and the model up
// to 90 % high.  Measured here, modelled here, measured by the large kernel (us, w out of HBM):
//   rows   4096 x 4096         4096 x 14336        two of 4096 x 4096   two of 11264 x 4096
//     33   10.0  11.9  23.9    24.7  34.1  66.3    16.6  18.6  23.2     30.9  30.5  46.1
//    128   12.4  18.0  24.6    32.3  55.5  67.0    18.3  25.0  22.5     37.0  37.3  47.4
//    256   16.9  24.9  24.7    44.2  79.7  67.2    26.8  33.0  22.8     50.6  56.6  48.2
//    300   18.2  26.8  24.9    45.8  86.4  67.5    30.4  37.0  23.6     73.7  79.2  58.7
//    512   24.4  33.0  25.3    65.2   108  67.8    35.3  44.9  24.2     84.8   102  63.6
//   1024   34.6  49.0  26.6    92.4   164  71.2    50.7  63.0  41.1      172   174   102
// The choice by it is right or within 8 % of these, but for some 260 to 380 rows of one
// weight, which go to the large kernel: 300 rows 24.9 in place of 18.2, 67 in place of 46.
// What bounds 64 to 512 rows is what a K-block brings into an SM, F + R rows of 128
// bytes, at 95 to 130 bytes a ns.
FewPlan few_plan(const GemmArgs &a, int mode, int sms) {
  const int64_t parts = mode == kGated ? 2 : 1, blocks = (a.K - 1) / kLinearBK + 1;
  FewPlan best{0, 0, INT64_MAX};
  for (int tiles_m = (a.M - 1) / 256 + 1; tiles_m <= 16 && tiles_m * 16 < a.M + 16; ++tiles_m) {
    const int64_t rows = round_up((a.M - 1) / tiles_m + 1, 16);
    // as few features as fill the SMs, in as few rounds as 128 of them allow
    const int64_t across = sms / tiles_m > 0 ? sms / tiles_m : 1;
    const int64_t rounds = (a.N - 1) / (128 * across) + 1;
    const int64_t features = round_up(static_cast<int>((a.N - 1) / (rounds * across) + 1), 8);
    const int64_t ctas = ((a.N - 1) / features + 1) * tiles_m, waves = (ctas - 1) / sms + 1;
    int64_t block = features <= 64 ? 75 + rows * 4 / 3 : 95 + rows * 3 / 2;
    if (parts == 2) block = block * 7 / 4;
    const int64_t tile = waves * blocks * block;
    const int64_t l2 = ctas * blocks * (parts * features + rows) * kRowBytes / 9700;
    const int64_t hbm = parts * a.N * a.K * 2 / 6700;
    int64_t ns = tile > l2 ? tile : l2;
    ns = 3000 + (ns > hbm ? ns : hbm);
    if (ns < best.ns)
      best = FewPlan{static_cast<int>(features), static_cast<int>(rows), ns};
  }
  return best;
}

// The large kernel's time of the same call: a round of tiles of 256 x 256 on pairs
// of SMs (of 128 features, where there are two weights), 345 ns a K-block, but 500
// below 64 rows (more than 4096 features take, 24 us at any of few rows, but there
// the other kernel is far ahead; two weights of 28672 x 1024: 40 rows 31.3 us, 64 rows 22.9; of 8192 x
// 4096: 13 rows 39.5, 48 rows 27.3; by the kernel for few rows 24.9 of the former's 40,
// and 22.7 and 24.4).
int64_t large_ns(const GemmArgs &a, int mode, int sms) {
  const int64_t tile_n = mode == kGated ? 128 : 256;
  const int64_t tiles = ((a.N - 1) / tile_n + 1) * ((int64_t{a.M} - 1) / 256 + 1);
  return 3000 + ((tiles - 1) / (sms / 2) + 1) * ((a.K - 1) / kLinearBK + 1) *
                    (a.M < 64 ? 500 : 345);
}

}  // namespace

pa_status launch_linear_few(const GemmArgs &a, int mode, bool &taken, cudaStream_t stream) {
  taken = false;
  FewParams p;
  int sms;
  const cudaError_t e = device_context(&p.status, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  const FewPlan plan = few_plan(a, mode, sms);
  if (plan.ns > large_ns(a, mode, sms)) return PA_OK;
  taken = true;
  p.bias = static_cast<const __nv_bfloat16 *>(a.bias);
  p.residual = static_cast<const __nv_bfloat16 *>(a.residual);
  p.y = static_cast<__nv_bfloat16 *>(a.y);
  p.y_stride = a.y_stride;
  p.residual_stride = a.residual_stride;
  p.act = a.act;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.k_blocks = (a.K - 1) / kLinearBK + 1;
  p.rows = plan.rows;
  p.features = plan.features;
  const int cols = (mode == kGated ? 2 : 1) * p.rows;
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(cols)) p.tmem_cols *= 2;
  if (mode == kGated)
    return p.features <= 64 ? launch<kGated, 64>(a, p, stream) : launch<kGated, 128>(a, p, stream);
  return p.features <= 64 ? launch<kAct, 64>(a, p, stream) : launch<kAct, 128>(a, p, stream);
}

}  // namespace pa
