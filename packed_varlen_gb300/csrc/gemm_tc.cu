// Batch-invariant packed-M linear layer on the 5th-generation tensor cores:
//
//   y[m, n] = sum_k x[m, k] * w[n, k]  (+ bias[n])
//
// with bf16 x, w, bias and y and fp32 accumulation.  The packed path runs
// the projections of every request at once on the flat [total_tokens, C]
// activations, and its batched and serial outputs are bit-identical because
// these GEMMs give a row the same result whatever the packed M is ("feat:
// Support dynamic batching for heterogeneous diffusion requests", packed
// varlen step batching: Setup, Determinism, and Notes, item 1).
//
// Batch invariance by construction: one tile shape (256 x 256 x 64 per CTA
// pair) for every M, no split-K, K walked in the same order in every tile, and an epilogue
// that treats each row alone.  A row's result therefore depends only on its
// own x row, w and bias: packed or alone, at any row offset, the bits agree.
//
// Kernel: persistent, one CTA per SM, CTAs in clusters of two that work as a
// cta_group::2 pair on 256 x 256 output tiles, ten warps each.  One MMA
// (M = 256, N = 256, K = 16) spans the pair: each CTA holds 128 rows of the
// x tile and one 128-row half of the w tile in its own shared memory, loaded
// by its own TMA from this GPU's memory (no CTA writes another's shared
// memory), and receives its 128 output rows in its own TMEM.  Per CTA that is the L2
// traffic of a 128 x 256 tile with only half of w, and one MMA instruction
// per pair instead of two.
//   warp 0      TMA producer (both CTAs) into a kStages-deep ring; both
//               CTAs count their bytes on the even CTA's full barrier.
//   warp 1      allocates TMEM in both CTAs (a collective pair allocation);
//               in the even CTA it issues the MMAs into one of two TMEM
//               accumulators (2 x 256 fp32 columns) and frees each ring slot
//               in both CTAs with one commit per CTA.
//   warps 2-9   drain a finished accumulator (two warps to a TMEM lane
//               quadrant, half the columns each), add the bias, round to bf16
//               and store, while the MMA warp fills the other; each warp then
//               reports the accumulator free on the even CTA's barrier.  A
//               warp's 32 rows x 64 columns go through 4 KB of shared memory
//               that copies fill with the residual, ahead of the accumulator,
//               and write out as y: a lane has a row of its own, and rows stored
//               by lanes would be 32 separate pieces of 16 bytes a time.
// Warps 0 and 1 run their loops warp-wide and one elected lane issues each
// copy, MMA and commit, so MMA operands are warp-uniform.  Tile pairs go
// round-robin over the clusters, in groups of kGroupM row blocks with the row
// block fastest: a wave of 76 pairs then spans about 8 x 10 tiles and reads the
// fewest rows of x and w.  Every wait is bounded; a timeout records
// PA_DEVICE_ERR_TIMEOUT.
//
// The same kernel with other epilogues:
//   kAct    y = residual + act(x w^T + bias)
//   kGated  y = act(x w_gate^T) * (x w_up^T): the even CTA's half of the w tile
//           is 128 rows of w_gate and the odd CTA's 128 rows of w_up, so one
//           accumulator holds both products of 128 columns of y.
// All of it is fp32, rounded once, and of a row alone, so the rows stay batch
// invariant.
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

constexpr int kBM = 128, kBN = 256;             // kBM rows per CTA, kBN columns per pair
constexpr int kBK = kLinearBK;
constexpr int kStages = 6;
constexpr int kCluster = 2;                     // the CTA pair of one MMA
constexpr int kThreads = 320;                   // TMA, MMA, 8 epilogue warps
constexpr int kGroupM = 8;                      // row blocks (of a pair) of a group
constexpr int kOutN = 64, kOutBytes = 32 * kOutN * 2;   // a warp's part of y in shared memory
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (~2 s)
constexpr long long kTileWaitLimit = 32 * kWaitLimit;   // of the epilogue: for all of a tile's K
constexpr long long kDrainLimit = 400000000LL;  // teardown after an abort (~0.2 s)

struct GemmCfg {
  static constexpr int kABytes = kBM * kBK * 2;                // 16 KB: 128 x rows x 128 B
  static constexpr int kBBytes = (kBN / kCluster) * kBK * 2;   // 16 KB: 128 w rows x 128 B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kOutOff = kStages * kStageBytes;        // 8 epilogue warps' buffers
  static constexpr int kBarOff = kOutOff + 8 * kOutBytes;
  static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages,
                       kAccEmpty = 2 * kStages + 2, kFinal = 2 * kStages + 4,
                       kResidual = 2 * kStages + 5;   // an epilogue warp's residual landed
  static constexpr int kNumBars = 2 * kStages + 13;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tmem base, abort flag
  static constexpr int kSmemBytes = kMiscOff + 16;
  static constexpr uint32_t kTmemCols = 2 * kBN;
  // A (x) and B (w) both K-major; M spans the pair
  static constexpr uint32_t kIdesc = idesc_bf16_f32(kCluster * kBM, kBN, false);
};
static_assert(GemmCfg::kSmemBytes <= 232448, "shared memory plan exceeds the per-CTA limit");

struct GemmParams {
  const __nv_bfloat16 *bias;  // [N] or nullptr
  int residual;               // add the residual (kAct)
  int act;
  int M, N, K;
  int tiles_m, tiles_n, n_pairs, k_blocks;   // n_pairs: (pair of 128-row blocks, N block)
  int32_t *status;
};

__device__ __forceinline__ void add8(float (&f)[8], const uint4 &v) {
  f[0] += bf16_lo(v.x); f[1] += bf16_hi(v.x);
  f[2] += bf16_lo(v.y); f[3] += bf16_hi(v.y);
  f[4] += bf16_lo(v.z); f[5] += bf16_hi(v.z);
  f[6] += bf16_lo(v.w); f[7] += bf16_hi(v.w);
}

// Tile pair tp -> its pair of 128-row blocks and its N block.
struct TilePair {
  int m, n;
};
__device__ __forceinline__ TilePair tile_pair(const GemmParams &p, int tp) {
  const int per_group = kGroupM * p.tiles_n;
  const int g = tp / per_group, r = tp - g * per_group;
  const int rows = min(kGroupM, p.tiles_m - g * kGroupM);
  TilePair t;
  t.n = r / rows;
  t.m = g * kGroupM + r - t.n * rows;
  return t;
}

// tm_w2: w_up (kGated only; tm_w is w_gate).  tm_r, tm_y: residual and y, in
// boxes of 32 rows x 64 columns.
template <int kMode>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    linear_bf16_kernel(const __grid_constant__ CUtensorMap tm_x,
                       const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_w2,
                       const __grid_constant__ CUtensorMap tm_r,
                       const __grid_constant__ CUtensorMap tm_y, const GemmParams p) {
  using C = GemmCfg;
  constexpr int kYN = kMode == kGated ? kBN / 2 : kBN;   // columns of y per tile
  extern __shared__ uint8_t smem_raw[];
  // 128-byte swizzle atoms need a 1024-byte aligned base.  Both CTAs of a
  // pair run the same code on the same layout, so both skip or neither.
  const uint32_t base = smem_u32(smem_raw);
  if (base & 1023u) {
    if (threadIdx.x == 0) record_error(p.status, PA_DEVICE_ERR_SMEM_ALIGN);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return base + C::kBarOff + 8u * i; };
  uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem_raw + C::kMiscOff);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(smem_raw + C::kMiscOff + 4);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(C::kFull + s), 1);    // the leader's expect_tx; bytes of both CTAs
      mbar_init(bar(C::kEmpty + s), 1);   // one commit from the leader's MMA warp
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(C::kAccFull + b), 1);
      mbar_init(bar(C::kAccEmpty + b), 8 * kCluster);   // every epilogue warp of the pair
    }
    for (int w = 0; w < 8; ++w) mbar_init(bar(C::kResidual + w), 1);
    mbar_init(bar(C::kFinal), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(base + C::kMiscOff, C::kTmemCols);
  fence_before_sync();
  __syncwarp();     // the cluster barrier is warp-aligned
  cluster_sync();   // barriers of both CTAs initialised before any remote use
  fence_after_sync();
  const uint32_t tmem = *tmem_ptr;
  // (launch_beside: everything above ran beside the kernel before)
  griddep_launch_dependents();
  griddep_wait();
  const int cl = blockIdx.x / kCluster, n_cl = gridDim.x / kCluster;

  if (warp == 0) {
    // ================= TMA producer (both CTAs) =================
    const bool lead = elect_one();
    const CUtensorMap *w_map = kMode == kGated && rank == 1 ? &tm_w2 : &tm_w;
    if (lead) {
      tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(w_map);
    }
    uint32_t loads = 0;
    bool ok = true;
    for (int tp = cl; tp < p.n_pairs && ok; tp += n_cl) {
      const TilePair t = tile_pair(p, tp);
      const int m0 = (t.m * kCluster + rank) * kBM;
      const int n0 = t.n * kYN + (kMode == kGated ? 0 : rank * (kBN / kCluster));
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        const uint32_t s = loads % kStages, use = loads / kStages;
        const bool w = bounded_wait_cluster(bar(C::kEmpty + s), (use & 1u) ^ 1u, abort_flag,
                                            p.status, kWaitLimit);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        const uint32_t dst = base + s * C::kStageBytes;
        const uint32_t full = mapa_shared(bar(C::kFull + s), 0);   // the leader's barrier
        if (lead) {
          if (leader) mbar_arrive_expect_tx(bar(C::kFull + s), kCluster * C::kStageBytes);
          tma_load_2d_pair(dst, &tm_x, full, kb * kBK, m0);
          tma_load_2d_pair(dst + C::kABytes, w_map, full, kb * kBK, n0);
        }
        ++loads;
      }
    }
    if (!ok && leader) {
      // give the copies already issued a bounded chance to land
      for (uint32_t s = 0; s < static_cast<uint32_t>(kStages) && s < loads; ++s) {
        const uint32_t n = (loads - s + kStages - 1) / kStages;  // loads into slot s
        drain_wait(bar(C::kFull + s), (n - 1) & 1u, kDrainLimit);
      }
    }
  } else if (warp == 1) {
    // ================= MMA issuer (the leader CTA only) =================
    // The whole warp runs the issuer, so every operand of an MMA is
    // warp-uniform, and one elected lane issues each MMA and commit:
    // tcgen05.mma issued from a lone lane's control flow pays a large
    // per-instruction cost.
    if (leader) {
      const bool lead = elect_one();
      auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
        const bool w = bounded_wait_cluster(b, parity, abort_flag, p.status, kWaitLimit);
        return __all_sync(0xffffffffu, w);
      };
      // commit to the same barrier in both CTAs of the pair
      auto commit_both = [&](uint32_t b) {
        mma_commit_pair(mapa_shared(b, 0));
        mma_commit_pair(mapa_shared(b, 1));
      };
      uint32_t uses = 0, tiles_done = 0;
      bool ok = true, issued = false;
      // descriptors advance by adding the byte offset >> 4 to the start
      // address field; every operand lies below 256 KB, so nothing carries
      const uint64_t adesc0 = sdesc_sw128(base, 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(base + C::kABytes, 16, 1024);
      for (int tp = cl; tp < p.n_pairs && ok; tp += n_cl, ++tiles_done) {
        const uint32_t buf = tiles_done & 1u, buse = tiles_done >> 1;
        if (!wait_all(bar(C::kAccEmpty + buf), (buse & 1u) ^ 1u)) {
          ok = false;
          break;
        }
        fence_after_sync();
        const uint32_t d = tmem + buf * kBN;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          const uint32_t s = uses % kStages;
          // both CTAs' bytes for this slot have landed once the wait returns
          if (!wait_all(bar(C::kFull + s), (uses / kStages) & 1u)) {
            ok = false;
            break;
          }
          const uint64_t a = adesc0 + ((s * C::kStageBytes) >> 4);
          const uint64_t b = bdesc0 + ((s * C::kStageBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            if (lead)
              mma_ss_pair(d, a + ((kk * 32) >> 4), b + ((kk * 32) >> 4), C::kIdesc,
                          (kb > 0 || kk > 0) ? 1u : 0u);
          issued = true;
          // the slot is free in both CTAs once these MMAs have read it
          if (lead) commit_both(bar(C::kEmpty + s));
          ++uses;
        }
        if (!ok) break;
        if (lead) commit_both(bar(C::kAccFull + buf));
      }
      // every MMA issued so far has finished before TMEM is released
      if (issued) {
        if (lead) mma_commit_pair(mapa_shared(bar(C::kFinal), 0));
        drain_wait(bar(C::kFinal), 0, kWaitLimit);
      }
    }
    __syncwarp();
  } else {
    // ================= epilogue: warps 2..9, TMEM lane quadrant warp % 4 =========
    constexpr int kParts = kYN / 2 / kOutN;   // parts of 64 columns of a warp
    const int quad = warp & 3, side = (warp - 2) >> 2;
    const bool lead = elect_one();
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t acc_empty0 = mapa_shared(bar(C::kAccEmpty), 0);   // the leader's
    const uint32_t out = base + C::kOutOff + (warp - 2) * kOutBytes;
    // this lane's row; the 128-byte swizzle permutes the 16-byte pieces of a row
    uint8_t *row = smem_raw + C::kOutOff + (warp - 2) * kOutBytes + lane * 128;
    const uint32_t landed = bar(C::kResidual + warp - 2);
    const bool add = kMode == kAct && p.residual;
    uint32_t tiles_done = 0, loads = 0, taken = 0;
    // part `part` of tile pair tp, if it has any of y
    int m0 = 0, c0 = 0;
    auto seek = [&](int tp, int part) -> bool {
      const TilePair t = tile_pair(p, tp);
      m0 = (t.m * kCluster + rank) * kBM + quad * 32;
      c0 = t.n * kYN + (side * kParts + part) * kOutN;
      return m0 < p.M && c0 < p.N;
    };
    // the residual of a part into the buffer, which the part before it has left
    auto load_residual = [&](int tp, int part) {
      if (!add || tp >= p.n_pairs || !seek(tp, part)) return;
      if (lead) {
        mbar_arrive_expect_tx(landed, kOutBytes);
        tma_load_2d(out, &tm_r, landed, c0, m0);
      }
      ++loads;
    };
    load_residual(cl, 0);
    for (int tp = cl; tp < p.n_pairs; tp += n_cl, ++tiles_done) {
      const uint32_t buf = tiles_done & 1u, buse = tiles_done >> 1;
      const bool ok = bounded_wait_cluster(bar(C::kAccFull + buf), buse & 1u, abort_flag, p.status,
                                           kTileWaitLimit);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after_sync();
      bool landed_ok = true;
#pragma unroll 1
      for (int part = 0; part < kParts; ++part) {
        const bool here = seek(tp, part);
        if (here && add) {
          landed_ok = bounded_wait(landed, taken & 1u, abort_flag, p.status, kWaitLimit);
          if (!__all_sync(0xffffffffu, landed_ok)) {
            landed_ok = false;
            break;
          }
          ++taken;
        }
        const uint32_t acc = lane_base + buf * kBN + (side * kParts + part) * kOutN;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0[32], a1[32];
          tmem_ld32(acc + h * 32, a0);
          if (kMode == kGated) tmem_ld32(acc + kYN + h * 32, a1);
          tmem_wait_ld();
          if (!here) continue;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 *piece = reinterpret_cast<uint4 *>(row + (((h * 4 + v) ^ (lane & 7)) << 4));
            const int c8 = c0 + h * 32 + 8 * v;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(a0[8 * v + e]);
            if (kMode != kGated && p.bias && c8 < p.N)   // N is a multiple of 8
              add8(f, __ldg(reinterpret_cast<const uint4 *>(p.bias + c8)));
            if (kMode != kLinear) activate(f, p.act);
            if (kMode == kGated) {
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] *= __uint_as_float(a1[8 * v + e]);
            }
            if (add) add8(f, *piece);
            *piece = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
          }
        }
        if (part == kParts - 1) {
          // every lane's TMEM reads are done; one arrival per warp on the
          // leader's barrier lets the MMA warp refill this accumulator
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(acc_empty0 + 8u * buf);
        }
        if (here) {
          fence_proxy_async();   // each lane's row, before the copy reads it
          __syncwarp();
          if (lead) {
            tma_store_2d(&tm_y, out, c0, m0);
            bulk_commit();
            bulk_wait_read();    // the buffer is free again
          }
          __syncwarp();
        }
        load_residual(part + 1 < kParts ? tp : tp + n_cl, part + 1 < kParts ? part + 1 : 0);
      }
      if (!landed_ok) break;
    }
    if (lead) bulk_wait();
    if (taken != loads) drain_wait(landed, taken & 1u, kDrainLimit);   // after an abort
  }

  // ---- teardown -------------------------------------------------------------
  // neither CTA leaves while the other may still write into its shared
  // memory, arrive on its barriers or run MMAs on its TMEM
  fence_before_sync();
  __syncwarp();     // the cluster barrier is warp-aligned
  cluster_sync();
  fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, C::kTmemCols);
}

template <int kMode>
pa_status launch_gemm(const GemmArgs &a, cudaStream_t stream) {
  int32_t *status;
  int sms;
  cudaError_t e = device_context(&status, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  CUtensorMap mx, mw, mw2, mr, my;
  if (!make_map_2d(&mx, a.x, a.M, a.K, a.x_stride, kBM) ||
      !make_map_2d(&mw, a.w, a.N, a.K, a.K, kBN / kCluster) ||
      !make_map_2d(&mw2, kMode == kGated ? a.w2 : a.w, a.N, a.K, a.K, kBN / kCluster) ||
      !make_map_2d(&mr, a.residual ? a.residual : a.y, a.M, a.N,
                   a.residual ? a.residual_stride : a.y_stride, 32) ||
      !make_map_2d(&my, a.y, a.M, a.N, a.y_stride, 32))
    return from_cuda(cudaErrorInvalidValue);
  GemmParams p;
  p.bias = static_cast<const __nv_bfloat16 *>(a.bias);
  p.residual = a.residual != nullptr;
  p.act = a.act;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  const int tile_n = kMode == kGated ? kBN / 2 : kBN;
  p.tiles_n = (a.N - 1) / tile_n + 1;
  p.tiles_m = (a.M - 1) / (kCluster * kBM) + 1;
  const int64_t pairs = int64_t{p.tiles_m} * p.tiles_n;
  if (pairs > 0x3fffffff) return PA_ERR_UNSUPPORTED;
  p.n_pairs = static_cast<int>(pairs);
  p.k_blocks = (a.K - 1) / kBK + 1;
  p.status = status;
  static unsigned long long configured = 0;
  e = set_smem_once(reinterpret_cast<const void *>(linear_bf16_kernel<kMode>),
                    GemmCfg::kSmemBytes, configured);
  if (e != cudaSuccess) return from_cuda(e);
  // whole clusters, at most one CTA per SM
  const int max_ctas = sms / kCluster * kCluster;
  const int grid = kCluster * p.n_pairs < max_ctas ? kCluster * p.n_pairs : max_ctas;
  return from_cuda(launch_beside(linear_bf16_kernel<kMode>, dim3(grid), kThreads,
                                 GemmCfg::kSmemBytes, stream, mx, mw, mw2, mr, my, p));
}

// Largest row stride, in elements (TMA strides are below 2^40 bytes).
constexpr int64_t kMostStride = int64_t{1} << 38;

// Longest sum where the kernel for few rows may be taken: half a second or so at most,
// which has to end within that kernel's waits for it.
constexpr int32_t kMostK = 1 << 26;

// The checks of the entry points with strides (bias, residual: may be null).
pa_status check_gemm(const GemmArgs &a) {
  if (a.M < 0 || a.N < 1 || a.K < 1 || a.act < PA_ACT_NONE || a.act > PA_ACT_GELU_TANH)
    return PA_ERR_INVALID_ARG;
  if (a.M > 0 && (!a.x || !a.y)) return PA_ERR_INVALID_ARG;
  if (a.x_stride < a.K || a.y_stride < a.N || (a.residual && a.residual_stride < a.N) ||
      (a.residual && a.residual == a.y && a.residual_stride != a.y_stride))
    return PA_ERR_INVALID_ARG;
  if (a.K > kMostK || a.x_stride > kMostStride || a.y_stride > kMostStride || a.residual_stride > kMostStride)
    return PA_ERR_UNSUPPORTED;
  if (((a.K | a.N | a.x_stride | a.y_stride) & 7) != 0 ||
      (a.residual && (a.residual_stride & 7) != 0) || !aligned_to(a.x, 16) ||
      !aligned_to(a.w, 16) || !aligned_to(a.w2, 16) || !aligned_to(a.y, 16) ||
      !aligned_to(a.bias, 16) || !aligned_to(a.residual, 16))
    return PA_ERR_MISALIGNED;
  return PA_OK;
}

template <int kMode>
pa_status linear_call(const GemmArgs &a, cudaStream_t stream) {
  pa_status st = check_gemm(a);
  if (st != PA_OK || a.M == 0) return st;
  bool taken = false;
  st = launch_linear_few(a, kMode, taken, stream);
  return taken ? st : launch_gemm<kMode>(a, stream);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status pa_linear_bf16(const void *x, const void *w, const void *bias, void *y,
                                    int32_t M, int32_t N, int32_t K, pa_stream_t stream) {
  using namespace pa;
  if (M < 0 || N < 1 || K < 1 || !w) return PA_ERR_INVALID_ARG;
  if (M == 0) return PA_OK;   // nothing to read or write; x and y may be NULL
  if (!x || !y) return PA_ERR_INVALID_ARG;
  if ((K & 7) != 0 || (N & 7) != 0 || !aligned16(x) || !aligned16(w) || !aligned16(y) ||
      (bias && !aligned16(bias)))
    return PA_ERR_MISALIGNED;
  const GemmArgs a{x, w, nullptr, bias, nullptr, y, M, N, K, K, 0, N, PA_ACT_NONE};
  return launch_gemm<kLinear>(a, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_linear_act_bf16(const void *x, const void *w, const void *bias,
                                        const void *residual, void *y, int32_t M, int32_t N,
                                        int32_t K, int64_t x_stride, int64_t residual_stride,
                                        int64_t y_stride, int32_t act, pa_stream_t stream) {
  using namespace pa;
  if (!w) return PA_ERR_INVALID_ARG;
  const GemmArgs a{x, w, nullptr, bias, residual, y, M, N, K, x_stride, residual_stride, y_stride,
                   act};
  return linear_call<kAct>(a, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_linear_gated_bf16(const void *x, const void *w_gate, const void *w_up,
                                          void *y, int32_t M, int32_t N, int32_t K,
                                          int64_t x_stride, int64_t y_stride, int32_t act,
                                          pa_stream_t stream) {
  using namespace pa;
  if (!w_gate || !w_up) return PA_ERR_INVALID_ARG;
  const GemmArgs a{x, w_gate, w_up, nullptr, nullptr, y, M, N, K, x_stride, 0, y_stride, act};
  return linear_call<kGated>(a, reinterpret_cast<cudaStream_t>(stream));
}
