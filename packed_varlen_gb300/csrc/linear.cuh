// What the linear layers' kernels share: a call's arguments, and the copies'
// maps.  gemm_tc.cu computes large calls, linear_few.cu those of few rows.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "tma_map.h"

namespace pa {

enum GemmMode { kLinear, kAct, kGated };

constexpr int kLinearBK = 64;   // depth of a K-block: 128 bytes, a swizzle row

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// [rows, K] bf16, rows row_elems apart, as a 2-D tensor (K, rows); box 64 x
// box_rows with 128-byte swizzle: one K-block of box_rows rows per load.
// Rows and columns past the end read as zero.
inline bool make_map_2d(CUtensorMap *map, const void *ptr, int rows, int K, int64_t row_elems,
                        int box_rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_elems) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kLinearBK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One call, as the entry points receive it (strides in elements).
struct GemmArgs {
  const void *x, *w, *w2, *bias, *residual;
  void *y;
  int32_t M, N, K;
  int64_t x_stride, residual_stride, y_stride;
  int32_t act;
};

// A call of mode kAct or kGated by the kernel for few rows, where it is the faster
// one (`taken`; else nothing is done).
pa_status launch_linear_few(const GemmArgs &a, int mode, bool &taken, cudaStream_t stream);

}  // namespace pa
