// Attention of packed prompts, causal and with grouped heads: the entry point.
// The kernels are those of pa_varlen_attn_fwd (attn_pair.cu, attn_tc.cu), which is
// the call with groups of one head and no causal order.
#include <math.h>

#include "internal.h"
#include "varlen_items.cuh"

namespace pa {
namespace {

// Largest token counts: sums of two stay within 32 bits.
constexpr int32_t kMostTokens = 1 << 30;
// Largest row stride, in elements (TMA strides are below 2^40 bytes).
constexpr int64_t kMostStride = int64_t{1} << 38;

}  // namespace
}  // namespace pa

extern "C" pa_status pa_prompt_attn_fwd(const void *q, const void *k, const void *v, void *out,
                                        const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                        int32_t batch, int32_t total_q, int32_t total_k,
                                        int32_t max_q, int32_t max_k, int64_t q_stride,
                                        int64_t k_stride, int64_t v_stride, int32_t Hq,
                                        int32_t Hkv, int32_t D, int32_t causal, float scale,
                                        pa_stream_t stream) {
  using namespace pa;
  if (!cu_seqlens_q || !cu_seqlens_k) return PA_ERR_INVALID_ARG;
  if (batch < 1 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0 || Hq < 1 || Hkv < 1 ||
      Hq % Hkv != 0 || D < 1)
    return PA_ERR_INVALID_ARG;
  if ((total_q > 0 && (!q || !out)) || (total_k > 0 && (!k || !v))) return PA_ERR_INVALID_ARG;
  if (q_stride < int64_t{Hq} * D || k_stride < int64_t{Hkv} * D || v_stride < int64_t{Hkv} * D)
    return PA_ERR_INVALID_ARG;
  if (!isfinite(scale * 1.4426950408889634f)) return PA_ERR_INVALID_ARG;
  if (Hq / Hkv > kVarlenTile) return PA_ERR_UNSUPPORTED;
  // (every sequence's last item may be a partial one)
  const int64_t items = (total_q / (2 * (kVarlenTile / (Hq / Hkv))) + int64_t{batch}) * Hkv;
  if (batch > PA_MAX_BATCH || (D != 64 && D != 128) || Hq > 65535 || total_q > kMostTokens ||
      total_k > kMostTokens || items > kMostTokens || q_stride > kMostStride ||
      k_stride > kMostStride || v_stride > kMostStride)
    return PA_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) ||
      !aligned_to(cu_seqlens_q, 4) || !aligned_to(cu_seqlens_k, 4) || (q_stride & 7) != 0 ||
      (k_stride & 7) != 0 || (v_stride & 7) != 0)
    return PA_ERR_MISALIGNED;
  if (total_q == 0 || max_q == 0) return PA_OK;  // no query rows: nothing to write
  if (total_k == 0) {   // no row is read, but the copies' maps need an address
    k = v = q;
    k_stride = v_stride = int64_t{Hkv} * D;
  }
  VarlenArgs a{q, k, v, out, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, max_q,
               max_k, Hq, D, scale, nullptr, 0, Hkv, causal != 0, q_stride, k_stride, v_stride};
  cudaError_t e = device_context(&a.status, &a.num_sms);
  if (e != cudaSuccess) return from_cuda(e);
  return from_cuda(launch_varlen_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}
