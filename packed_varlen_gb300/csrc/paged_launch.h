// Launchers of the paged attention kernels (paged_attn.cu calls them).
#pragma once

#include <cuda_runtime.h>

namespace pa {

struct PagedAttnParams;   // paged.cuh

// Sequences of more than kFewRows rows: tiled kernel.
cudaError_t launch_paged_chunk(const PagedAttnParams &p, bool quant, int num_sms,
                               cudaStream_t stream);

// 8-bit rows of the sequences that chunk_widens() names, as bf16 (kv_cache.cu).
cudaError_t launch_paged_widen(const PagedAttnParams &p, int num_sms, cudaStream_t stream);

// The others: streaming kernel; after_chunk: launched behind the tiled one.
cudaError_t launch_paged_decode(const PagedAttnParams &p, bool quant, int num_sms,
                                bool after_chunk, cudaStream_t stream);
// Whether that kernel joins its parts itself and needs no workspace.
bool paged_decode_is_local(int batch, int tokens, int max_k, int G, int Hkv);

// Join of the parts that both leave, behind whichever was launched last.
cudaError_t launch_paged_join(const PagedAttnParams &p, int num_sms, cudaStream_t stream);

}  // namespace pa
