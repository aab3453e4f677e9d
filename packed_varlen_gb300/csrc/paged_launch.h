// Launchers of the paged attention kernels (paged_attn.cu calls them).
#pragma once

#include <cuda_runtime.h>

namespace pa {

struct PagedAttnParams;   // paged.cuh

// Sequences of at most kDecodeRows rows: streaming kernel, and the join of its parts.
cudaError_t launch_paged_decode(const PagedAttnParams &p, bool quant, int num_sms,
                                cudaStream_t stream);

// Whether that kernel joins its parts itself and needs no workspace.
bool paged_decode_is_local(int batch, int tokens, int max_k, int G, int Hkv);

// Longer sequences: tiled kernel, and the join of the parts that its shares leave.
cudaError_t launch_paged_chunk(const PagedAttnParams &p, bool quant, int num_sms,
                               cudaStream_t stream);

}  // namespace pa
