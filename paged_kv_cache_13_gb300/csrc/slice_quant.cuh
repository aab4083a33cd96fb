// Multi-query attention over the quantised cache, many rows per (sequence, KV
// head): the arguments both kernels take (multi_query_quant.cu) and the
// tensor-core kernel's launch (slice_quant.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

struct QuantCache {
    const void* q;
    const int32_t* q_start;
    const uint8_t* codes[2];  // K, V
    const __half* scale[2];
    const __half* zero[2];
    const void* sink[2];
    const void* win[2];
    int n_sink, window, ring;
    const int32_t* tables;
    const int32_t* ctx_lens;
    int batch, hq, hkv, G, num_blocks, max_blocks, max_q_len;
    int groups;  // (scale, zero) pairs per token and head
    bool int4;
    float scale_log2;
    void* out;
    int* status;
};

// Bytes of the split's partials, 0 when the call is not split.
size_t slice_quant_workspace(int64_t batch, int64_t hq, int64_t hkv, int64_t D, int64_t max_blocks, int64_t max_q_len);

// Arguments already checked; workspace as slice_quant_workspace says.
int launch_slice_quant(const QuantCache& a, int D, bool bf16, float* workspace, cudaStream_t st);

}  // namespace pkv
