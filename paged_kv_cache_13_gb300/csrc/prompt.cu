// Attention of packed prompts over their own (unpaged) K/V rows:
// pkv_prompt_attention.
//
// What it computes: query row i of sequence b sits at position p = S_b - L_b
// + i of its S_b K/V rows, and
//   out[q_start[b] + i, h] = sum_{t <= p} softmax_t(scale <q, k_t>) v_t
// over KV head h / G ("The 8GB VRAM Breakthrough", §5: the prefill that
// precedes the decode loop).  One warp per (query row, query head): the lanes
// share the head dim, the keys are taken one at a time with an online softmax
// in fp32.

#include <math.h>

#include "common.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct PromptArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* q_start;
    const int32_t* kv_start;
    int batch, T, S, hq, hkv;
    int64_t qs, ks, vs;
    float scale_log2;
    void* out;
    int* status;
};

// The sequence of query row t: the last b with q_start[b] <= t.
__device__ __forceinline__ int sequence_of(const int32_t* q_start, int batch, int t) {
    int lo = 0, hi = batch;  // q_start[lo] <= t < q_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (q_start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T, int D>
__global__ void prompt_rows_kernel(PromptArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.T) * a.hq) return;
    if (row == 0) {  // the ranges are checked once per call
        bool bad = false;
        for (int j = lane; j < a.batch; j += 32) {
            const int q0 = a.q_start[j], q1 = a.q_start[j + 1], k0 = a.kv_start[j], k1 = a.kv_start[j + 1];
            bad |= q0 < 0 || q1 < q0 || q1 > a.T || k0 < 0 || k1 < k0 || k1 > a.S || k1 - k0 < q1 - q0;
        }
        if (bad) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
    }
    const int t = static_cast<int>(row / a.hq), h = static_cast<int>(row % a.hq);
    const int b = sequence_of(a.q_start, a.batch, t);
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
    if (t < q0 || t >= q1) return;  // a row of no sequence
    const int k0 = a.kv_start[b], k1 = a.kv_start[b + 1];
    const int ka = max(k0, 0), kb = min(k1, a.S);
    const int last = min(k0 + (k1 - k0) - (q1 - q0) + (t - q0), kb - 1);
    const T* q = static_cast<const T*>(a.q) + t * a.qs + h * D + lane * E;
    const int kvh = h / (a.hq / a.hkv);
    float x[E], o[E], m = neg_inf(), l = 0.f;
    for (int e = 0; e < E; ++e) {
        x[e] = Half16<T>::to_float(q[e]);
        o[e] = 0.f;
    }
    for (int j = ka; j <= last; ++j) {
        const T* k = static_cast<const T*>(a.k) + j * a.ks + kvh * D + lane * E;
        const T* v = static_cast<const T*>(a.v) + j * a.vs + kvh * D + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += x[e] * Half16<T>::to_float(k[e]);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale_log2;
        if (s == neg_inf()) continue;
        const float mn = fmaxf(m, s);
        const float al = ex2(m - mn), p = ex2(s - mn);
        m = mn;
        l = l * al + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * al + p * Half16<T>::to_float(v[e]);
    }
    T* out = static_cast<T*>(a.out) + row * D + lane * E;
    for (int e = 0; e < E; ++e) out[e] = Half16<T>::from_float(l > 0.f || l != l ? o[e] / l : 0.f);
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_prompt_attention_workspace_bytes(int32_t batch, int32_t num_tokens, int32_t num_kv_tokens,
                                                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                    size_t* out) {
    if (!out || batch < 0 || num_tokens < 0 || num_kv_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || num_q_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    *out = 0;
    return PKV_OK;
}

extern "C" int pkv_prompt_attention(const void* q, const void* k, const void* v, const int32_t* q_start,
                                    const int32_t* kv_start, int32_t batch, int32_t num_tokens,
                                    int32_t num_kv_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t head_dim, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                    float scale, void* out, void* workspace, size_t workspace_bytes, int dtype,
                                    void* stream) {
    if (batch < 0 || num_tokens < 0 || num_kv_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0 || !isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || num_q_heads / num_kv_heads > 128 || num_kv_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    const int64_t dq = static_cast<int64_t>(num_q_heads) * head_dim, dk = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (q_stride < dq || k_stride < dk || v_stride < dk) return PKV_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !q_start || !out || (num_kv_tokens > 0 && (!k || !v))) return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(q) || !pkv::aligned16(k) || !pkv::aligned16(v) || !pkv::aligned16(out) || q_stride % 8 != 0 ||
        k_stride % 8 != 0 || v_stride % 8 != 0 || (reinterpret_cast<uintptr_t>(q_start) & 3u) ||
        (reinterpret_cast<uintptr_t>(kv_start) & 3u))
        return PKV_ERR_MISALIGNED;
    int* st = pkv::status_word();
    if (!st) return PKV_ERR_CUDA;
    pkv::PromptArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_start = q_start;
    a.kv_start = kv_start ? kv_start : q_start;
    a.batch = batch;
    a.T = num_tokens;
    a.S = num_kv_tokens;
    a.hq = num_q_heads;
    a.hkv = num_kv_heads;
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.scale_log2 = scale * pkv::kLog2e;
    a.out = out;
    a.status = st;
    const int64_t rows = static_cast<int64_t>(num_tokens) * num_q_heads;
    const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_DTYPE_BF16) {
        if (head_dim == 128) pkv::prompt_rows_kernel<__nv_bfloat16, 128><<<grid, 128, 0, cs>>>(a);
        else pkv::prompt_rows_kernel<__nv_bfloat16, 64><<<grid, 128, 0, cs>>>(a);
    } else {
        if (head_dim == 128) pkv::prompt_rows_kernel<__half, 128><<<grid, 128, 0, cs>>>(a);
        else pkv::prompt_rows_kernel<__half, 64><<<grid, 128, 0, cs>>>(a);
    }
    return pkv::launch_status();
}
