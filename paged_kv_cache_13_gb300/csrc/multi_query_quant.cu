// Multi-query attention over the quantised cache:
// pkv_paged_attention_multi_query_quant.
//
// What it computes: the masks and positions of multi_query.cu (query i of
// sequence b at p = ctx_b - L_b + i, causal) over the values of
// decode_quant.cu: (c - z) s for INT4, e4m3(c) s for FP8, 16-bit rows for
// positions < n_sink and for the window blocks of the sequence ("The 8GB VRAM
// Breakthrough", §4 with §6: the verify pass over the quantised cache).
// One warp per (query token, query head) row: the lanes share the head dim,
// the keys are taken one at a time with an online softmax in fp32.

#include <math.h>

#include "balanced.cuh"

namespace pkv {
namespace {

constexpr int BS = 16;
constexpr float kLog2e = 1.4426950408889634f;

struct MQQArgs {
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
    float scale_log2;
    void* out;
    int* status;
};

// E consecutive values, from column col on, of the K (x = 0) or V (x = 1) row
// at position t of sequence b; false on a bad table entry.
template <typename T, int D, int QMODE, int E>
__device__ __forceinline__ bool row_values(const MQQArgs& a, int x, int b, int kvh, int t, int w0, int group, int col,
                                           float (&v)[E]) {
    const T* src = nullptr;
    if (t >= w0)
        src = static_cast<const T*>(a.win[x]) +
              (((static_cast<int64_t>(b) * a.ring + (t / BS) % a.ring) * a.hkv + kvh) * BS + t % BS) * D;
    else if (t < a.n_sink)
        src = static_cast<const T*>(a.sink[x]) + ((static_cast<int64_t>(b) * a.n_sink + t) * a.hkv + kvh) * D;
    if (src) {
        for (int e = 0; e < E; ++e) v[e] = Half16<T>::to_float(src[col + e]);
        return true;
    }
    const int phys = a.tables[static_cast<int64_t>(b) * a.max_blocks + t / BS];
    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(a.num_blocks)) return false;
    const int64_t row = (static_cast<int64_t>(phys) * a.hkv + kvh) * BS + t % BS;
    for (int e = 0; e < E; ++e) {
        const int d = col + e;
        if (QMODE == PKV_QMODE_INT4_ASYM) {
            const int ng = D / group, gi = d / group;
            const int c = (a.codes[x][row * (D / 2) + d / 2] >> (4 * (d & 1))) & 15;
            v[e] = (c - __half2float(a.zero[x][row * ng + gi])) * __half2float(a.scale[x][row * ng + gi]);
        } else {
            unsigned pair;
            const unsigned short code = a.codes[x][row * D + d];
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(pair) : "h"(code));
            v[e] = __half2float(__ushort_as_half(static_cast<unsigned short>(pair & 0xffff))) *
                   __half2float(a.scale[x][row]);
        }
    }
    return true;
}

template <typename T, int D, int QMODE>
__global__ void mqq_rows_kernel(MQQArgs a, int group) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int h = blockIdx.y, b = blockIdx.z, kvh = h / a.G;
    const int q0 = a.q_start[b], L = a.q_start[b + 1] - q0;
    const int cap = a.max_blocks * BS;
    int ctx = a.ctx_lens[b];
    if (L <= 0 || i >= min(L, a.max_q_len)) return;
    if ((ctx < L || ctx > cap || L > a.max_q_len) && lane == 0 && h == 0 && i == 0)
        atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
    ctx = min(max(ctx, 0), cap);
    const int pos = ctx - L + i;
    const int w0 = a.window > 0 ? max(ctx - a.window, 0) / BS * BS : ctx;
    const T* q = static_cast<const T*>(a.q) + ((static_cast<int64_t>(q0) + i) * a.hq + h) * D + lane * E;
    float x[E], o[E], m = neg_inf(), l = 0.f;
    for (int e = 0; e < E; ++e) {
        x[e] = Half16<T>::to_float(q[e]);
        o[e] = 0.f;
    }
    for (int t = 0; t <= pos; ++t) {
        float v[E];
        if (!row_values<T, D, QMODE, E>(a, 0, b, kvh, t, w0, group, lane * E, v)) {
            if (lane == 0) atomicOr(a.status, PKV_STATUS_BAD_BLOCK);
            continue;
        }
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += x[e] * v[e];
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale_log2;
        if (s == neg_inf()) continue;
        const float mn = fmaxf(m, s);
        const float al = ex2(m - mn), p = ex2(s - mn);
        m = mn;
        l = l * al + p;
        row_values<T, D, QMODE, E>(a, 1, b, kvh, t, w0, group, lane * E, v);
        for (int e = 0; e < E; ++e) o[e] = o[e] * al + p * v[e];
    }
    T* out = static_cast<T*>(a.out) + ((static_cast<int64_t>(q0) + i) * a.hq + h) * D + lane * E;
    for (int e = 0; e < E; ++e) out[e] = Half16<T>::from_float(l > 0.f || l != l ? o[e] / l : 0.f);
}

template <typename T, int D, int QMODE>
void launch_rows(const MQQArgs& a, int group, cudaStream_t st) {
    mqq_rows_kernel<T, D, QMODE><<<dim3((a.max_q_len + 3) / 4, a.hq, a.batch), 128, 0, st>>>(a, group);
}

template <typename T>
void launch_rows_t(const MQQArgs& a, int D, int qmode, int group, cudaStream_t st) {
    const bool int4 = qmode == PKV_QMODE_INT4_ASYM;
    if (D == 128 && int4) launch_rows<T, 128, PKV_QMODE_INT4_ASYM>(a, group, st);
    else if (D == 128) launch_rows<T, 128, PKV_QMODE_FP8_E4M3>(a, group, st);
    else if (int4) launch_rows<T, 64, PKV_QMODE_INT4_ASYM>(a, group, st);
    else launch_rows<T, 64, PKV_QMODE_FP8_E4M3>(a, group, st);
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_multi_query_quant_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                     int32_t head_dim, int32_t max_blocks, int32_t block_size,
                                                     int32_t max_q_len, size_t* out) {
    if (!out || batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_blocks < 0 ||
        block_size <= 0 || max_q_len < 0 || num_q_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != pkv::BS) return PKV_ERR_UNSUPPORTED;
    *out = 0;
    return PKV_OK;
}

extern "C" int pkv_paged_attention_multi_query_quant(
    const void* q, const int32_t* q_start, const void* k_codes, const void* k_scale, const void* k_zero,
    const void* v_codes, const void* v_scale, const void* v_zero, const void* sink_k, const void* sink_v,
    int32_t n_sink, const void* win_k, const void* win_v, int32_t window, const int32_t* block_tables,
    const int32_t* context_lens, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t num_blocks, int32_t block_size, int32_t max_blocks, int32_t max_q_len, int32_t group_size, float scale,
    void* out, void* workspace, size_t workspace_bytes, int qmode, int dtype, void* stream) {
    if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || block_size <= 0 ||
        max_blocks < 0 || max_q_len < 0 || n_sink < 0 || window < 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_INVALID_ARG;
    if (qmode != PKV_QMODE_INT4_ASYM && qmode != PKV_QMODE_FP8_E4M3) return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0 || !isfinite(scale) || window % block_size != 0) return PKV_ERR_INVALID_ARG;
    const bool int4 = qmode == PKV_QMODE_INT4_ASYM;
    if (block_size != pkv::BS || (head_dim != 64 && head_dim != 128) || num_q_heads / num_kv_heads > 8 ||
        n_sink > block_size || batch > 65535 || num_kv_heads > 8191 || max_q_len > (1 << 17) ||
        static_cast<int64_t>(max_blocks) * block_size > (1LL << 30))
        return PKV_ERR_UNSUPPORTED;
    if (int4 && group_size != head_dim && group_size != 64) return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || max_q_len == 0) return PKV_OK;
    if (!q || !q_start || !k_codes || !k_scale || !v_codes || !v_scale || !block_tables || !context_lens || !out ||
        (int4 && (!k_zero || !v_zero)) || (n_sink > 0 && (!sink_k || !sink_v)) || (window > 0 && (!win_k || !win_v)))
        return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(q) || !pkv::aligned16(k_codes) || !pkv::aligned16(v_codes) || !pkv::aligned16(k_scale) ||
        !pkv::aligned16(v_scale) || !pkv::aligned16(out) ||
        (int4 && (!pkv::aligned16(k_zero) || !pkv::aligned16(v_zero))) ||
        (n_sink > 0 && (!pkv::aligned16(sink_k) || !pkv::aligned16(sink_v))) ||
        (window > 0 && (!pkv::aligned16(win_k) || !pkv::aligned16(win_v))) ||
        (reinterpret_cast<uintptr_t>(q_start) & 3u) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(context_lens) & 3u))
        return PKV_ERR_MISALIGNED;
    int* st = pkv::status_word();
    if (!st) return PKV_ERR_CUDA;
    pkv::MQQArgs a;
    a.q = q;
    a.q_start = q_start;
    a.codes[0] = static_cast<const uint8_t*>(k_codes);
    a.codes[1] = static_cast<const uint8_t*>(v_codes);
    a.scale[0] = static_cast<const __half*>(k_scale);
    a.scale[1] = static_cast<const __half*>(v_scale);
    a.zero[0] = static_cast<const __half*>(k_zero);
    a.zero[1] = static_cast<const __half*>(v_zero);
    a.sink[0] = sink_k;
    a.sink[1] = sink_v;
    a.win[0] = win_k;
    a.win[1] = win_v;
    a.n_sink = n_sink;
    a.window = window;
    a.ring = window / block_size + 1;
    a.tables = block_tables;
    a.ctx_lens = context_lens;
    a.batch = batch;
    a.hq = num_q_heads;
    a.hkv = num_kv_heads;
    a.G = num_q_heads / num_kv_heads;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks;
    a.max_q_len = max_q_len;
    a.scale_log2 = scale * pkv::kLog2e;
    a.out = out;
    a.status = st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_DTYPE_BF16) pkv::launch_rows_t<__nv_bfloat16>(a, head_dim, qmode, group_size, cs);
    else pkv::launch_rows_t<__half>(a, head_dim, qmode, group_size, cs);
    return pkv::launch_status();
}
