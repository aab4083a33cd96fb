// Multi-query attention over the quantised cache for more than 24 rows per
// (sequence, KV head): slices of a prompt, wide verify passes.
// One warp per (query token, query head) row: the lanes share the head dim,
// the keys are taken one at a time with an online softmax in fp32.

#include "slice_quant.cuh"

#include "common.cuh"

namespace pkv {
namespace {

constexpr int BS = 16;

// E consecutive values, from column col on, of the K (x = 0) or V (x = 1) row
// at position t of sequence b; false on a bad table entry.
template <typename T, int D, int QMODE, int E>
__device__ __forceinline__ bool row_values(const QuantCache& a, int x, int b, int kvh, int t, int w0, int group, int col,
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
__global__ void slice_rows_kernel(const __grid_constant__ QuantCache a, int group) {
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
void launch_rows(const QuantCache& a, int group, cudaStream_t st) {
    slice_rows_kernel<T, D, QMODE><<<dim3((a.max_q_len + 3) / 4, a.hq, a.batch), 128, 0, st>>>(a, group);
}

template <typename T>
void launch_rows_t(const QuantCache& a, int D, cudaStream_t st) {
    const int group = D / a.groups;
    if (D == 128 && a.int4) launch_rows<T, 128, PKV_QMODE_INT4_ASYM>(a, group, st);
    else if (D == 128) launch_rows<T, 128, PKV_QMODE_FP8_E4M3>(a, group, st);
    else if (a.int4) launch_rows<T, 64, PKV_QMODE_INT4_ASYM>(a, group, st);
    else launch_rows<T, 64, PKV_QMODE_FP8_E4M3>(a, group, st);
}

}  // namespace

size_t slice_quant_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

int launch_slice_quant(const QuantCache& a, int D, bool bf16, float*, cudaStream_t st) {
    if (bf16) launch_rows_t<__nv_bfloat16>(a, D, st);
    else launch_rows_t<__half>(a, D, st);
    return launch_status();
}

}  // namespace pkv
