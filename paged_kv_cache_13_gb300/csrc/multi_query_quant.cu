// Multi-query attention over the quantised cache:
// pkv_paged_attention_multi_query_quant.
//
// What it computes: the masks and positions of multi_query.cu (query i of
// sequence b at p = ctx_b - L_b + i, causal) over the values of
// decode_quant.cu: (c - z) s for INT4, e4m3(c) s for FP8, 16-bit rows for
// positions < n_sink and for the window blocks of the sequence ("The 8GB VRAM
// Breakthrough", §4 with §6: the verify pass over the quantised cache).
//
// Up to 24 (query token, query head) rows per (sequence, KV head) -- gamma + 1
// = 6 tokens at a GQA group of 4 -- take the balanced split of balanced.cuh:
// warp i streams an equal share of the call's (sequence, KV head, 16-token
// block) items and holds all rows of its runs, NT n-tiles of 8, so each code
// is read and unpacked once for all of them; a merge kernel folds the partial
// rows behind it.  More rows go to slice_quant.cu.
//
// The MMAs (mma.sync m16n8k16, tokens as M of QK^T, head dim as M of PV, rows
// as N) see exact codes, the scales and zero points factored out:
//   QK^T: S_t = s_t (sum_d q_d c_td - z_t sum_d q_d)
//   PV:   O_d = sum_t W_t c_td - sum_t W_t z_t,  W_t = P_t s_t (fp16)
// INT4 codes of K are used as fp16 subnormals (a nibble masked in place: c
// 2^-24, the next nibble 16 c 2^-24; the query columns that meet the latter are
// divided by 16), those of V as c - 8 (the nibble put under 1024's mantissa,
// 1032 taken off; 16 (c - 8) for the next nibble, undone at the end): sums over
// a long context of codes that are all positive, less the zero points', would
// lose ten bits to cancellation (16k tokens: 1.5e-3 relative).  FP8 codes
// convert exactly.  sum_t W_t (z_t - 8) is one more MMA per n-tile: the zero
// points as a 17th row of V, for fp16 what rounding z - 8 left as an 18th
// (without it outputs were off by 4.2e-4 instead of 2.9e-4; bf16 ones, off by
// 1.8e-3 either way, would pay 6% of the time for it).
// Sinks and window blocks are 16-bit blocks attended after the quantised ones
// of a run, with the accumulator taken to true units first.
//
// A block's K and V codes, scales and zero points are 6 contiguous runs (4 for
// FP8): lanes 0 .. 5 copy one each into the warp's ring of kStages blocks in
// shared memory (untiled asynchronous copies, one mbarrier a stage), kStages
// blocks ahead; 16-bit blocks go through the same ring, two at a time.
// Bound: HBM in bytes (1,088 per token and layer for 8 heads of INT4), in
// practice the chains of the 8 warps an SM's registers hold at 24 rows: 42% of
// the issue slots, 517 instructions a block (32 x 16,384 tokens, 8 heads, 6
// queries, INT4: 263 us, 2,178 GB/s; FP8, 64 x 512 .. 4,096, 2 .. 4 queries: 84
// us, 3,610 GB/s).  The next block's QK^T beside this one's PV was slower (277
// us, it spills), scalar arithmetic for the packed pairs no faster.

#include <math.h>

#include "balanced.cuh"
#include "slice_quant.cuh"
#include "tc5.cuh"

#include <type_traits>

namespace pkv {
namespace {

using namespace tc5;

constexpr int BS = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;           // log2 units a logit may exceed the reference maximum by
constexpr float kLazyMaxScale = 128.f;  // V scales above it take the exact maximum (W = P s stays in fp16)
constexpr float kNoMax = -1e30f;        // reference maximum of a row that has seen no token
constexpr float kTwo24 = 16777216.f;    // 2^24
constexpr int kWarps = 2;               // warps per CTA
constexpr int kMaxNT = 3;               // n-tiles of 8 rows per warp, at most
constexpr int kStages = 4;              // quantised blocks in a warp's ring
// resident CTAs per SM, as the registers of NT n-tiles (and, for one, the
// rings) allow
constexpr int ctas_per_sm(int nt) { return nt == 3 ? 4 : 5; }
// Fewest items a warp takes: short runs cost a partial row set each, which
// the merge reads back.
constexpr int kMinItems = 8;

__device__ __forceinline__ uint32_t nib_even(uint32_t w) { return w & 0x000F000Fu; }
__device__ __forceinline__ uint32_t nib_odd(uint32_t w) { return w & 0x00F000F0u; }
__device__ __forceinline__ uint32_t f16pair(float lo, float hi) { return Half16<__half>::pack(lo, hi); }
__device__ __forceinline__ uint32_t sub16x2(uint32_t a, uint32_t b) {
    const __half2 d = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    Half16<__half>::mma(d, a0, a1, a2, a3, b0, b1);
}
// two e4m3 codes in the low 16 bits of w -> fp16 pair
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {
    uint32_t d;
    const unsigned short a = static_cast<unsigned short>(w & 0xffffu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(a));
    return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(addr));
    return r;
}
template <typename T>
constexpr bool kFine = std::is_same<T, __half>::value;  // see Scales
template <typename T>
constexpr bool kSplitP = false;
template <>
constexpr bool kSplitP<__nv_bfloat16> = true;

// The element of PV that m-tile mt, half hf (M rows g / g + 8) holds for lane
// group g, and its head-dim column.  One column group per head: the lane
// group's D / 8 consecutive columns; two groups of 64 (NG = 2): 8 columns of
// each group, both halves of an m-tile in one group (its weights).
template <int D, int NG>
__host__ __device__ constexpr int pv_e(int mt, int hf) {
    return NG == 1 ? mt + hf * (D / 16) : 8 * (mt / 4) + mt % 4 + 4 * hf;
}
template <int D, int NG>
__device__ __forceinline__ int pv_column(int e, int g) {
    return NG == 1 ? g * (D / 8) + e : (e >> 3) * 64 + 8 * g + (e & 7);
}

template <int D, int QMODE, int NG>
struct Shape {
    static constexpr bool INT4 = QMODE == PKV_QMODE_INT4_ASYM;
    static constexpr int KSTEPS = D / 16;              // k-steps of QK^T
    static constexpr int MT = D / 16;                  // m-tiles of PV
    static constexpr int CB = INT4 ? D / 2 : D;        // code bytes per row
    static constexpr int KW = INT4 ? D / 32 : D / 16;  // 32-bit K-code words per lane and row
    static constexpr int VW = INT4 ? D / 64 : D / 32;  // 32-bit V-code words per lane and row
    static constexpr int KPG = KW / NG, VPG = VW / NG;
    // a block of one KV head in the ring: K codes, V codes, then the scales of
    // K and V and the zero points of K and V
    static constexpr int CODES = BS * CB, SCALES = BS * NG * 2;
    static constexpr int COPIES = INT4 ? 6 : 4;
    static constexpr int STAGE = 2 * CODES + (COPIES - 2) * SCALES;
    static constexpr int STAGE16 = 2 * BS * D * 2;  // a 16-bit block: K rows, V rows
    static_assert(NG == 1 || (INT4 && D == 128 && NG == 2), "groups: one per head, or 64 columns at D 128");
};

// One block's codes of a lane, from the ring: K rows g, g + 8; V rows 2c, 2c +
// 1, 8 + 2c, 9 + 2c.  p points at the lane's first bytes of the first row.
template <int D, int QMODE, int NG>
struct KCodes {
    using S = Shape<D, QMODE, NG>;
    uint32_t r0[S::KW], r1[S::KW];
    __device__ __forceinline__ void load(const uint8_t* p) {
        if constexpr (!S::INT4) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) put<4>(4 * i, p + 64 * i);
        } else if constexpr (NG == 2) {
            put<2>(0, p);
            put<2>(2, p + 32);
        } else {
            put<S::KW>(0, p);
        }
    }
    template <int N>
    __device__ __forceinline__ void put(int at, const uint8_t* p) {
        if constexpr (N == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 8 * S::CB);
            r0[at] = x.x; r0[at + 1] = x.y; r0[at + 2] = x.z; r0[at + 3] = x.w;
            r1[at] = y.x; r1[at + 1] = y.y; r1[at + 2] = y.z; r1[at + 3] = y.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(p + 8 * S::CB);
            r0[at] = x.x; r0[at + 1] = x.y;
            r1[at] = y.x; r1[at + 1] = y.y;
        }
    }
};

template <int D, int QMODE, int NG>
struct VCodes {
    using S = Shape<D, QMODE, NG>;
    uint32_t r[4][S::VW];
    __device__ __forceinline__ void load(const uint8_t* p) {
        row(0, p);
        row(1, p + S::CB);
        row(2, p + 8 * S::CB);
        row(3, p + 9 * S::CB);
    }
    __device__ __forceinline__ void row(int i, const uint8_t* p) {
        if constexpr (NG == 2) {
            r[i][0] = *reinterpret_cast<const uint32_t*>(p);
            r[i][1] = *reinterpret_cast<const uint32_t*>(p + 32);
        } else if constexpr (S::VW == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            r[i][0] = x.x; r[i][1] = x.y; r[i][2] = x.z; r[i][3] = x.w;
        } else if constexpr (S::VW == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            r[i][0] = x.x; r[i][1] = x.y;
        } else {
            r[i][0] = *reinterpret_cast<const uint32_t*>(p);
        }
    }
    // A fragment word: element e of token pair pr (rows 2 pr, 2 pr + 1)
    __device__ __forceinline__ uint32_t frag(int e, int pr) const {
        const uint32_t *a = r[2 * pr], *b = r[2 * pr + 1];
        if constexpr (S::INT4) {
            const int word = e >> 3, sub = (e >> 2) & 1, nib = e & 3;
            const uint32_t x = __byte_perm(a[word], b[word], sub ? 0x7632u : 0x5410u);
            const uint32_t y = nib >= 2 ? x >> 8 : x;
            // c - 8, or 16 (c - 8): exact in fp16
            const uint32_t h = ((nib & 1) ? nib_odd(y) : nib_even(y)) | 0x64006400u;
            return sub16x2(h, (nib & 1) ? 0x64806480u : 0x64086408u);
        } else {
            const int word = e >> 2, sub = e & 3;
            const uint32_t x = __byte_perm(a[word], b[word], (sub >> 1) ? 0x7362u : 0x5140u);
            return e4m3x2((sub & 1) ? (x >> 16) : x);
        }
    }
};

// K scale / zero of tokens g, g + 8; V scale of the same tokens; V zero points
// of tokens 2c, 2c + 1 and 8 + 2c, 9 + 2c as fragment words.
// FINE: with what the rounding of z - 8 leaves.
template <int D, int QMODE, int NG, bool FINE>
struct Scales {
    __half2 ks[NG], vs[NG], kz[NG];  // low: token g, high: token g + 8
    uint32_t vz[NG][2];
    __device__ __forceinline__ void load(const uint8_t* p, int g, int c) {  // p: the stage's scales
        const __half* k = reinterpret_cast<const __half*>(p) + g * NG;
        const __half* v = k + BS * NG;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            ks[i] = __halves2half2(k[i], k[8 * NG + i]);
            vs[i] = __halves2half2(v[i], v[8 * NG + i]);
        }
        if constexpr (Shape<D, QMODE, NG>::INT4) {
            const __half* kzp = k + 2 * BS * NG;
            const __half* z = reinterpret_cast<const __half*>(p) + 3 * BS * NG + 2 * c * NG;
#pragma unroll
            for (int i = 0; i < NG; ++i) kz[i] = __halves2half2(kzp[i], kzp[8 * NG + i]);
            if constexpr (NG == 1) {
                vz[0][0] = *reinterpret_cast<const uint32_t*>(z);
                vz[0][1] = *reinterpret_cast<const uint32_t*>(z + 8);
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(z), y = *reinterpret_cast<const uint2*>(z + 16);
                vz[0][0] = __byte_perm(x.x, x.y, 0x5410u);
                vz[NG - 1][0] = __byte_perm(x.x, x.y, 0x7632u);
                vz[0][1] = __byte_perm(y.x, y.y, 0x5410u);
                vz[NG - 1][1] = __byte_perm(y.x, y.y, 0x7632u);
            }
            // z - 8, as V's codes are taken: lanes g = 0 (row 0 of the zero
            // points' MMA) hold it rounded, lanes g = 1 what the rounding left
            // (exact for |z| <= 8; nothing is left from 4 up), the others 0
#pragma unroll
            for (int i = 0; i < NG; ++i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t hi = sub16x2(vz[i][k], 0x48004800u);
                    const uint32_t lo = FINE ? sub16x2(vz[i][k], sub16x2(hi, 0xC800C800u)) : 0u;
                    vz[i][k] = g == 0 ? hi : FINE && g == 1 ? lo : 0u;
                }
            }
        }
    }
};

// A warp's state over its run: lane (g, c) holds rows 8 nt + 2c (x), 8 nt + 2c +
// 1 (y) of every n-tile.  nm: minus the reference maximum.  corr: the
// zero-point MMA's accumulator (rows 0, 1 and 8, 9 of its 16: column groups 0
// and 1; lanes g = 0, 1).
template <int MT, int NT>
struct State {
    float2 nm[NT], l[NT];
    float o[MT][NT][4];
    float corr[NT][4];
};

// Raises n-tile nt's reference maxima to cover the logits x (tokens g: 0, 1;
// tokens g + 8: 2, 3) and rescales what was accumulated against the old ones.
template <int MT, int NT>
__device__ __forceinline__ void raise_max(State<MT, NT>& w, int nt, const float (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float b = fmaxf(x[k], x[k + 2]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
        float& nm = k ? w.nm[nt].y : w.nm[nt].x;
        float& l = k ? w.l[nt].y : w.l[nt].x;
        const float mn = fmaxf(-nm, b);
        const float al = ex2(-nm - mn);
        nm = -mn;
        l *= al;
        w.corr[nt][k] *= al;
        w.corr[nt][k + 2] *= al;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            w.o[mt][nt][k] *= al;
            w.o[mt][nt][k + 2] *= al;
        }
    }
}

// Adds V's non-finite values v(t, column) of tokens [t0, t1) to the rows that
// see them; the MMA was given zeros in their place (0 x NaN would have reached
// the rows that do not).
template <int D, int NG, int NT, typename V>
__device__ __forceinline__ void add_non_finite(State<D / 16, NT>& w, const int (&pos)[NT][2], int t0, int t1, int g, V v) {
    for (int t = t0; t < t1; ++t) {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float x = v(t, pv_column<D, NG>(pv_e<D, NG>(mt, hf), g));
                if (fabsf(x) <= 3.4e38f) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (t <= pos[nt][0]) w.o[mt][nt][2 * hf] += x;
                    if (t <= pos[nt][1]) w.o[mt][nt][2 * hf + 1] += x;
                }
            }
        }
    }
}

template <typename T, int D, int QMODE, int NG, int NT>
__global__ void __launch_bounds__(kWarps * 32, ctas_per_sm(NT))
    mqq_balanced_kernel(const __grid_constant__ QuantCache a, int nwt_launch, float* ws_o, float* ws_ml) {
    using S = Shape<D, QMODE, NG>;
    constexpr int KW = S::KW, MT = S::MT, R = 8 * NT, QW = S::KSTEPS / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;");
    // per warp: the run's query fragments ([NT][QW][32] uint4) and the ring,
    // which takes the run's R x D partial outputs when the run is done
    constexpr int kMax = S::STAGE * kStages > 2 * S::STAGE16 ? S::STAGE * kStages : 2 * S::STAGE16;
    constexpr int kRing = kMax > R * D * 4 ? kMax : R * D * 4;
    static_assert(kStages == 4 && kRing % 16 == 0, "ring");
    __shared__ __align__(128) uint8_t rings[kWarps][kRing];
    __shared__ __align__(16) uint4 queries[kWarps][NT * QW * 32];
    __shared__ __align__(8) uint64_t bars[kWarps][kStages];
    uint8_t* ring = rings[warp];
    const uint32_t ring_addr = sh_addr(ring), bar0 = sh_addr(bars[warp]);
    uint4* sq = queries[warp] + lane;
    const uint32_t qs_addr = sh_addr(sq);
    if (lane < kStages) mbar_init(bar0 + 8 * lane, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_shared();
    __syncwarp();
    uint32_t par = 0;  // parity of each stage's next fill
    // waits for stage s; false (and the status bit) when its copies never land
    auto landed = [&](int s) {
        const bool ok = __all_sync(0xffffffffu, wait_bar(bar0 + 8 * s, (par >> s) & 1u));
        par ^= 1u << s;
        if (!ok && lane == 0) atomicOr(a.status, PKV_STATUS_COPY_TIMEOUT);
        return ok;
    };

    const int i = blockIdx.x * kWarps + warp;
    const int cap = a.max_blocks * BS;
    WarpSplit sp;
    bool bad = false;
    const bool any = sp.begin(a.ctx_lens, a.batch, cap, a.hkv, nwt_launch, kMinItems, i, bad);
    if (i == 0 && bad && lane == 0) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
    if (!any) return;
    while (sp.next()) {
        const int b = sp.b, kvh = sp.kvh, ctx = sp.ctx;
        const int q0 = a.q_start[b], L = a.q_start[b + 1] - q0;
        if (L <= 0) continue;
        const int rows = min(L, a.max_q_len) * a.G;
        if ((L > a.max_q_len || ctx < L) && lane == 0 && sp.lb0 == 0 && kvh == 0)
            atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
        const int first_pos = ctx - L;
        const T* qbase = static_cast<const T*>(a.q) + (static_cast<int64_t>(q0) * a.hq + kvh * a.G) * D;
        auto qrow = [&](int row) {
            const int tok = row / a.G;
            return qbase + (static_cast<int64_t>(tok) * a.hq + (row - tok * a.G)) * D;
        };

        // ---- query fragments in fp16, in the k order of the codes, and the
        // rows' sums per column group
        float qs[NT][NG][2];
        __syncwarp();  // the previous run's partial rows have been copied out
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + g;
            const bool valid = row < rows;
            const T* q = qrow(valid ? row : 0);
            float sum[NG];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) sum[gi] = 0.f;
#pragma unroll
            for (int k = 0; k < QW; ++k) {
                // INT4: word k covers 8 columns; FP8: 8 columns of load k / 2
                const int col = S::INT4 ? (k / S::KPG) * (D / NG) + (D / NG / 4) * c + 8 * (k % S::KPG)
                                        : 64 * (k / 2) + 16 * c + 8 * (k % 2);
                const uint4 raw = valid ? *reinterpret_cast<const uint4*>(q + col) : make_uint4(0, 0, 0, 0);
                const T* e = reinterpret_cast<const T*>(&raw);
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // fp16, saturating, as the MMA sees it
                    x[j] = __half2float(__float2half_rn(fminf(fmaxf(Half16<T>::to_float(e[j]), -65504.f), 65504.f)));
                    if (Half16<T>::to_float(e[j]) != Half16<T>::to_float(e[j])) x[j] = Half16<T>::to_float(e[j]);
                    sum[S::INT4 ? k / S::KPG : 0] += x[j];
                }
                uint4 f;
                if constexpr (S::INT4) {
                    // k-step 2k: nibbles {0, 4} and {1, 5}; 2k + 1: {2, 6}, {3, 7}; the
                    // odd nibbles enter 16 x larger
                    f.x = f16pair(x[0], x[4]);
                    f.y = f16pair(x[1] * 0.0625f, x[5] * 0.0625f);
                    f.z = f16pair(x[2], x[6]);
                    f.w = f16pair(x[3] * 0.0625f, x[7] * 0.0625f);
                } else {
                    f.x = f16pair(x[0], x[1]);
                    f.y = f16pair(x[2], x[3]);
                    f.z = f16pair(x[4], x[5]);
                    f.w = f16pair(x[6], x[7]);
                }
                sq[(nt * QW + k) * 32] = f;
            }
            if constexpr (S::INT4) {
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 1);
                    sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 2);
                    qs[nt][gi][0] = __shfl_sync(0xffffffffu, sum[gi], 8 * c);
                    qs[nt][gi][1] = __shfl_sync(0xffffffffu, sum[gi], 8 * c + 4);
                }
            }
        }
        __syncwarp();
        int pos[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = 8 * nt + 2 * c + k;
                const int p = row < rows ? first_pos + row / a.G : -1;
                pos[nt][k] = p < 0 ? -1 : p;
            }
        }
        State<MT, NT> w;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            w.nm[nt] = make_float2(-kNoMax, -kNoMax);
            w.l[nt] = make_float2(0.f, 0.f);
            w.corr[nt][0] = w.corr[nt][1] = w.corr[nt][2] = w.corr[nt][3] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) w.o[mt][nt][0] = w.o[mt][nt][1] = w.o[mt][nt][2] = w.o[mt][nt][3] = 0.f;
        }
        // window blocks start at win_lb; block 0's first n_sink tokens are sinks
        const int win_lb = a.window > 0 ? max(ctx - a.window, 0) / BS : 0x7fffffff;
        const int q_end = min(sp.lb1, win_lb);
        const int sinks = win_lb > 0 ? a.n_sink : 0;
        // blocks below full_lb are seen whole by every row (rows that do not
        // exist aside: their outputs go nowhere)
        const int full_lb = max(first_pos + 1, 0) / BS;

        // ---- quantised blocks.  Lane j copies run j of a block (see Shape):
        // from src + phys * step into the stage at dst.
        const bool scales = lane >= 2;
        const uint8_t* src = lane == 0   ? a.codes[0]
                             : lane == 1 ? a.codes[1]
                                         : reinterpret_cast<const uint8_t*>(lane < 4 ? a.scale[lane & 1] : a.zero[lane & 1]);
        const uint32_t bytes = scales ? S::SCALES : S::CODES, step = bytes * a.hkv;
        const uint32_t dst = ring_addr + (scales ? 2 * S::CODES + (lane - 2) * S::SCALES : lane * S::CODES);
        src += static_cast<uint32_t>(kvh) * bytes;
        const int32_t* trow = a.tables + static_cast<int64_t>(b) * a.max_blocks;
        const int nq = q_end - sp.lb0;
        int tab = -1;
        uint32_t filled = 0;  // stages with a block to attend
        auto issue = [&](int k) {  // block lb0 + k into stage k % kStages
            if ((k & 31) == 0) {
                tab = k + lane < nq ? trow[sp.lb0 + k + lane] : -1;
                if (__any_sync(0xffffffffu, k + lane < nq && static_cast<unsigned>(tab) >= static_cast<unsigned>(a.num_blocks)) &&
                    lane == 0)
                    atomicOr(a.status, PKV_STATUS_BAD_BLOCK);
            }
            const int phys = __shfl_sync(0xffffffffu, tab, k & 31);
            const int s = k % kStages;
            filled &= ~(1u << s);
            if (static_cast<unsigned>(phys) < static_cast<unsigned>(a.num_blocks)) {
                filled |= 1u << s;
                if (lane == 0) mbar_arrive_expect_tx(bar0 + 8 * s, S::STAGE);
                __syncwarp();
                if (lane < S::COPIES)
                    bulk_load(dst + s * S::STAGE, src + static_cast<uint64_t>(static_cast<uint32_t>(phys)) * step, bytes,
                              bar0 + 8 * s);
            }
        };
        for (int k = 0; k < min(nq, kStages); ++k) issue(k);
        for (int k = 0; k < nq; ++k) {
            const int lb = sp.lb0 + k;
            const uint8_t* stage = ring + (k % kStages) * S::STAGE;
            if (!((filled >> (k % kStages)) & 1u)) {  // a bad table entry: nothing to attend
                if (k + kStages < nq) issue(k + kStages);
                continue;
            }
            if (!landed(k % kStages)) {  // the copies still in flight land (bounded), then the warp stops
                for (int j = k + 1; j < min(nq, k + kStages); ++j)
                    if ((filled >> (j % kStages)) & 1u) landed(j % kStages);
                return;
            }
            KCodes<D, QMODE, NG> kc;
            kc.load(stage + g * S::CB + (!S::INT4 ? 16 * c : NG == 2 ? 8 * c : (KW == 4 ? 16 * c : 8 * c)));
            Scales<D, QMODE, NG, kFine<T>> sc;
            sc.load(stage + 2 * S::CODES, g, c);
            // ---- S^T = C Q^T over the code values, per column group
            float s[NG][NT][4];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[gi][nt][0] = s[gi][nt][1] = s[gi][nt][2] = s[gi][nt][3] = 0.f;
#pragma unroll
            for (int t = 0; t < QW; ++t) {
                uint32_t f[8];
                if constexpr (S::INT4) {
                    const uint32_t u0 = kc.r0[t] >> 8, u1 = kc.r1[t] >> 8;
                    f[0] = nib_even(kc.r0[t]); f[1] = nib_even(kc.r1[t]); f[2] = nib_odd(kc.r0[t]); f[3] = nib_odd(kc.r1[t]);
                    f[4] = nib_even(u0); f[5] = nib_even(u1); f[6] = nib_odd(u0); f[7] = nib_odd(u1);
                } else {
                    const int j = 2 * t;  // k-steps 2t, 2t + 1 use words 2t, 2t + 1
                    f[0] = e4m3x2(kc.r0[j]); f[1] = e4m3x2(kc.r1[j]); f[2] = e4m3x2(kc.r0[j] >> 16); f[3] = e4m3x2(kc.r1[j] >> 16);
                    f[4] = e4m3x2(kc.r0[j + 1]); f[5] = e4m3x2(kc.r1[j + 1]);
                    f[6] = e4m3x2(kc.r0[j + 1] >> 16); f[7] = e4m3x2(kc.r1[j + 1] >> 16);
                }
                const int gi = S::INT4 ? t / S::KPG : 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 q = lds128(qs_addr + (nt * QW + t) * 512);
                    mma_f16(s[gi][nt], f[0], f[1], f[2], f[3], q.x, q.y);
                    mma_f16(s[gi][nt], f[4], f[5], f[6], f[7], q.z, q.w);
                }
            }
            // ---- logits (base 2) less the reference maxima; k0, z0: token g's
            // scale and -scale * zero point, k1, z1: token g + 8's
            float k0[NG], k1[NG], z0[NG], z1[NG], vs0[NG], vs1[NG];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                k0[gi] = __low2float(sc.ks[gi]) * a.scale_log2;
                k1[gi] = __high2float(sc.ks[gi]) * a.scale_log2;
                if constexpr (S::INT4) {
                    z0[gi] = -k0[gi] * __low2float(sc.kz[gi]);
                    z1[gi] = -k1[gi] * __high2float(sc.kz[gi]);
                    k0[gi] *= kTwo24;
                    k1[gi] *= kTwo24;
                }
                vs0[gi] = __low2float(sc.vs[gi]);
                vs1[gi] = __high2float(sc.vs[gi]);
            }
            // from: what is added to the scaled products
            auto logits = [&](int nt, float2 from, float2& e0, float2& e1) {
                e0 = e1 = from;
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    if constexpr (S::INT4) {
                        const float2 q = make_float2(qs[nt][gi][0], qs[nt][gi][1]);
                        e0 = fma2(make_float2(z0[gi], z0[gi]), q, e0);
                        e1 = fma2(make_float2(z1[gi], z1[gi]), q, e1);
                    }
                    e0 = fma2(make_float2(s[gi][nt][0], s[gi][nt][1]), make_float2(k0[gi], k0[gi]), e0);
                    e1 = fma2(make_float2(s[gi][nt][2], s[gi][nt][3]), make_float2(k1[gi], k1[gi]), e1);
                }
            };
            float2 d0[NT], d1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) logits(nt, w.nm[nt], d0[nt], d1[nt]);
            VCodes<D, QMODE, NG> vc;
            vc.load(stage + S::CODES + 2 * c * S::CB + (S::INT4 ? (NG == 2 ? 4 * g : D / 16 * g) : D / 8 * g));
            const int t0 = lb * BS;
            const bool masked = lb >= full_lb || (lb == 0 && sinks > 0);
            bool fix_nan = false;
            if (masked) {
                const bool in0 = t0 + g < ctx && t0 + g >= sinks, in1 = t0 + g + 8 < ctx && t0 + g + 8 >= sinks;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (!in0 || t0 + g > pos[nt][0]) d0[nt].x = neg_inf();
                    if (!in0 || t0 + g > pos[nt][1]) d0[nt].y = neg_inf();
                    if (!in1 || t0 + g + 8 > pos[nt][0]) d1[nt].x = neg_inf();
                    if (!in1 || t0 + g + 8 > pos[nt][1]) d1[nt].y = neg_inf();
                }
                // slots that hold no token, and sinks: any bits; their weight is
                // 0, their scale and zero point are taken out
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    if (!in0) vs0[gi] = 0.f;
                    if (!in1) vs1[gi] = 0.f;
                    if constexpr (S::INT4) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int t = t0 + 2 * c + 8 * hf;
                            if (t >= ctx || t < sinks) sc.vz[gi][hf] &= 0xffff0000u;
                            if (t + 1 >= ctx || t + 1 < sinks) sc.vz[gi][hf] &= 0x0000ffffu;
                        }
                    }
                }
                if constexpr (!S::INT4) {
                    // codes of slots without a token, and NaN codes
                    bool odd = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = t0 + 2 * c + (j & 1) + 8 * (j >> 1);
#pragma unroll
                        for (int v = 0; v < S::VW; ++v) {
                            if (t >= ctx || t < sinks) vc.r[j][v] = 0;
                            const uint32_t nan = __vcmpeq4(vc.r[j][v] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            odd |= nan != 0;
                            vc.r[j][v] &= ~nan;
                        }
                    }
                    fix_nan = __any_sync(0xffffffffu, odd);
                }
            }

            // ---- online softmax: the reference maxima move only when a logit
            // exceeds one by more than kSlack, or a V scale is large
            float top = neg_inf(), vtop = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) top = max3f(top, fmaxf(d0[nt].x, d0[nt].y), fmaxf(d1[nt].x, d1[nt].y));
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) vtop = max3f(vtop, vs0[gi], vs1[gi]);
            if (__any_sync(0xffffffffu, top > kSlack || vtop > kLazyMaxScale)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float2 x0, x1;
                    logits(nt, make_float2(0.f, 0.f), x0, x1);
                    const float x[4] = {d0[nt].x == neg_inf() ? neg_inf() : x0.x, d0[nt].y == neg_inf() ? neg_inf() : x0.y,
                                        d1[nt].x == neg_inf() ? neg_inf() : x1.x, d1[nt].y == neg_inf() ? neg_inf() : x1.y};
                    raise_max<MT, NT>(w, nt, x);
                    d0[nt] = add2(make_float2(x[0], x[1]), w.nm[nt]);
                    d1[nt] = add2(make_float2(x[2], x[3]), w.nm[nt]);
                }
            }
            uint32_t b0[NG][NT], b1[NG][NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 p0 = make_float2(ex2(d0[nt].x), ex2(d0[nt].y)), p1 = make_float2(ex2(d1[nt].x), ex2(d1[nt].y));
                w.l[nt] = add2(w.l[nt], add2(p0, p1));
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    const float2 w0 = mul2(p0, make_float2(vs0[gi], vs0[gi])), w1 = mul2(p1, make_float2(vs1[gi], vs1[gi]));
                    b0[gi][nt] = movmatrix_trans(f16pair(w0.x, w0.y));
                    b1[gi][nt] = movmatrix_trans(f16pair(w1.x, w1.y));
                }
            }
            // ---- sum_t W_t (z_t - 8): zero points as rows 0, 1 (group 0) and 8, 9
            // (group 1)
            if constexpr (S::INT4) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(w.corr[nt], sc.vz[0][0], 0u, sc.vz[0][1], 0u, b0[0][nt], b1[0][nt]);
                    if constexpr (NG == 2)
                        mma_f16(w.corr[nt], 0u, sc.vz[NG - 1][0], 0u, sc.vz[NG - 1][1], b0[NG - 1][nt],
                                b1[NG - 1][nt]);
                }
            }
            // ---- O^T += C_v^T W^T
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int el = pv_e<D, NG>(mt, 0), eh = pv_e<D, NG>(mt, 1);
                const uint32_t f0 = vc.frag(el, 0), f1 = vc.frag(eh, 0), f2 = vc.frag(el, 1), f3 = vc.frag(eh, 1);
                const int gi = S::INT4 ? (el >> 3) / S::VPG : 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(w.o[mt][nt], f0, f1, f2, f3, b0[gi][nt], b1[gi][nt]);
            }
            if constexpr (!S::INT4) {
                if (fix_nan) {
                    const uint8_t* codes = stage + S::CODES;
                    add_non_finite<D, NG, NT>(w, pos, max(t0, sinks), min(t0 + BS, ctx), g, [&](int t, int col) {
                        return (codes[(t - t0) * S::CB + col] & 0x7f) == 0x7f ? __int_as_float(0x7fc00000) : 0.f;
                    });
                }
            }
            __syncwarp();  // the stage is read
            if (k + kStages < nq) issue(k + kStages);
        }

        // ---- INT4: the odd nibbles' 16 and the zero points come off
        if constexpr (S::INT4) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float cr[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cr[j] = __shfl_sync(0xffffffffu, w.corr[nt][j], c);
                    if constexpr (kFine<T>) cr[j] += __shfl_sync(0xffffffffu, w.corr[nt][j], 4 + c);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int el = pv_e<D, NG>(mt, 0);
                    const int gi = (el >> 3) / S::VPG;
                    const float u = (el & 1) ? 0.0625f : 1.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) w.o[mt][nt][j] = fmaf(w.o[mt][nt][j], u, -cr[2 * gi + (j & 1)]);
                }
            }
        }

        // ---- 16-bit blocks: the sinks (their rows stand in for block 0's first
        // n_sink tokens), then the window, through the ring two at a time: lane
        // r < 16 copies K row r, lane 16 + r V row r.
        constexpr int kRow16 = D * 2;
        const int win0 = max(sp.lb0, win_lb), n_win = max(sp.lb1 - win0, 0);
        const int sink_rows = sp.lb0 == 0 ? min(sinks, ctx) : 0;
        const int n16 = (sink_rows > 0 ? 1 : 0) + n_win;
        auto rows16 = [&](int k, int& t0, int& n) {  // the k-th 16-bit block's first token and rows
            const int lb = win0 + k - (sink_rows > 0 ? 1 : 0);
            t0 = sink_rows > 0 && k == 0 ? 0 : lb * BS;
            n = sink_rows > 0 && k == 0 ? sink_rows : min(BS, ctx - lb * BS);
        };
        auto issue16 = [&](int k) {
            int t0, n;
            rows16(k, t0, n);
            const int x = lane >> 4, r = lane & 15, s = k & 1;
            const T* p = sink_rows > 0 && k == 0
                             ? static_cast<const T*>(a.sink[x]) +
                                   ((static_cast<int64_t>(b) * a.n_sink + r) * a.hkv + kvh) * D
                             : static_cast<const T*>(a.win[x]) +
                                   (((static_cast<int64_t>(b) * a.ring + (t0 / BS) % a.ring) * a.hkv + kvh) * BS + r) * D;
            if (lane == 0) mbar_arrive_expect_tx(bar0 + 8 * s, 2 * n * kRow16);
            __syncwarp();
            if (r < n) bulk_load(ring_addr + s * S::STAGE16 + (x * BS + r) * kRow16, p, kRow16, bar0 + 8 * s);
        };
        auto attend16 = [&](const T* kr, const T* vr, int t0, int n) {
            using H = Half16<T>;
            constexpr int KC = D / 32, VC = D / 64;
            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const uint4 k0 = *reinterpret_cast<const uint4*>(kr + g * D + 32 * k + 8 * c);
                const uint4 k1 = *reinterpret_cast<const uint4*>(kr + (g + 8) * D + 32 * k + 8 * c);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = 8 * nt + g;
                    const uint4 q = row < rows ? *reinterpret_cast<const uint4*>(qrow(row) + 32 * k + 8 * c)
                                               : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        H::mma(x[nt], word(k0, 2 * e), word(k1, 2 * e), word(k0, 2 * e + 1), word(k1, 2 * e + 1),
                               word(q, 2 * e), word(q, 2 * e + 1));
                }
            }
            bool up = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = g + 8 * (j >> 1);  // rows past n: whatever the ring held
                    x[nt][j] = r < n && t0 + r <= pos[nt][j & 1] ? x[nt][j] * a.scale_log2 : neg_inf();
                    up |= x[nt][j] + (j & 1 ? w.nm[nt].y : w.nm[nt].x) > kSlack;
                }
            }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) raise_max<MT, NT>(w, nt, x[nt]);
            }
            uint32_t b0[NT], b1[NT], e0[NT], e1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = ex2(x[nt][0] + w.nm[nt].x), p1 = ex2(x[nt][1] + w.nm[nt].y);
                const float p2 = ex2(x[nt][2] + w.nm[nt].x), p3 = ex2(x[nt][3] + w.nm[nt].y);
                w.l[nt].x += p0 + p2;
                w.l[nt].y += p1 + p3;
                const uint32_t h01 = H::pack(p0, p1), h23 = H::pack(p2, p3);
                b0[nt] = movmatrix_trans(h01);
                b1[nt] = movmatrix_trans(h23);
                if constexpr (kSplitP<T>) {  // bf16 P goes in as value and rounding residual
                    e0[nt] = movmatrix_trans(H::pack(p0 - __uint_as_float(h01 << 16), p1 - __uint_as_float(h01 & 0xffff0000u)));
                    e1[nt] = movmatrix_trans(H::pack(p2 - __uint_as_float(h23 << 16), p3 - __uint_as_float(h23 & 0xffff0000u)));
                }
            }
            uint4 v[4][VC];
            bool odd = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 2 * c + (j & 1) + 8 * (j >> 1);
#pragma unroll
                for (int y = 0; y < VC; ++y) {
                    v[j][y] = make_uint4(0, 0, 0, 0);
                    if (r < n)
                        v[j][y] = *reinterpret_cast<const uint4*>(vr + r * D + (NG == 2 ? 64 * y + 8 * g : g * (D / 8) + 8 * y));
                    // non-finite values: out of the product (see add_non_finite)
                    constexpr uint32_t kExp = kSplitP<T> ? 0x7F80u : 0x7C00u;
                    uint32_t* wd = reinterpret_cast<uint32_t*>(&v[j][y]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        if ((wd[z] & kExp) == kExp) { wd[z] &= 0xffff0000u; odd = true; }
                        if (((wd[z] >> 16) & kExp) == kExp) { wd[z] &= 0x0000ffffu; odd = true; }
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t f[4];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int e = pv_e<D, NG>(mt, hf), ch = e >> 3, wd = (e & 7) >> 1;
                    const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
                    f[hf] = __byte_perm(word(v[0][ch], wd), word(v[1][ch], wd), sel);
                    f[hf + 2] = __byte_perm(word(v[2][ch], wd), word(v[3][ch], wd), sel);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    H::mma(w.o[mt][nt], f[0], f[1], f[2], f[3], b0[nt], b1[nt]);
                    if constexpr (kSplitP<T>) H::mma(w.o[mt][nt], f[0], f[1], f[2], f[3], e0[nt], e1[nt]);
                }
            }
            if (__any_sync(0xffffffffu, odd))
                add_non_finite<D, NG, NT>(w, pos, t0, t0 + n, g,
                                          [&](int t, int col) { return Half16<T>::to_float(vr[(t - t0) * D + col]); });
        };
        __syncwarp();  // the quantised stages are read
        for (int k = 0; k < min(n16, 2); ++k) issue16(k);
        for (int k = 0; k < n16; ++k) {
            if (!landed(k & 1)) {
                if (k + 1 < n16) landed((k + 1) & 1);
                return;
            }
            int t0, n;
            rows16(k, t0, n);
            const T* kr = reinterpret_cast<const T*>(ring + (k & 1) * S::STAGE16);
            attend16(kr, kr + BS * D, t0, n);
            __syncwarp();  // the stage is read
            if (k + 2 < n16) issue16(k + 2);
        }

        // ---- the run's partial rows: l totalled over the token lanes, o
        // staged through the ring so rows go out in 16-byte stores
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                w.l[nt].x += __shfl_xor_sync(0xffffffffu, w.l[nt].x, off);
                w.l[nt].y += __shfl_xor_sync(0xffffffffu, w.l[nt].y, off);
            }
        }
        __syncwarp();  // the ring is no longer read
        float* so = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = pv_column<D, NG>(pv_e<D, NG>(mt, j >> 1), g);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) so[(8 * nt + 2 * c + (j & 1)) * D + d] = w.o[mt][nt][j];
            }
        }
        __syncwarp();
        const int64_t slot = i + static_cast<int64_t>(b) * a.hkv + kvh;
        float4* po = reinterpret_cast<float4*>(ws_o + slot * R * D);
        const float4* s4 = reinterpret_cast<const float4*>(so);
        for (int y = lane; y < rows * D / 4; y += 32) po[y] = s4[y];
        fence_async_shared();  // before the next run's copies into the ring
        if (g == 0) {
            float* pml = ws_ml + slot * R * 2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = 8 * nt + 2 * c + k;
                    if (row < rows)
                        *reinterpret_cast<float2*>(pml + 2 * row) =
                            k ? make_float2(-w.nm[nt].y, w.l[nt].y) : make_float2(-w.nm[nt].x, w.l[nt].x);
                }
            }
        }
    }
}

// Merge of the partial rows: one CTA per (8 rows, KV head, sequence), a warp
// per row, lanes over the head dim (and, for the weights, over the partials).
// Where the run's partials sit follows from the context lengths alone, so it
// is worked out before the wait on the split grid.
constexpr int kMergeWarps = 8;

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kMergeWarps * 32)
    mqq_merge_kernel(const __grid_constant__ QuantCache a, int nwt_launch, const float* __restrict__ ws_o,
                     const float* __restrict__ ws_ml) {
    constexpr int R = 8 * NT, E = D / 32;
    const int kvh = blockIdx.x / NT, r = blockIdx.x % NT * 8 + (threadIdx.x >> 5), b = blockIdx.y;
    const int lane = threadIdx.x & 31, cap = a.max_blocks * BS;
    int before = 0, total = 0;
    for (int j = lane; j < a.batch; j += 32) {
        const int nbj = blocks_of(a.ctx_lens[j], cap);
        total += nbj;
        before += j < b ? nbj : 0;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    const int q0 = a.q_start[b], L = a.q_start[b + 1] - q0;
    const int rows = L > 0 ? min(L, a.max_q_len) * a.G : 0;
    const int nb = blocks_of(a.ctx_lens[b], cap);
    const int W = total * a.hkv;
    const int nwt = max(min(W / kMinItems, nwt_launch), 1);
    int64_t slot0 = 0;
    int np = 0;
    if (nb > 0) {
        const int at = before * a.hkv + kvh * nb;
        const int64_t i0 = first_warp(at, W, nwt), i1 = first_warp(at + nb - 1, W, nwt);
        slot0 = i0 + static_cast<int64_t>(b) * a.hkv + kvh;
        np = static_cast<int>(i1 - i0 + 1);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (r >= rows) return;
    const float2* ml = reinterpret_cast<const float2*>(ws_ml) + slot0 * R + r;  // partial p: ml[p R]
    const float* po = ws_o + (slot0 * R + r) * D + lane * E;
    float M = kNoMax;
    for (int p = lane; p < np; p += 32) M = fmaxf(M, __ldcg(ml + static_cast<int64_t>(p) * R).x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float Ls = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int p0 = 0; p0 < np; p0 += 32) {
        float wt = 0.f;
        if (p0 + lane < np) {
            const float2 v = __ldcg(ml + static_cast<int64_t>(p0 + lane) * R);
            wt = ex2(v.x - M);
            Ls += wt * v.y;
        }
        const int n = min(32, np - p0);
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
            const float f = __shfl_sync(0xffffffffu, wt, j);
            const float* p = po + static_cast<int64_t>(p0 + j) * R * D;
            if constexpr (E == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
                o[0] += f * v.x;
                o[1] += f * v.y;
                o[2] += f * v.z;
                o[3] += f * v.w;
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
                o[0] += f * v.x;
                o[1] += f * v.y;
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, off);
    const float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);  // NaN stays
    const int tok = r / a.G;
    T* dst = static_cast<T*>(a.out) +
             ((static_cast<int64_t>(q0) + tok) * a.hq + kvh * a.G + (r - tok * a.G)) * D + lane * E;
    uint32_t v[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) v[e] = Ls == 0.f ? 0u : Half16<T>::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
    if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(v[0], v[1]);
    else *reinterpret_cast<uint32_t*>(dst) = v[0];
}

// n-tiles of the balanced split for rows per (sequence, KV head), 0: too many
// rows (or too many items to index).
int small_nt(int64_t batch, int64_t hkv, int64_t max_blocks, int64_t rows) {
    if (rows > 8 * kMaxNT || batch * hkv * max_blocks >= (1LL << 30)) return 0;
    return rows <= 0 ? 1 : static_cast<int>((rows + 7) / 8);
}

// Warps the split launches: all resident at once, kMinItems items each.
int small_warps(int64_t items, int nt) {
    const int64_t full = static_cast<int64_t>(num_sms()) * kWarps * ctas_per_sm(nt);
    const int64_t n = items / kMinItems;
    return static_cast<int>(n < 1 ? 1 : (n > full ? full : n));
}

size_t small_bytes(int64_t batch, int64_t hkv, int D, int nt, int nwt) {
    return static_cast<size_t>(nwt + batch * hkv) * 8 * nt * (D + 2) * sizeof(float);
}

template <typename T, int D, int QMODE, int NG, int NT>
int run_small(const QuantCache& a, int nwt, float* ws_o, float* ws_ml, cudaStream_t st) {
    mqq_balanced_kernel<T, D, QMODE, NG, NT><<<(nwt + kWarps - 1) / kWarps, kWarps * 32, 0, st>>>(a, nwt, ws_o, ws_ml);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.hkv * NT, a.batch);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mqq_merge_kernel<T, D, NT>, a, nwt, static_cast<const float*>(ws_o),
                              static_cast<const float*>(ws_ml)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

template <typename T, int D, int QMODE, int NG>
int run_small_nt(const QuantCache& a, int nt, int nwt, float* ws_o, float* ws_ml, cudaStream_t st) {
    if (nt == 1) return run_small<T, D, QMODE, NG, 1>(a, nwt, ws_o, ws_ml, st);
    if (nt == 2) return run_small<T, D, QMODE, NG, 2>(a, nwt, ws_o, ws_ml, st);
    return run_small<T, D, QMODE, NG, 3>(a, nwt, ws_o, ws_ml, st);
}

template <typename T>
int run_small_t(const QuantCache& a, int D, int nt, int nwt, float* ws_o, float* ws_ml, cudaStream_t st) {
    if (a.int4) {
        if (D == 64) return run_small_nt<T, 64, PKV_QMODE_INT4_ASYM, 1>(a, nt, nwt, ws_o, ws_ml, st);
        if (a.groups == 2) return run_small_nt<T, 128, PKV_QMODE_INT4_ASYM, 2>(a, nt, nwt, ws_o, ws_ml, st);
        return run_small_nt<T, 128, PKV_QMODE_INT4_ASYM, 1>(a, nt, nwt, ws_o, ws_ml, st);
    }
    if (D == 64) return run_small_nt<T, 64, PKV_QMODE_FP8_E4M3, 1>(a, nt, nwt, ws_o, ws_ml, st);
    return run_small_nt<T, 128, PKV_QMODE_FP8_E4M3, 1>(a, nt, nwt, ws_o, ws_ml, st);
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
    const int64_t rows = static_cast<int64_t>(max_q_len) * (num_q_heads / num_kv_heads);
    const int nt = pkv::small_nt(batch, num_kv_heads, max_blocks, rows);
    if (batch == 0 || max_q_len == 0) {
        *out = 0;
    } else if (nt > 0) {
        const int nwt = pkv::small_warps(static_cast<int64_t>(batch) * num_kv_heads * max_blocks, nt);
        *out = pkv::small_bytes(batch, num_kv_heads, head_dim, nt, nwt);
    } else {
        *out = pkv::slice_quant_workspace(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, max_q_len);
    }
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
    size_t need = 0;
    const int rc = pkv_multi_query_quant_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_blocks,
                                                         block_size, max_q_len, &need);
    if (rc != PKV_OK) return rc;
    if (need > 0 && (!workspace || workspace_bytes < need)) return PKV_ERR_WORKSPACE;
    if (need > 0 && !pkv::aligned16(workspace)) return PKV_ERR_MISALIGNED;
    pkv::QuantCache a;
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
    a.groups = int4 ? head_dim / group_size : 1;
    a.int4 = int4;
    a.scale_log2 = scale * pkv::kLog2e;
    a.out = out;
    a.status = st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == PKV_DTYPE_BF16;
    const int nt = pkv::small_nt(batch, num_kv_heads, max_blocks, static_cast<int64_t>(max_q_len) * a.G);
    if (nt == 0) return pkv::launch_slice_quant(a, head_dim, bf16, static_cast<float*>(workspace), cs);
    const int nwt = pkv::small_warps(static_cast<int64_t>(batch) * num_kv_heads * max_blocks, nt);
    float* ws_o = static_cast<float*>(workspace);
    float* ws_ml = ws_o + static_cast<size_t>(nwt + static_cast<int64_t>(batch) * num_kv_heads) * 8 * nt * head_dim;
    return bf16 ? pkv::run_small_t<__nv_bfloat16>(a, head_dim, nt, nwt, ws_o, ws_ml, cs)
                : pkv::run_small_t<__half>(a, head_dim, nt, nwt, ws_o, ws_ml, cs);
}
