// Causal attention of 256 query rows over tiles of 128 keys on the 5th-
// generation tensor cores: the parts shared by prompt.cu (K/V rows copied by
// TMA) and slice_quant.cu (quantised blocks unpacked into shared memory).
//
// A row is one (query token, query head) pair of one (sequence, KV head): row
// x is token x / G, head x % G, so a group's heads share every K/V tile.  A
// CTA's 256 rows are two MMA tiles of 128 that take turns: while the softmax
// of one runs, the tensor cores work for the other.
// * K and V tiles (128 keys x D, 16-bit, 128-byte swizzle) come through a ring
//   of kStages shared-memory slots, in the order K0 V0 K1 V1 ..
// * S = Q K^T (M 128, N 128) goes to TMEM; thread r of a tile's softmax
//   warpgroup owns row r whole: no exchange between threads (two threads a row
//   halved the chain but not the time: the special-function unit, at 4 cycles
//   per warp, and the exchange took it back).  Online softmax in base 2, the
//   reference maximum raised only by more than kSlack (O is then rescaled in
//   TMEM; S done implies the previous O += P V done, both being issued by one
//   thread in order).
// * P, rounded to the 16-bit type, overwrites S in TMEM and is the A operand of
//   O += P V; V is the MN-major B operand.  The first kFirst keys of P are
//   handed over while the rest is computed.
// * One warp issues every MMA: O0 += P0 V(j), S0(j + 1), O1 += P1 V(j), S1(j +
//   1), so each warpgroup has the other's two products (2 x 512 cycles at D =
//   128) for its softmax.
// Every wait is bounded in time: one that runs out sets
// PKV_STATUS_COPY_TIMEOUT and the stop flag, every role leaves its loop, waits
// (bounded) for its own copies and MMAs, and the CTA frees its TMEM.
#pragma once

#include <atomic>

#include "tc5.cuh"

namespace pkv {
namespace tcattn {

using namespace tc5;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // log2 units a score may exceed the reference maximum by
constexpr int kRows = 128;     // query rows per MMA tile
constexpr int kCtaRows = 256;  // two tiles
constexpr int kKeys = 128;     // keys per tile
constexpr int kFirst = 64;     // keys of P handed to the MMAs before the rest is computed
constexpr int kTmemCols = 512;  // S0, S1, O0, O1: 128 columns each

template <int D>
struct Layout {
    static constexpr int kTile = kRows * D * 2;  // bytes of a 128 x D 16-bit tile
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = 2 * kTile;
    static constexpr int kOffBar = kOffRing + kStages * kTile;
    // mbarriers: ring slot filled / read, S done (per tile), P written (first
    // keys of tile 0, 1, then the rest), O done, everything issued done
    static constexpr int kFull = 0, kFree = kStages, kS = 2 * kStages, kP = kS + 2, kO = kP + 4, kDrain = kO + 2;
    static constexpr int kBars = kDrain + 1;
    static constexpr int kOffVars = kOffBar + 8 * kBars;
    static constexpr int kBytes = kOffVars + 16;
};
static_assert(Layout<128>::kBytes <= 232448 && Layout<64>::kBytes <= 232448, "shared memory");

// A CTA's shared memory.
template <int D>
struct Smem {
    using Y = Layout<D>;
    uint8_t* p;
    uint32_t base;
    __device__ __forceinline__ explicit Smem(uint8_t* raw) : p(raw), base(sh_addr(raw)) {}  // raw: 1 KiB-aligned
    __device__ __forceinline__ uint32_t bar(int i) const { return base + Y::kOffBar + 8 * i; }
    __device__ __forceinline__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(p + Y::kOffVars); }
    // raised when a wait ran out
    __device__ __forceinline__ volatile int* stop() const { return reinterpret_cast<int*>(p + Y::kOffVars + 4); }
    // raised when a non-finite V value was taken out of a masked tile
    __device__ __forceinline__ volatile int* odd() const { return reinterpret_cast<int*>(p + Y::kOffVars + 8); }
    __device__ __forceinline__ bool stopped() const { return *stop() != 0; }
    __device__ __forceinline__ void give_up(int* status) const {
        atomicOr(status, PKV_STATUS_COPY_TIMEOUT);
        *stop() = 1;
    }
    // ring item 2 jj is K of the jj-th tile, 2 jj + 1 its V
    static __device__ __forceinline__ int slot(int it) { return it % Y::kStages; }
    static __device__ __forceinline__ uint32_t phase(int it) { return static_cast<uint32_t>(it / Y::kStages) & 1u; }
    __device__ __forceinline__ uint8_t* ring(int it) const { return p + Y::kOffRing + slot(it) * Y::kTile; }
    // by one thread, before any other uses the barriers; full: arrivals that
    // fill a ring slot
    __device__ __forceinline__ void init(int full) const {
        for (int i = 0; i < Y::kBars; ++i)
            mbar_init(bar(i), i < Y::kFree ? full : (i >= Y::kP && i < Y::kO ? 4 : 1));
        *stop() = 0;
        *odd() = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
};

// What a CTA computes: rows row0 .. row0 + 255 of a sequence's `rows`, token x
// / G at position first_pos + x / G, over key tiles [js, js + n), row tile i
// over the first cnt[i] of them.
struct Work {
    int row0, rows, G, first_pos;
    int js, n, cnt[2];
    __device__ __forceinline__ int count(int tile) const { return tile ? cnt[1] : cnt[0]; }
    // the share of split `split` of `splits` of the key tiles
    __device__ __forceinline__ void set_tiles(int split, int splits) {
        int total = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r1 = min(row0 + (i + 1) * kRows, rows);
            const int last = first_pos + (r1 - 1) / G;
            cnt[i] = r1 > row0 + i * kRows && last >= 0 ? last / kKeys + 1 : 0;
            total = max(total, cnt[i]);
        }
        js = static_cast<int>(static_cast<int64_t>(total) * split / splits);
        const int je = static_cast<int>(static_cast<int64_t>(total) * (split + 1) / splits);
#pragma unroll
        for (int i = 0; i < 2; ++i) cnt[i] = max(min(cnt[i], je) - js, 0);
        n = max(cnt[0], cnt[1]);
    }
    __device__ __forceinline__ int first_seen() const { return first_pos + row0 / G; }  // the first row's position
    // whether a tile holds keys that some row must not see
    __device__ __forceinline__ bool masked(int jj) const { return (js + jj) * kKeys + kKeys - 1 > first_seen(); }
    // the first key of the first masked tile of this split
    __device__ __forceinline__ int masked_from() const { return max(max(first_seen() + 1, 0) / kKeys, js) * kKeys; }
};

// Byte offset of (row, 16-byte chunk ch) in a swizzled tile of 128-byte rows
// (64 columns per half, halves kRows x 128 bytes apart).
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
    return (ch >> 3) * (kRows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// The MMA warp, whole: one elected lane issues, so what the MMAs take is
// warp-uniform (base descriptors plus constants) and an MMA of K 16 costs its
// 64 cycles; issued from a lane of a divergent branch it cost ~110 (8,192
// tokens: 490 instead of 380 us).
template <typename T, int D>
__device__ __forceinline__ void mma_warp(const Smem<D>& sm, uint32_t tmem, const Work& w, int* status) {
    using Y = Layout<D>;
    if (w.n == 0) return;
    constexpr uint32_t id_s = instr_desc<T>(kKeys, false), id_o = instr_desc<T>(D, true);
    constexpr uint32_t kTile16 = Y::kTile >> 4, kHalf16 = (kRows * 128) >> 4;  // descriptor units
    const bool el = elect();
    const uint64_t dq = smem_desc(sm.base + Y::kOffQ, 16384, 1024), dr = smem_desc(sm.base + Y::kOffRing, 16384, 1024);
    auto issue_s = [&](int i, int s) {
        const uint64_t qa = dq + i * kTile16, kb = dr + s * kTile16;
        if (el) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
                mma_ss(tmem + i * kKeys, qa + off, kb + off, id_s, kk > 0);
            }
            mma_commit(sm.bar(Y::kS + i));
        }
    };
    // keys 16 k0 .. 16 k1 - 1
    auto issue_o = [&](int i, int s, int k0, int k1, bool acc) {
        const uint64_t vb = dr + s * kTile16;
        if (el) {
#pragma unroll
            for (int kk = k0; kk < k1; ++kk)
                mma_ts(tmem + 2 * kKeys + i * kKeys, tmem + i * kKeys + kk * 8, vb + kk * 128, id_o, acc || kk > 0);
        }
    };
    int s = 0;  // ring slot and its phase, walking K0 V0 K1 V1 ..
    uint32_t ph = 0;
    auto next = [&]() {
        if (++s == Y::kStages) {
            s = 0;
            ph ^= 1u;
        }
    };
    bool ok = wait_bar(sm.bar(Y::kFull), 0);
    if (ok) {
        fence_after_sync();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (w.cnt[i] > 0) issue_s(i, 0);
        if (el) mma_commit(sm.bar(Y::kFree));
    }
    next();
    for (int jj = 0; ok && jj < w.n; ++jj) {
        const int sv = s;  // V(jj), then K(jj + 1)
        ok = !sm.stopped() && wait_bar(sm.bar(Y::kFull + sv), ph);
        next();
        bool have_k = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!ok || jj >= w.cnt[i]) continue;
            ok = wait_bar(sm.bar(Y::kP + i), jj & 1);
            if (!ok) continue;
            fence_after_sync();
            issue_o(i, sv, 0, kFirst / 16, jj > 0);
            ok = wait_bar(sm.bar(Y::kP + 2 + i), jj & 1);
            if (!ok) continue;
            fence_after_sync();
            issue_o(i, sv, kFirst / 16, kKeys / 16, true);
            if (jj + 1 < w.cnt[i]) {
                if (!have_k) ok = wait_bar(sm.bar(Y::kFull + s), ph);
                have_k = ok;
                if (ok) {
                    fence_after_sync();
                    issue_s(i, s);
                }
            } else if (el) {
                mma_commit(sm.bar(Y::kO + i));
            }
        }
        if (!ok) break;
        if (el) {
            mma_commit(sm.bar(Y::kFree + sv));
            if (jj + 1 < w.n) mma_commit(sm.bar(Y::kFree + s));
        }
        next();
    }
    if (!ok && (threadIdx.x & 31) == 0) sm.give_up(status);
    // every MMA and every arrival of theirs is done (bounded) before the CTA
    // gives up its shared memory and TMEM
    if (el) mma_commit(sm.bar(Y::kDrain));
    wait_bar(sm.bar(Y::kDrain), 0);
}

// The softmax of row tile `tile` by its warpgroup, through all its key tiles
// and the last O += P V; false when a wait ran out.  m, l: the row's
// reference maximum (base 2) and sum.  before_p(jj): called by the whole warp
// before tile jj's P is handed over; false to stop.
template <typename T, int D, typename BeforeP>
__device__ __forceinline__ bool softmax_tile(const Smem<D>& sm, uint32_t tmem, const Work& w, int tile, float scale_log2,
                                             int* status, float& m, float& l, BeforeP before_p) {
    using Y = Layout<D>;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + tile * kKeys + lanes, tO = tmem + 2 * kKeys + tile * kKeys + lanes;
    // rows past the sequence's last take its position (their output is not
    // written)
    const int row = w.row0 + tile * kRows + warp * 32 + lane;
    const int my_pos = w.first_pos + min(row, w.rows - 1) / w.G;
    const int warp_pos = __shfl_sync(0xffffffffu, my_pos, 0);  // the warp's first
    const bool pos_scale = scale_log2 > 0.f;
    const float mul = pos_scale ? scale_log2 : 1.f;
    const int count = w.count(tile);
    m = neg_inf();
    l = 0.f;
    bool ok = true;
    for (int jj = 0; jj < count; ++jj) {
        const int key0 = (w.js + jj) * kKeys;
        ok = !sm.stopped() && wait_bar(sm.bar(Y::kS + tile), jj & 1);
        if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
        }
        fence_after_sync();
        float x[kKeys / 32][32];
#pragma unroll
        for (int cc = 0; cc < kKeys / 32; ++cc) tmem_ld32(tS + cc * 32, x[cc]);
        tmem_wait_ld32(x[0]);
#pragma unroll
        for (int cc = 1; cc < kKeys / 32; ++cc) tmem_tie32(x[cc]);
        // with a positive scale the maximum is taken over raw scores and the
        // scale enters the exponent's FMA
        if (!pos_scale) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i) x[i / 32][i % 32] *= scale_log2;
        }
        if (key0 + kKeys - 1 > warp_pos) {
            const int last = my_pos - key0;
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
                if (i > last) x[i / 32][i % 32] = neg_inf();
        }
        float mq[4] = {x[0][0], x[0][1], x[0][2], x[0][3]};
#pragma unroll
        for (int i = 4; i + 7 < kKeys; i += 8) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                mq[c] = max3f(mq[c], x[(i + c) / 32][(i + c) % 32], x[(i + 4 + c) / 32][(i + 4 + c) % 32]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) mq[c] = fmaxf(mq[c], x[kKeys / 32 - 1][28 + c]);
        const float mx = max3f(mq[0], mq[1], fmaxf(mq[2], mq[3])) * mul;
        const bool raise = mx > m + kSlack;
        float alpha = 1.f;
        if (raise) {
            alpha = ex2(m - mx);  // 0 while m is -inf
            m = mx;
            l *= alpha;
        }
        if (jj > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                tmem_ld32(tO + cc * 32, o);
                tmem_wait_ld32(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= alpha;
                tmem_st32(tO + cc * 32, reinterpret_cast<const uint32_t*>(o));
            }
        }
        if (!before_p(jj)) {
            ok = false;
            break;
        }
        const float mref = m == neg_inf() ? 0.f : m;
        const float2 mul2 = make_float2(mul, mul), ref2 = make_float2(-mref, -mref);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int cc = 0; cc < kKeys / 32; ++cc) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float2 e = fma2(make_float2(x[cc][2 * i], x[cc][2 * i + 1]), mul2, ref2);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                sum[i & 1] = add2(sum[i & 1], e);
                p[i] = Half16<T>::pack(e.x, e.y);
            }
            tmem_st16(tS + cc * 16, p);
            if (cc + 1 == kFirst / 32 || cc + 1 == kKeys / 32) {
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.bar(Y::kP + (cc + 1 == kKeys / 32 ? 2 : 0) + tile));
            }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    if (ok && count > 0) {
        ok = wait_bar(sm.bar(Y::kO + tile), 0);
        fence_after_sync();
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) sm.give_up(status);
    return ok;
}

// Position p of 8 consecutive stored columns holds column (PERM) 0, 4, 1, 5,
// 2, 6, 3, 7 of the eight; stored position of column e:
template <bool PERM>
__host__ __device__ constexpr int stored(int e) {
    return PERM ? 2 * (e & 3) + (e >> 2) : e;
}

// Writes the warp's 32 rows of O / l of row tile `tile` to out[token * hq +
// head], through the tile's Q (no longer read) so that they go out in whole
// 128-byte lines.  fix(d0, o): called before the division with the thread's
// columns d0 .. d0 + 31 (stored order).
template <typename TO, int D, bool PERM, typename Fix>
__device__ __forceinline__ void store_tile(const Smem<D>& sm, uint32_t tmem, const Work& w, int tile, float l, bool ok,
                                           TO* out, int hq, Fix fix) {
    using Y = Layout<D>;
    constexpr int kCh = D / 8, kStep = 32 / kCh;  // 16-byte chunks of a row, rows per store
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t tO = tmem + 2 * kKeys + tile * kKeys + (static_cast<uint32_t>(warp * 32) << 16);
    uint8_t* st = sm.p + Y::kOffQ + tile * Y::kTile + warp * 32 * (D * 2);
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
#pragma unroll 1
    for (int cc = 0; cc < D / 32; ++cc) {
        float o[32];
        if (w.count(tile) > 0) {
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld32(o);
        }
        fix(cc * 32, o);
        if (l == 0.f) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint4 v;
            v.x = Half16<TO>::pack(o[8 * c + stored<PERM>(0)] * inv, o[8 * c + stored<PERM>(1)] * inv);
            v.y = Half16<TO>::pack(o[8 * c + stored<PERM>(2)] * inv, o[8 * c + stored<PERM>(3)] * inv);
            v.z = Half16<TO>::pack(o[8 * c + stored<PERM>(4)] * inv, o[8 * c + stored<PERM>(5)] * inv);
            v.w = Half16<TO>::pack(o[8 * c + stored<PERM>(6)] * inv, o[8 * c + stored<PERM>(7)] * inv);
            *reinterpret_cast<uint4*>(st + lane * (D * 2) + (((cc * 4 + c) ^ (lane & 7)) << 4)) = v;
        }
    }
    __syncwarp();
    const int ch = lane % kCh;
    int rr = lane / kCh, row = w.row0 + tile * kRows + warp * 32 + rr;
    int t = row / w.G, h = row - t * w.G;
#pragma unroll 4
    for (int x = 0; x < kCh; ++x) {
        const uint4 v = *reinterpret_cast<const uint4*>(st + rr * (D * 2) + ((ch ^ (rr & 7)) << 4));
        if (ok && row < w.rows) *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(t) * hq + h) * D + ch * 8) = v;
        rr += kStep;
        row += kStep;
        h += kStep;
        while (h >= w.G) {
            h -= w.G;
            ++t;
        }
    }
}

// The same rows as fp32 partials of a split: (m, l) and unnormalised O at
// partial row prow (the thread's row).
template <int D, bool PERM, typename Fix>
__device__ __forceinline__ void store_partial(uint32_t tmem, const Work& w, int tile, float m, float l, bool put,
                                              float* ws_o, float* ws_ml, int64_t prow, Fix fix) {
    const uint32_t tO = tmem + 2 * kKeys + tile * kKeys + (((threadIdx.x >> 5) & 3) * 32 << 16);
    if (put) *reinterpret_cast<float2*>(ws_ml + prow * 2) = make_float2(m, l);
    if (w.count(tile) == 0) return;
#pragma unroll 1
    for (int cc = 0; cc < D / 32; ++cc) {
        float o[32];
        tmem_ld32(tO + cc * 32, o);
        tmem_wait_ld32(o);
        fix(cc * 32, o);
        if (put) {
            float* p = ws_o + prow * D + cc * 32;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                *reinterpret_cast<float4*>(p + 8 * c) =
                    make_float4(o[8 * c + stored<PERM>(0)], o[8 * c + stored<PERM>(1)], o[8 * c + stored<PERM>(2)],
                                o[8 * c + stored<PERM>(3)]);
                *reinterpret_cast<float4*>(p + 8 * c + 4) =
                    make_float4(o[8 * c + stored<PERM>(4)], o[8 * c + stored<PERM>(5)], o[8 * c + stored<PERM>(6)],
                                o[8 * c + stored<PERM>(7)]);
            }
        }
    }
}

// One row of the merge of the splits, by a warp: out = sum_s 2^(m_s - M) o_s /
// sum_s 2^(m_s - M) l_s; split s's partial row is s * step + prow.
constexpr int kMaxSplits = 32;  // one per lane

template <typename TO, int D>
__device__ __forceinline__ void merge_row(const float* ws_o, const float* ws_ml, int splits, int64_t step, int64_t prow,
                                          TO* dst) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float ms = neg_inf(), ls = 0.f;
    if (lane < splits) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(ws_ml + (lane * step + prow) * 2));
        ms = ml.x;
        ls = ml.y;
    }
    float M = ms;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    // a split without a key has (-inf, 0); one whose scores are all NaN (-inf, NaN)
    const float wt = ms == neg_inf() ? ls : ex2(ms - M);
    float Ls = ms == neg_inf() ? ls : wt * ls;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, off);
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int s = 0; s < splits; ++s) {
        const float wgt = __shfl_sync(0xffffffffu, wt, s);
        if (wgt == 0.f) continue;
        const float* p = ws_o + (s * step + prow) * D + lane * E;
        if constexpr (E == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
            o[0] += wgt * v.x;
            o[1] += wgt * v.y;
            o[2] += wgt * v.z;
            o[3] += wgt * v.w;
        } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
            o[0] += wgt * v.x;
            o[1] += wgt * v.y;
        }
    }
    const float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);
    uint32_t v[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) v[e] = Half16<TO>::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
    if constexpr (E == 4) *reinterpret_cast<uint2*>(dst + lane * E) = make_uint2(v[0], v[1]);
    else *reinterpret_cast<uint32_t*>(dst + lane * E) = v[0];
}

// Splits of the key axis: 1 unless the CTAs leave SMs idle; then as many as
// fill them, each at least kMinTiles of the `tiles` long.
constexpr int kMinTiles = 4;
inline int num_splits(int64_t ctas, int64_t tiles, int sms) {
    if (ctas <= 0) return 1;
    int64_t n = sms / ctas;
    if (n > tiles / kMinTiles) n = tiles / kMinTiles;
    if (n > kMaxSplits) n = kMaxSplits;
    return n < 1 ? 1 : static_cast<int>(n);
}

// Sets the kernel's shared memory limit, once per device, and checks that it
// was built with the registers its warpgroups' split needs (setmaxnreg.inc
// would otherwise wait for them).
template <auto kernel>
int prepare_kernel(int bytes, int regs) {
    static std::atomic<int> state[64];  // 0: not yet, 1: ready, 2: too few registers
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
    int s = state[dev].load(std::memory_order_acquire);
    if (s == 0) {
        cudaFuncAttributes fa;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
            cudaFuncGetAttributes(&fa, kernel) != cudaSuccess)
            return PKV_ERR_CUDA;
        s = fa.numRegs >= regs ? 1 : 2;
        state[dev].store(s, std::memory_order_release);
    }
    return s == 1 ? PKV_OK : PKV_ERR_UNSUPPORTED;
}

}  // namespace tcattn
}  // namespace pkv
