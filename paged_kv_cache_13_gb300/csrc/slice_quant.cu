// Multi-query attention over the quantised cache for more than 24 rows per
// (sequence, KV head): slices of a prompt, wide verify passes.
//
// The tensor-core attention of attend_tc.cuh with K/V tiles made by seven
// unpacking warps: they read the codes of a block (16 bytes a lane, whole
// rows), dequantise them to fp16 -- (c - z) and the product with s each rounded
// to fp16 -- and write them into the ring with the MMAs' swizzle, so a block is
// unpacked once per 256 query rows.  Sink and window rows are copied as fp16,
// slots past the context as zeros.  Everything is fp16: queries and values
// beyond +-65504 saturate (bf16 would cost each value 8 times the rounding
// error, and K and V are within a factor of 2 of their originals).
// INT4 codes come out of a word as the pairs (0, 4) (1, 5) (2, 6) (3, 7) of its
// eight columns and stay in that order: the query takes the same order, the
// output is put back when it is stored.
// Measured (8 slices of 512 tokens, the last of 4,096, 32 heads over 8, INT4):
// 262 us, 980 TFLOP/s.  Bound by the issue slots the unpacking and the softmax
// share (52% taken, ~2,700 instructions a tile and scheduler) and the softmax's
// chain.  On the way here: four unpacking warps and five instructions a pair of
// codes 444 us; blocks without branches and (c - z) in one FMA 362; table
// entries a tile ahead 343; seven warps 324; nothing spilled 262.

#include "slice_quant.cuh"

#include "attend_tc.cuh"
#include "balanced.cuh"

namespace pkv {
namespace {

using namespace tcattn;

constexpr int BS = 16;
constexpr int kThreads = 512;  // warps 0-3, 4-7: softmax of tiles 0, 1; 8-14: unpacking; 15: MMAs
constexpr int kWarpUnpack = 8, kUnpackWarps = 7, kWarpMma = 15;
constexpr int kBlocks = kKeys / BS;  // blocks of a ring item
// Registers: launched at 128 a thread, then softmax 176, the others 80.
constexpr int kLaunchRegs = 128;
static_assert(2 * 128 * 176 + 2 * 128 * 80 <= kThreads * kLaunchRegs, "register split");

template <int D, int QMODE, int NG>
struct Codes {
    static constexpr bool INT4 = QMODE == PKV_QMODE_INT4_ASYM;
    static constexpr int CB = INT4 ? D / 2 : D;  // code bytes per row
    static constexpr int CPR = CB / 16;          // 16-byte pieces per row
    static constexpr int RPI = 32 / CPR;         // rows a warp reads per load
    static constexpr int LPB = BS / RPI;         // loads per block and lane
    static constexpr int OUT = INT4 ? 4 : 2;     // 16-byte fp16 chunks per piece
};

__device__ __forceinline__ uint32_t h2(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// two e4m3 codes in the low 16 bits of w -> fp16 pair
__device__ __forceinline__ __half2 e4m3x2(uint32_t w) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<unsigned short>(w & 0xffffu)));
    return as_h2(d);
}

// Whether every value of a (scale, zero point) pair is finite and comes out of
// the short way as of the long one: 0 <= s < 128, and z 0 or 2^-5 <= |z| <=
// 496, so that s 2^9 is finite, (15 + |z|) s <= 65504, and c - z, a multiple of
// 2^-15, stays exact at 2^-9 of its size even as a subnormal.
template <bool INT4>
__device__ __forceinline__ bool ordinary(__half scale, __half zero) {
    const unsigned z = __half_as_ushort(zero) & 0x7fffu;
    return __half_as_ushort(scale) < 0x5800u && (!INT4 || z == 0 || z - 0x2800u <= 0x5FC0u - 0x2800u);
}

// fp16 of x, finite values saturating
__device__ __forceinline__ __half sat16(float x) {
    return __float2half_rn(fabsf(x) <= 3.4e38f ? fminf(fmaxf(x, -65504.f), 65504.f) : x);
}

// Eight 16-bit values as fp16 in stored order.
template <typename T, bool PERM>
__device__ __forceinline__ uint4 as_fp16(uint4 v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (!std::is_same<T, __half>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T* e = reinterpret_cast<const T*>(&w[i]);
            w[i] = h2(__halves2half2(sat16(Half16<T>::to_float(e[0])), sat16(Half16<T>::to_float(e[1]))));
        }
    }
    if constexpr (!PERM) return make_uint4(w[0], w[1], w[2], w[3]);
    return make_uint4(__byte_perm(w[0], w[2], 0x5410u), __byte_perm(w[0], w[2], 0x7632u),
                      __byte_perm(w[1], w[3], 0x5410u), __byte_perm(w[1], w[3], 0x7632u));
}

// The sequence a CTA works for.
struct Seq {
    int b, kvh, ctx, w0, sinks, nblk;
};

// The value at (token t, column d) of V, as the kernel reads it (the rare path
// that puts non-finite values back).
template <typename T, int D, int QMODE, int NG>
__device__ float value_at(const QuantCache& a, const Seq& s, int t, int d) {
    const T* src = nullptr;
    if (t >= s.w0)
        src = static_cast<const T*>(a.win[1]) +
              (((static_cast<int64_t>(s.b) * a.ring + (t / BS) % a.ring) * a.hkv + s.kvh) * BS + t % BS) * D;
    else if (t < s.sinks)
        src = static_cast<const T*>(a.sink[1]) + ((static_cast<int64_t>(s.b) * a.n_sink + t) * a.hkv + s.kvh) * D;
    if (src) return Half16<T>::to_float(src[d]);
    if (QMODE == PKV_QMODE_INT4_ASYM) return 0.f;  // always finite
    const int phys = a.tables[static_cast<int64_t>(s.b) * a.max_blocks + t / BS];
    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(a.num_blocks)) return 0.f;
    const int64_t row = (static_cast<int64_t>(phys) * a.hkv + s.kvh) * BS + t % BS;
    return (a.codes[1][row * D + d] & 0x7f) == 0x7f ? __int_as_float(0x7fc00000) : 0.f;
}

// The unpacking warps: block x of ring item it is job 8 it + x, and warp u takes
// jobs u, u + 7, ..: each at its own pace, a job's codes loaded while the one
// before is unpacked and its table entry a job earlier still (the codes'
// addresses wait for it).
template <typename T, int D, int QMODE, int NG>
__device__ __forceinline__ void unpack_warp(const Smem<D, false>& sm, const QuantCache& a, const Work& w, const Seq& s, int u) {
    using C = Codes<D, QMODE, NG>;
    using Y = Layout<D, false>;
    constexpr bool PERM = C::INT4;
    const int lane = threadIdx.x & 31, r = lane % C::RPI, c = lane / C::RPI;
    const int gi = NG == 2 ? c / (C::CPR / 2) : 0;
    const int32_t* trow = a.tables + static_cast<int64_t>(s.b) * a.max_blocks;
    const int jobs = 2 * w.n * kBlocks;
    struct Piece {
        uint4 code;
        __half scale, zero;
    };
    Piece p[C::LPB];
    bool bad = false;
    // a job's block of the sequence; its table entry (-1: nothing to read
    // there: past the context, or in the window)
    auto block = [&](int job) { return (w.js + job / (2 * kBlocks)) * kBlocks + job % kBlocks; };
    auto fetch = [&](int job) {
        const int lb = block(job);
        return job < jobs && lb < s.nblk && lb * BS < s.w0 ? __ldg(trow + lb) : -1;
    };
    auto find = [&](int job, int phys) -> int64_t {  // the block's first row in the pool, or -1
        if (static_cast<unsigned>(phys) < static_cast<unsigned>(a.num_blocks))
            return (static_cast<int64_t>(phys) * a.hkv + s.kvh) * BS;
        const int lb = block(job);
        if (job < jobs && lb < s.nblk && lb * BS < s.w0) bad = true;
        return -1;
    };
    auto load = [&](int i, int kv, int64_t row0) {
        if (row0 < 0) return;
        const int64_t row = row0 + i * C::RPI + r;
        p[i].code = ldg_stream((kv ? a.codes[1] : a.codes[0]) + row * C::CB + 16 * c);
        p[i].scale = (kv ? a.scale[1] : a.scale[0])[row * NG + gi];
        if constexpr (C::INT4) p[i].zero = (kv ? a.zero[1] : a.zero[0])[row * NG + gi];
    };
    int64_t next = find(u, fetch(u));
    int phys = fetch(u + kUnpackWarps);
#pragma unroll
    for (int i = 0; i < C::LPB; ++i) load(i, 0, next);
    bool odd = false;
    for (int job = u; job < jobs && !__any_sync(0xffffffffu, sm.stopped()); job += kUnpackWarps) {
        const int it = job / kBlocks, jj = it >> 1, kv = it & 1;
        if (it >= Y::kStages && !__all_sync(0xffffffffu, wait_bar(sm.bar(Y::kFree + sm.slot(it)), sm.phase(it - Y::kStages)))) {
            if (lane == 0) sm.give_up(a.status);
            break;
        }
        uint8_t* tile = sm.ring(it);
        const bool guard = kv && w.masked(jj);  // V of a tile some row must not see whole
        const int64_t cur = next;
        const int t0 = block(job) * BS, row_in = job % kBlocks * BS;
        const int kv_next = (job + kUnpackWarps) / kBlocks & 1;
        next = find(job + kUnpackWarps, phys);
        phys = fetch(job + 2 * kUnpackWarps);
        // ordinary blocks (quantised and whole, scales and zero points in range)
        // go straight through, no branch between the pieces
        bool plain = cur >= 0 && t0 + BS <= s.ctx && t0 >= s.sinks && (C::INT4 || !guard);  // (INT4: finite)
#pragma unroll
        for (int i = 0; i < C::LPB; ++i) plain &= ordinary<C::INT4>(p[i].scale, p[i].zero);
        if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
            for (int i = 0; i < C::LPB; ++i) {
                const Piece& q = p[i];
                const uint32_t word4[4] = {q.code.x, q.code.y, q.code.z, q.code.w};
                const int rr = row_in + i * C::RPI + r;
                uint4 out[C::OUT];
                if constexpr (C::INT4) {
                    // a nibble masked in place is the subnormal c 2^-24 or 16 c
                    // 2^-24: (c - z) 2^-9 in one FMA
                    const __half2 even = as_h2(0x78007800u), odd4 = as_h2(0x68006800u);  // 2^15, 2^11
                    const __half2 mz = __half2half2(__hmul(q.zero, __ushort_as_half(0x9800)));    // -z 2^-9
                    const __half2 sc = __half2half2(__hmul(q.scale, __ushort_as_half(0x6000)));   // s 2^9
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = word4[j], hi = lo >> 8;
                        out[j].x = h2(__hmul2(__hfma2(as_h2(lo & 0x000F000Fu), even, mz), sc));
                        out[j].y = h2(__hmul2(__hfma2(as_h2(lo & 0x00F000F0u), odd4, mz), sc));
                        out[j].z = h2(__hmul2(__hfma2(as_h2(hi & 0x000F000Fu), even, mz), sc));
                        out[j].w = h2(__hmul2(__hfma2(as_h2(hi & 0x00F000F0u), odd4, mz), sc));
                    }
                } else {
                    const __half2 sc = __half2half2(q.scale);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        out[j] = make_uint4(h2(__hmul2(e4m3x2(word4[2 * j]), sc)), h2(__hmul2(e4m3x2(word4[2 * j] >> 16), sc)),
                                            h2(__hmul2(e4m3x2(word4[2 * j + 1]), sc)),
                                            h2(__hmul2(e4m3x2(word4[2 * j + 1] >> 16), sc)));
                }
#pragma unroll
                for (int j = 0; j < C::OUT; ++j)
                    *reinterpret_cast<uint4*>(tile + tile_off(rr, C::OUT * c + j)) = out[j];
                load(i, kv_next, next);
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.bar(Y::kFull + sm.slot(it)));
            continue;
        }
        // blocks with sinks, window rows or slots past the context
        const bool special = cur < 0 || t0 + BS > s.ctx || t0 < s.sinks;
#pragma unroll
        for (int i = 0; i < C::LPB; ++i) {
            const int row = i * C::RPI + r, t = t0 + row;
            uint4 out[C::OUT];
            const Piece& q = p[i];
            const uint32_t word4[4] = {q.code.x, q.code.y, q.code.z, q.code.w};
            const __half2 sc = __half2half2(q.scale);
            if constexpr (C::INT4) {
                const __half2 z = __half2half2(q.zero), k1024 = as_h2(0x64006400u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        // 1024 + c, c, c - z, (c - z) s
                        const __half2 h = as_h2(((word4[j] >> (4 * n)) & 0x000F000Fu) | 0x64006400u);
                        v[n] = h2(__hmul2(__hsub2(__hsub2(h, k1024), z), sc));
                    }
                    out[j] = make_uint4(v[0], v[1], v[2], v[3]);
                }
                const float zf = __half2float(q.zero);
                if (fmaxf(fabsf(zf), fabsf(15.f - zf)) * __half2float(q.scale) > 65504.f) {  // may saturate
                    uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        o[n] = h2(__hmax2(__hmin2(as_h2(o[n]), as_h2(0x7BFF7BFFu)), as_h2(0xFBFFFBFFu)));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t v[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        v[n] = h2(__hmul2(e4m3x2(word4[2 * j + n / 2] >> (16 * (n & 1))), sc));
                    }
                    out[j] = make_uint4(v[0], v[1], v[2], v[3]);
                }
                if (__half2float(q.scale) > 65504.f / 448.f) {  // may saturate; NaN codes stay
                    uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
                    for (int n = 0; n < 8; ++n)
                        o[n] = h2(__hmax2_nan(__hmin2_nan(as_h2(o[n]), as_h2(0x7BFF7BFFu)), as_h2(0xFBFFFBFFu)));
                }
            }
            if (special) {
                const T* src = nullptr;
                if (t < s.ctx) {
                    if (t >= s.w0)
                        src = static_cast<const T*>(kv ? a.win[1] : a.win[0]) +
                              (((static_cast<int64_t>(s.b) * a.ring + (t / BS) % a.ring) * a.hkv + s.kvh) * BS + t % BS) * D;
                    else if (t < s.sinks)
                        src = static_cast<const T*>(kv ? a.sink[1] : a.sink[0]) +
                              ((static_cast<int64_t>(s.b) * a.n_sink + t) * a.hkv + s.kvh) * D;
                }
                if (src || t >= s.ctx || cur < 0) {
#pragma unroll
                    for (int j = 0; j < C::OUT; ++j)
                        out[j] = src ? as_fp16<T, PERM>(*reinterpret_cast<const uint4*>(src + (C::OUT * c + j) * 8))
                                     : make_uint4(0, 0, 0, 0);
                }
            }
            if (guard) {  // non-finite values: out, and back in for the rows that see them
                uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
                for (int n = 0; n < 4 * C::OUT; ++n) {
                    if ((o[n] & 0x7C00u) == 0x7C00u) { o[n] &= 0xffff0000u; odd = true; }
                    if ((o[n] & 0x7C000000u) == 0x7C000000u) { o[n] &= 0x0000ffffu; odd = true; }
                }
            }
            const int rr = row_in + row;
#pragma unroll
            for (int j = 0; j < C::OUT; ++j) *reinterpret_cast<uint4*>(tile + tile_off(rr, C::OUT * c + j)) = out[j];
            load(i, kv_next, next);
        }
        if (__any_sync(0xffffffffu, odd) && lane == 0) *sm.odd(0) = 1;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.bar(Y::kFull + sm.slot(it)));
    }
    if (bad) atomicOr(a.status, PKV_STATUS_BAD_BLOCK);
}

template <typename T, int D, int QMODE, int NG>
__global__ void __launch_bounds__(kThreads, 1)
    slice_tc_kernel(const __grid_constant__ QuantCache a, int splits, float* ws_o, float* ws_ml) {
    using Y = Layout<D, false>;
    constexpr bool PERM = QMODE == PKV_QMODE_INT4_ASYM;
    constexpr int kCh = D / 8;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Smem<D, false> sm(smem_raw);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // a sequence's later rows see more keys: they go first
    const int x = gridDim.x - 1 - blockIdx.x, split = x % splits, tile_row = x / splits;
    Seq s;
    s.kvh = blockIdx.y;
    s.b = blockIdx.z;
    const int q0 = a.q_start[s.b], L = a.q_start[s.b + 1] - q0, cap = a.max_blocks * BS;
    const int ctx = a.ctx_lens[s.b];
    s.ctx = min(max(ctx, 0), cap);
    s.w0 = a.window > 0 ? max(s.ctx - a.window, 0) / BS * BS : s.ctx;
    s.sinks = s.w0 > 0 ? a.n_sink : 0;
    s.nblk = (s.ctx + BS - 1) / BS;
    Work w;
    w.row0 = tile_row * kCtaRows;
    w.G = a.G;
    w.rows = min(L, a.max_q_len) * a.G;
    w.first_pos = s.ctx - L;
    if (L <= 0 || w.row0 >= w.rows) return;
    if (threadIdx.x == 0 && tile_row == 0 && s.kvh == 0 && split == 0 &&
        (ctx < L || ctx > cap || L > a.max_q_len))
        atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
    w.set_tiles(split, splits);
    const int tile = warp >> 2;  // 0, 1: softmax
    const T* qbase = static_cast<const T*>(a.q) + (static_cast<int64_t>(q0) * a.hq + s.kvh * a.G) * D;
    if (warp == kWarpUnpack && lane == 0) {
        sm.init(kBlocks, 0);
    } else if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sh_addr(sm.tmem_slot())),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (tile < 2) {
        // the warp's 32 query rows as fp16, whole 128-byte lines at a time
        constexpr int kStep = 32 / kCh;
        const int rr0 = (warp & 3) * 32 + lane / kCh, ch = lane % kCh;
        int row = w.row0 + tile * kRows + rr0;
        int tok = row / a.G, h = row - tok * a.G;
        uint4 v[kCh];
#pragma unroll
        for (int y = 0; y < kCh; ++y) {
            v[y] = make_uint4(0, 0, 0, 0);
            if (row < w.rows)
                v[y] = *reinterpret_cast<const uint4*>(qbase + (static_cast<int64_t>(tok) * a.hq + h) * D + ch * 8);
            row += kStep;
            h += kStep;
            while (h >= a.G) {
                h -= a.G;
                ++tok;
            }
        }
#pragma unroll
        for (int y = 0; y < kCh; ++y)
            *reinterpret_cast<uint4*>(sm.p + Y::kOffQ + tile * Y::kTile + tile_off(rr0 + y * kStep, ch)) =
                as_fp16<T, PERM>(v[y]);
        fence_async_shared();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *sm.tmem_slot();

    if (tile >= 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kWarpMma) {
            mma_end(sm, mma_job<__half>(sm, tmem, w, Before()), a.status);
        } else {
            unpack_warp<T, D, QMODE, NG>(sm, a, w, s, warp - kWarpUnpack);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        float m, l;
        bool ok = softmax_tile<__half>(sm, tmem, w, Before(), tile, a.scale_log2, m, l);
        ok = wait_o(sm, w, Before(), tile, ok, a.status);
        const int row = w.row0 + tile * kRows + (warp & 3) * 32 + lane;
        const int tok = row / a.G, h = row - tok * a.G;
        const bool odd = w.count(tile) > 0 && *sm.odd(0) != 0;
        const int my_pos = w.first_pos + min(row, w.rows - 1) / a.G;
        auto put_back = [&](int d0, float (&o)[32]) {
            if (!odd) return;
            for (int t = w.masked_from(); t <= my_pos && t < min((w.js + w.n) * kKeys, s.ctx); ++t) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float f = value_at<T, D, QMODE, NG>(a, s, t, d0 + (i & ~7) + (i & 7));
                    if (!(fabsf(f) <= 3.4e38f)) o[(i & ~7) + stored<PERM>(i & 7)] += f;
                }
            }
        };
        if (splits == 1) {
            store_tile<T, D, PERM>(sm, tmem, w, tile, l, ok,
                                   static_cast<T*>(a.out) + (static_cast<int64_t>(q0) * a.hq + s.kvh * a.G) * D, a.hq,
                                   put_back, [] {});
        } else {
            const int64_t prow = ((static_cast<int64_t>(split) * a.batch + s.b) * a.max_q_len + tok) * a.hq + s.kvh * a.G + h;
            store_partial<D, PERM>(tmem, w, tile, m, l, ok && row < w.rows, ws_o, ws_ml, prow, put_back);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Merge of the splits: one CTA per 256 rows, a warp per row at a time.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    slice_merge_kernel(const __grid_constant__ QuantCache a, int splits, const float* ws_o, const float* ws_ml) {
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int q0 = a.q_start[b], L = a.q_start[b + 1] - q0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (L <= 0) return;
    const int rows = min(L, a.max_q_len) * a.G, end = min((static_cast<int>(blockIdx.x) + 1) * kCtaRows, rows);
    for (int row = blockIdx.x * kCtaRows + (threadIdx.x >> 5); row < end; row += kMergeWarps) {
        const int tok = row / a.G, h = kvh * a.G + row - tok * a.G;
        merge_row<T, D>(ws_o, ws_ml, splits, static_cast<int64_t>(a.batch) * a.max_q_len * a.hq,
                        (static_cast<int64_t>(b) * a.max_q_len + tok) * a.hq + h,
                        static_cast<T*>(a.out) + ((static_cast<int64_t>(q0) + tok) * a.hq + h) * D);
    }
}

int64_t row_tiles(int64_t max_q_len, int64_t G) { return (max_q_len * G + kCtaRows - 1) / kCtaRows; }

int slice_splits(int64_t batch, int64_t hkv, int64_t G, int64_t max_blocks, int64_t max_q_len) {
    return num_splits(row_tiles(max_q_len, G) * hkv * batch, (max_blocks * BS + kKeys - 1) / kKeys, num_sms());
}

template <typename T, int D, int QMODE, int NG>
int launch(const QuantCache& a, float* workspace, cudaStream_t st) {
    const int rc = prepare_kernel<slice_tc_kernel<T, D, QMODE, NG>>(Layout<D, false>::kBytes, kLaunchRegs);
    if (rc != PKV_OK) return rc;
    const int splits = slice_splits(a.batch, a.hkv, a.G, a.max_blocks, a.max_q_len);
    const unsigned tiles = static_cast<unsigned>(row_tiles(a.max_q_len, a.G));
    float* ws_ml = splits > 1 ? workspace + static_cast<size_t>(splits) * a.batch * a.max_q_len * a.hq * D : nullptr;
    slice_tc_kernel<T, D, QMODE, NG>
        <<<dim3(tiles * splits, a.hkv, a.batch), kThreads, Layout<D, false>::kBytes, st>>>(a, splits, workspace, ws_ml);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
    if (splits == 1) return PKV_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, a.hkv, a.batch);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, slice_merge_kernel<T, D>, a, splits, static_cast<const float*>(workspace),
                              static_cast<const float*>(ws_ml)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

template <typename T>
int launch_t(const QuantCache& a, int D, float* ws, cudaStream_t st) {
    if (a.int4) {
        if (D == 64) return launch<T, 64, PKV_QMODE_INT4_ASYM, 1>(a, ws, st);
        return a.groups == 2 ? launch<T, 128, PKV_QMODE_INT4_ASYM, 2>(a, ws, st)
                             : launch<T, 128, PKV_QMODE_INT4_ASYM, 1>(a, ws, st);
    }
    return D == 64 ? launch<T, 64, PKV_QMODE_FP8_E4M3, 1>(a, ws, st) : launch<T, 128, PKV_QMODE_FP8_E4M3, 1>(a, ws, st);
}

}  // namespace

size_t slice_quant_workspace(int64_t batch, int64_t hq, int64_t hkv, int64_t D, int64_t max_blocks, int64_t max_q_len) {
    const int n = slice_splits(batch, hkv, hq / hkv, max_blocks, max_q_len);
    return n == 1 ? 0 : static_cast<size_t>(n) * batch * max_q_len * hq * (D + 2) * sizeof(float);
}

int launch_slice_quant(const QuantCache& a, int D, bool bf16, float* workspace, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, D, workspace, st) : launch_t<__half>(a, D, workspace, st);
}

}  // namespace pkv
