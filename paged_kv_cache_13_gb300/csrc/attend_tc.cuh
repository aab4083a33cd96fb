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
// * A tile of keys takes ~3,300 cycles at D = 128 (2,048 of them products), a
//   chain: S read and its maximum, 128 exponentials a thread, P written, both
//   products.  Nothing may spill: with the ring in shared memory hardly any L1
//   is left, and 30 spilled registers cost 40%.
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

// QUEUE: the CTA takes one job after another (see prompt.cu); else one.
template <int D, bool QUEUE>
struct Layout {
    static constexpr int kTile = kRows * D * 2;  // bytes of a 128 x D 16-bit tile
    static constexpr int kStages = D == 128 ? (QUEUE ? 4 : 5) : 8;
    static constexpr int kQueue = 4;  // jobs handed out and not done with, at most
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = 2 * kTile;
    // output rows on their way out, 64 columns at a time, 16 KiB a row tile: in
    // Q's place when no other job's Q can be there yet
    static constexpr int kOffOut = QUEUE ? kOffRing + kStages * kTile : kOffQ;
    static constexpr int kOutTile = QUEUE ? kRows * 128 : kTile;
    static constexpr int kOffBar = kOffRing + kStages * kTile + (QUEUE ? 2 * kOutTile : 0);
    // mbarriers: ring slot filled / read, S done (per tile), P written (first
    // keys of tile 0, 1, then the rest), O done, everything issued done; with a
    // queue also Q written, O read (per tile), job written / done with (per
    // entry), claim answered, V looked through (per slot; see prompt.cu)
    static constexpr int kFull = 0, kFree = kStages, kS = 2 * kStages, kP = kS + 2, kO = kP + 4, kDrain = kO + 2;
    static constexpr int kQ = kDrain + 1, kORead = kQ + 2, kJob = kORead + 2, kJobDone = kJob + kQueue,
                         kClaim = kJobDone + kQueue, kClean = kClaim + 1;
    static constexpr int kBars = QUEUE ? kClean + kStages : kQ;
    static_assert(!QUEUE || kStages % 2 == 0, "V in the odd slots");
    static constexpr int kOffVars = (kOffBar + 8 * kBars + 15) / 16 * 16;
    static constexpr int kOffClaim = kOffVars + 32, kOffJobs = kOffClaim + 16, kJobBytes = 80;
    static constexpr int kBytes = QUEUE ? kOffJobs + kQueue * kJobBytes : kOffClaim;
};
static_assert(Layout<128, true>::kBytes <= 232448 && Layout<64, true>::kBytes <= 232448 &&
                  Layout<128, false>::kBytes <= 232448 && Layout<64, false>::kBytes <= 232448,
              "shared memory");

// A CTA's shared memory.
template <int D, bool QUEUE>
struct Smem {
    using Y = Layout<D, QUEUE>;
    uint8_t* p;
    uint32_t base;
    __device__ __forceinline__ explicit Smem(uint8_t* raw) : p(raw), base(sh_addr(raw)) {}  // raw: 1 KiB-aligned
    __device__ __forceinline__ uint32_t bar(int i) const { return base + Y::kOffBar + 8 * i; }
    __device__ __forceinline__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(p + Y::kOffVars); }
    // raised when a wait ran out
    __device__ __forceinline__ volatile int* stop() const { return reinterpret_cast<int*>(p + Y::kOffVars + 4); }
    // raised when a non-finite V value was taken out of a masked tile of job n
    __device__ __forceinline__ volatile int* odd(int n) const { return reinterpret_cast<int*>(p + Y::kOffVars + 8) + n % Y::kQueue; }
    __device__ __forceinline__ bool stopped() const { return *stop() != 0; }
    __device__ __forceinline__ void give_up(int* status) const {
        atomicOr(status, PKV_STATUS_COPY_TIMEOUT);
        *stop() = 1;
    }
    // the CTA's ring items in order: of a job, item 2 jj is K of its jj-th
    // tile, 2 jj + 1 V
    static __device__ __forceinline__ int slot(int it) { return it % Y::kStages; }
    static __device__ __forceinline__ uint32_t phase(int it) { return static_cast<uint32_t>(it / Y::kStages) & 1u; }
    __device__ __forceinline__ uint8_t* ring(int it) const { return p + Y::kOffRing + slot(it) * Y::kTile; }
    // by one thread, before any other uses the barriers; full: arrivals that
    // fill a ring slot; readers: warps that read a job
    __device__ __forceinline__ void init(int full, int readers) const {
        for (int i = 0; i < Y::kBars; ++i) {
            int n = 1;
            if (i < Y::kFree) n = full;
            if ((i >= Y::kP && i < Y::kO) || (i >= Y::kQ && i < Y::kJob)) n = 4;  // a tile's warps
            if (QUEUE && i >= Y::kJobDone && i < Y::kClaim) n = readers;
            if (QUEUE && i >= Y::kClean) n = 2;
            mbar_init(bar(i), n);
        }
        *stop() = 0;
        for (int i = 0; i < Y::kQueue; ++i) *odd(i) = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
};

// What a CTA has done before the job at hand: ring items, key tiles per row
// tile, jobs in which the row tile had any.  The barriers' phases follow from
// it.
struct Before {
    int items = 0, tiles[2] = {0, 0}, jobs[2] = {0, 0};
    __device__ __forceinline__ int t(int tile) const { return tile ? tiles[1] : tiles[0]; }
    __device__ __forceinline__ int j(int tile) const { return tile ? jobs[1] : jobs[0]; }
    template <typename W>
    __device__ __forceinline__ void add(const W& w) {
        items += 2 * w.n;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tiles[i] += w.cnt[i];
            jobs[i] += w.cnt[i] > 0;
        }
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
// One job; false when a wait ran out.
template <typename T, int D, bool QUEUE>
__device__ __forceinline__ bool mma_job(const Smem<D, QUEUE>& sm, uint32_t tmem, const Work& w, const Before& before) {
    using Y = Layout<D, QUEUE>;
    if (w.n == 0) return true;
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
    // ring slot and its phase, walking K0 V0 K1 V1 .. (by a shuffle, so that the
    // compiler takes the slot as warp-uniform)
    int s = QUEUE ? __shfl_sync(0xffffffffu, sm.slot(before.items), 0) : 0;
    uint32_t ph = sm.phase(before.items);
    auto next = [&]() {
        if (++s == Y::kStages) {
            s = 0;
            ph ^= 1u;
        }
    };
    bool ok = wait_bar(sm.bar(Y::kFull + s), ph);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!ok || w.cnt[i] == 0) continue;
        if (QUEUE) ok = wait_bar(sm.bar(Y::kQ + i), before.jobs[i] & 1);
        fence_after_sync();
        if (ok) issue_s(i, s);
    }
    if (ok && el) mma_commit(sm.bar(Y::kFree + s));
    next();
    for (int jj = 0; ok && jj < w.n; ++jj) {
        const int sv = s;  // V(jj), then K(jj + 1)
        ok = !sm.stopped() && wait_bar(sm.bar(Y::kFull + sv), ph);
        if (QUEUE && ok) ok = wait_bar(sm.bar(Y::kClean + sv), ph);
        next();
        bool have_k = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!ok || jj >= w.cnt[i]) continue;
            const uint32_t turn = (before.tiles[i] + jj) & 1;
            ok = wait_bar(sm.bar(Y::kP + i), turn);
            // the last job's O has been read
            if (QUEUE && ok && jj == 0 && before.jobs[i] > 0) ok = wait_bar(sm.bar(Y::kORead + i), (before.jobs[i] - 1) & 1);
            if (!ok) continue;
            fence_after_sync();
            issue_o(i, sv, 0, kFirst / 16, jj > 0);
            ok = wait_bar(sm.bar(Y::kP + 2 + i), turn);
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
    return ok;
}

// Every MMA and every arrival of theirs is done (bounded) before the CTA gives
// up its shared memory and TMEM.
template <int D, bool QUEUE>
__device__ __forceinline__ void mma_end(const Smem<D, QUEUE>& sm, bool ok, int* status) {
    if (!ok && (threadIdx.x & 31) == 0) sm.give_up(status);
    if (elect()) mma_commit(sm.bar(Layout<D, QUEUE>::kDrain));
    wait_bar(sm.bar(Layout<D, QUEUE>::kDrain), 0);
}

// The softmax of row tile `tile` by its warpgroup, through all its key tiles;
// false when a wait ran out.  m, l: the row's reference maximum (base 2) and
// sum.
template <typename T, int D, bool QUEUE>
__device__ __forceinline__ bool softmax_tile(const Smem<D, QUEUE>& sm, uint32_t tmem, const Work& w, const Before& before,
                                             int tile, float scale_log2, float& m, float& l) {
    using Y = Layout<D, QUEUE>;
    const int turn = before.t(tile);
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
        ok = !sm.stopped() && wait_bar(sm.bar(Y::kS + tile), (turn + jj) & 1);
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
#pragma unroll 1
            for (int cc = 0; cc < D / 16; ++cc) {  // the scores' registers leave room for 16 columns
                float o[16];
                tmem_ld16_wait(tO + cc * 16, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                tmem_st16(tO + cc * 16, reinterpret_cast<const uint32_t*>(o));
            }
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
    return ok;
}

// The last O += P V of the job is done; ok: of softmax_tile.
template <int D, bool QUEUE>
__device__ __forceinline__ bool wait_o(const Smem<D, QUEUE>& sm, const Work& w, const Before& before, int tile, bool ok,
                                       int* status) {
    if (ok && w.count(tile) > 0) {
        ok = wait_bar(sm.bar(Layout<D, QUEUE>::kO + tile), before.j(tile) & 1);
        fence_after_sync();
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && (threadIdx.x & 31) == 0) sm.give_up(status);
    return ok;
}

// Position p of 8 consecutive stored columns holds column (PERM) 0, 4, 1, 5,
// 2, 6, 3, 7 of the eight; stored position of column e:
template <bool PERM>
__host__ __device__ constexpr int stored(int e) {
    return PERM ? 2 * (e & 3) + (e >> 2) : e;
}

// Writes the warp's 32 rows of O / l of row tile `tile` to out[token * hq +
// head], 64 columns at a time through shared memory so that they go out in
// whole 128-byte lines.  fix(d0, o): called before the division with the
// thread's columns d0 .. d0 + 31 (stored order); read(): once O has been read.
template <typename TO, int D, bool PERM, bool QUEUE, typename Fix, typename Read>
__device__ __forceinline__ void store_tile(const Smem<D, QUEUE>& sm, uint32_t tmem, const Work& w, int tile, float l, bool ok,
                                           TO* out, int hq, Fix fix, Read read) {
    using Y = Layout<D, QUEUE>;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t tO = tmem + 2 * kKeys + tile * kKeys + (static_cast<uint32_t>(warp * 32) << 16);
    uint8_t* st = sm.p + Y::kOffOut + tile * Y::kOutTile + warp * 32 * 128;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
#pragma unroll 1
    for (int half = 0; half < D / 64; ++half) {
#pragma unroll 1
        for (int cc = 0; cc < 2; ++cc) {
            float o[32];
            // (set either way: a register that only one way sets would be live
            // all through a loop over jobs)
            if (w.count(tile) > 0) {
                tmem_ld32(tO + half * 64 + cc * 32, o);
                tmem_wait_ld32(o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            fix(half * 64 + cc * 32, o);
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
                *reinterpret_cast<uint4*>(st + lane * 128 + (((cc * 4 + c) ^ (lane & 7)) << 4)) = v;
            }
        }
        if (half + 1 == D / 64) read();
        __syncwarp();
        int rr = lane / 8, row = w.row0 + tile * kRows + warp * 32 + rr;
        int t = row / w.G, h = row - t * w.G;
#pragma unroll 4
        for (int x = 0; x < 8; ++x) {
            const uint4 v = *reinterpret_cast<const uint4*>(st + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (ok && row < w.rows)
                *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(t) * hq + h) * D + half * 64 + (lane & 7) * 8) = v;
            rr += 4;
            row += 4;
            h += 4;
            while (h >= w.G) {
                h -= w.G;
                ++t;
            }
        }
        __syncwarp();
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
