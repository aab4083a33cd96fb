// Attention of packed prompts over their own (unpaged) K/V rows:
// pkv_prompt_attention.
//
// What it computes: query row i of sequence b sits at position p = S_b - L_b
// + i of its S_b K/V rows, and
//   out[q_start[b] + i, h] = sum_{t <= p} softmax_t(scale <q, k_t>) v_t
// over KV head h / G ("The 8GB VRAM Breakthrough", §5: the prefill that
// precedes the decode loop).
//
// Design: one CTA per 256 (query token, query head) rows of one (sequence, KV
// head) -- a row is token i / G, head i % G, so a group's heads share every
// K/V tile -- as two MMA tiles of 128 rows that take turns: while the softmax
// of one runs, the tensor cores work for the other.
// * Tiles of 128 keys of K and V come by TMA (one box each, 128-byte swizzle)
//   through a ring of kStages shared-memory slots, in the order K0 V0 K1 V1 ..
// * S = Q K^T (M 128, N 128) goes to TMEM; thread r of a tile's softmax
//   warpgroup owns row r whole: no exchange between threads.  Online softmax
//   in base 2, the reference maximum raised only by more than kSlack (O is
//   then rescaled in TMEM; S done implies the previous O += P V done, both
//   being issued by one thread in order).
// * P, rounded to the 16-bit type, overwrites its S in TMEM and is the A
//   operand of O += P V; V is the MN-major B operand.
// * One thread issues every MMA: O0 += P0 V(j), S0(j + 1), O1 += P1 V(j),
//   S1(j + 1), so each warpgroup has the other's two products (2 x 512 cycles
//   at D = 128) for its softmax.
// * Long K/V axes with few rows: gridded over splits of the key tiles, fp32
//   partials (m, l, o) merged by a second kernel.
// Causal masks touch only tiles that reach past a warp's first position.  A
// V row that a tile's other rows must not see may hold NaN or infinities (0 x
// NaN would reach them through the product): those tiles are scanned, their
// non-finite values taken out, and added back to the rows that do see them.

#include <cuda.h>
#include <math.h>

#include <atomic>
#include <mutex>

#include "balanced.cuh"
#include "tc5.cuh"

namespace pkv {
namespace {

using namespace tc5;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // log2 units a score may exceed the reference maximum by
constexpr int kRows = 128;     // query rows per MMA tile
constexpr int kCtaRows = 256;  // two tiles
constexpr int kKeys = 128;     // keys per tile
constexpr int kFirst = 64;     // keys of P handed to the MMAs before the rest is computed
constexpr int kThreads = 384;  // warps 0-3, 4-7: softmax of tiles 0, 1; 8: copies; 9: MMAs
constexpr int kWarpLoad = 8, kWarpMma = 9;
// Registers: launched at 168 a thread; the softmax warpgroups take 232, the
// third gives its own back down to 40: 2 x 128 x 232 + 128 x 40 = 384 x 168.
constexpr int kLaunchRegs = 168;
static_assert(2 * 128 * 232 + 128 * 40 <= kThreads * kLaunchRegs, "register split exceeds the launch's registers");
constexpr int kTmemCols = 512;  // S0, S1, O0, O1: 128 columns each

template <int D>
struct Layout {
    static constexpr int kTile = kRows * D * 2;  // bytes of a 128 x D 16-bit tile
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = 2 * kTile;
    static constexpr int kOffBar = kOffRing + kStages * kTile;
    static constexpr int kFull = 0, kFree = kStages, kS = 2 * kStages, kP = kS + 2, kO = kP + 4, kDrain = kO + 2;
    static constexpr int kBars = kDrain + 1;
    static constexpr int kOffVars = kOffBar + 8 * kBars;
    static constexpr int kBytes = kOffVars + 16 + 1024;  // and the alignment of the base
};
static_assert(Layout<128>::kBytes <= 232448 && Layout<64>::kBytes <= 232448, "shared memory");

struct PromptArgs {
    const void* q;
    const void* v;
    const int32_t* q_start;
    const int32_t* kv_start;
    int batch, T, S, hq, hkv, G, splits;
    int64_t qs, vs;
    float scale_log2;
    void* out;
    float* ws_o;   // [splits, T, Hq, D]
    float* ws_ml;  // [splits, T, Hq, 2]
    int* status;
};

// The rows of one CTA.  Slot u of the grid belongs to the last sequence b
// with off(b) = floor(q_start[b] G / 256) + b <= u and is its rows 256 (u -
// off(b)) ..: off(b + 1) - off(b) is at least the sequence's 256-row tiles,
// so each has a slot, and the grid's size follows from T and the batch alone.
struct Job {
    int b, q0, L, k0, S, first_pos;
    int row0, rows;  // first row in the sequence, rows of the sequence
};

// Warp-collective; false when the slot has no rows.
__device__ __forceinline__ bool find_job(const int32_t* q_start, const int32_t* kv_start, int batch, int T, int S, int G,
                                         int u, Job& job) {
    const int lane = threadIdx.x & 31;
    auto start = [&](int b) { return min(max(q_start[b], 0), T); };
    int lo = 0, n = batch;
    int qa, qe, ka, ke;
    if (batch < 32) {  // every start in one round of loads
        const int qv = lane <= batch ? start(lane) : 0, kv = lane <= batch ? min(max(kv_start[lane], 0), S) : 0;
        const unsigned le = __ballot_sync(0xffffffffu, lane < batch &&
                                                           static_cast<int64_t>(qv) * G / kCtaRows + lane <= u);
        if (le == 0) return false;
        lo = __popc(le) - 1;
        qa = __shfl_sync(0xffffffffu, qv, lo);
        qe = __shfl_sync(0xffffffffu, qv, lo + 1);
        ka = __shfl_sync(0xffffffffu, kv, lo);
        ke = __shfl_sync(0xffffffffu, kv, lo + 1);
    } else {
    for (;;) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const bool le = lane * step < n &&
                        static_cast<int64_t>(start(b)) * G / kCtaRows + b <= u;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        if (c == 0) return false;
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
        if (n == 1) break;
    }
    qa = start(lo);
    qe = start(lo + 1);
    ka = min(max(kv_start[lo], 0), S);
    ke = min(max(kv_start[lo + 1], 0), S);
    }
    job.b = lo;
    job.q0 = qa;
    job.L = qe - qa;
    job.k0 = ka;
    job.S = max(ke - ka, 0);
    if (job.L <= 0) return false;
    const int64_t off = static_cast<int64_t>(job.q0) * G / kCtaRows + lo;
    const int64_t row0 = (u - off) * kCtaRows;
    if (row0 < 0 || row0 >= static_cast<int64_t>(job.L) * G) return false;  // < 0: starts out of order
    job.row0 = static_cast<int>(row0);
    job.rows = job.L * G;
    job.first_pos = job.S - job.L;
    return true;
}

// Byte offset of (row, 16-byte chunk ch) in a swizzled tile of 128-byte rows
// (64 columns per half, halves kRows x 128 bytes apart).
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
    return (ch >> 3) * (kRows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
};
template <>
struct Pair<__half> {
    using type = __half2;
};

// acc + 0 * (the eight values of w): NaN once any of them is not finite
template <typename T>
__device__ __forceinline__ void probe(typename Pair<T>::type (&acc)[4], uint4 w) {
    using P = typename Pair<T>::type;
    const uint32_t zero = 0;
    const P z = *reinterpret_cast<const P*>(&zero);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __hfma2(*reinterpret_cast<const P*>(&x[i]), z, acc[i]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ PromptArgs a) {
    using Y = Layout<D>;
    constexpr int kCh = D / 8;  // 16-byte chunks per row
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = sh_addr(sm);
    const uint32_t bar0 = sbase + Y::kOffBar;
    auto bar = [&](int i) { return bar0 + 8 * i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Y::kOffVars);
    volatile int* stop_flag = reinterpret_cast<int*>(sm + Y::kOffVars + 4);
    volatile int* odd_flag = reinterpret_cast<int*>(sm + Y::kOffVars + 8);  // a non-finite V value was taken out

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // slots from the last one down: a sequence's later rows see more keys
    const int per_slot = a.hkv * a.splits;
    const int u = (gridDim.x - 1 - blockIdx.x) / per_slot;
    const int kvh = (gridDim.x - 1 - blockIdx.x) % per_slot / a.splits;
    const int split = (gridDim.x - 1 - blockIdx.x) % a.splits;

    if (blockIdx.x == 0 && warp == kWarpMma) {  // the ranges are checked once per call
        bool bad = false;
        for (int j = lane; j < a.batch; j += 32) {
            const int q0 = a.q_start[j], q1 = a.q_start[j + 1], k0 = a.kv_start[j], k1 = a.kv_start[j + 1];
            bad |= q0 < 0 || q1 < q0 || q1 > a.T || k0 < 0 || k1 < k0 || k1 > a.S || k1 - k0 < q1 - q0;
        }
        if (bad) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
    }
    Job job;
    if (!find_job(a.q_start, a.kv_start, a.batch, a.T, a.S, a.G, u, job)) return;
    // key tiles of the two row tiles, and this split's share [js, je) of them
    int cnt[2], total = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r1 = min(job.row0 + (i + 1) * kRows, job.rows);
        const int last = job.first_pos + (r1 - 1) / a.G;
        cnt[i] = r1 > job.row0 + i * kRows && last >= 0 ? last / kKeys + 1 : 0;
        total = max(total, cnt[i]);
    }
    const int js = static_cast<int>(static_cast<int64_t>(total) * split / a.splits);
    const int je = static_cast<int>(static_cast<int64_t>(total) * (split + 1) / a.splits);
#pragma unroll
    for (int i = 0; i < 2; ++i) cnt[i] = max(min(cnt[i], je) - js, 0);
    const int n = max(cnt[0], cnt[1]);

    // ring item 2 jj is K of the jj-th tile, 2 jj + 1 its V
    auto slot = [&](int it) { return it % Y::kStages; };
    auto phase = [&](int it) { return static_cast<uint32_t>(it / Y::kStages) & 1u; };
    auto load_item = [&](int it) {
        const int s = slot(it);
        mbar_arrive_expect_tx(bar(Y::kFull + s), Y::kTile);
        tma_load(sbase + Y::kOffRing + s * Y::kTile, it & 1 ? &vmap : &kmap, job.k0 + (js + it / 2) * kKeys, kvh,
                 bar(Y::kFull + s));
    };
    const int early = min(2 * n, Y::kStages);  // items the empty ring takes
    const int tile = warp >> 2;                // softmax: 0 or 1
    if (warp == kWarpLoad && lane == 0) {
        for (int i = 0; i < Y::kBars; ++i) mbar_init(bar(i), i >= Y::kP && i < Y::kP + 4 ? 4 : 1);
        *stop_flag = 0;
        *odd_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
        for (int it = 0; it < early; ++it) load_item(it);  // on their way while Q is fetched
    } else if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sh_addr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (tile < 2) {
        // the warp's 32 query rows, whole 128-byte lines at a time: lane l
        // takes chunk l % kCh of rows l / kCh, l / kCh + kStep, ..
        constexpr int kStep = 32 / kCh;
        const int rr0 = (warp & 3) * 32 + lane / kCh, ch = lane % kCh;
        int row = job.row0 + tile * kRows + rr0;
        int tok = row / a.G, h = row - tok * a.G;
        const T* base = static_cast<const T*>(a.q) + static_cast<int64_t>(job.q0) * a.qs + kvh * a.G * D + ch * 8;
        uint4 w[kCh];
#pragma unroll
        for (int x = 0; x < kCh; ++x) {
            w[x] = make_uint4(0, 0, 0, 0);
            if (row < job.rows) w[x] = *reinterpret_cast<const uint4*>(base + tok * a.qs + h * D);
            row += kStep;
            h += kStep;
            while (h >= a.G) {
                h -= a.G;
                ++tok;
            }
        }
#pragma unroll
        for (int x = 0; x < kCh; ++x)
            *reinterpret_cast<uint4*>(sm + Y::kOffQ + tile * Y::kTile + tile_off(rr0 + x * kStep, ch)) = w[x];
        fence_async_shared();
    }
    const int r = (warp & 3) * 32 + lane;  // softmax: the thread's row of the tile (and TMEM lane)
    const int row = job.row0 + tile * kRows + r;
    const int tok = row / a.G, h = row - tok * a.G;
    const bool valid = row < job.rows;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto stopped = [&]() { return *stop_flag != 0; };
    auto give_up = [&]() {
        atomicOr(a.status, PKV_STATUS_COPY_TIMEOUT);
        *stop_flag = 1;
    };
    if (tile == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == kWarpLoad && lane == 0) {
            int it = early;
            for (; it < 2 * n && !stopped(); ++it) {
                if (!wait_bar(bar(Y::kFree + slot(it)), phase(it - Y::kStages))) {
                    give_up();
                    break;
                }
                load_item(it);
            }
            // stopping early: the copies in flight land (bounded) before the
            // shared memory is given up
            if (stopped())
                for (int x = max(it - Y::kStages, 0); x < it; ++x) wait_bar(bar(Y::kFull + slot(x)), phase(x));
        } else if (warp == kWarpMma && n > 0) {
            // The whole warp walks the loop, one elected lane issues: what the
            // MMAs take is then warp-uniform (base descriptors plus constants),
            // and an MMA of K 16 costs its 64 cycles; issued from a lane of a
            // divergent branch it cost ~110 (8,192 tokens: 490 us).
            constexpr uint32_t id_s = instr_desc<T>(kKeys, false), id_o = instr_desc<T>(D, true);
            constexpr uint32_t kTile16 = Y::kTile >> 4;  // descriptor units
            const bool el = elect();
            const uint64_t dq = smem_desc(sbase + Y::kOffQ, 16384, 1024);
            const uint64_t dr = smem_desc(sbase + Y::kOffRing, 16384, 1024);
            auto issue_s = [&](int i, int s) {
                const uint64_t qa = dq + i * kTile16, kb = dr + s * kTile16;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        constexpr uint32_t kHalf16 = (kRows * 128) >> 4;
                        const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
                        mma_ss(tmem + i * kKeys, qa + off, kb + off, id_s, kk > 0);
                    }
                    mma_commit(bar(Y::kS + i));
                }
            };
            // keys 16 k0 .. 16 k1 - 1
            auto issue_o = [&](int i, int s, int k0, int k1, bool acc) {
                const uint64_t vb = dr + s * kTile16;
                if (el) {
#pragma unroll
                    for (int kk = k0; kk < k1; ++kk)
                        mma_ts(tmem + 2 * kKeys + i * kKeys, tmem + i * kKeys + kk * 8, vb + kk * 128, id_o,
                               acc || kk > 0);
                }
            };
            auto next = [&](int& s, uint32_t& ph) {
                if (++s == Y::kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            };
            int s = 0;  // ring slot and its phase, walking K0 V0 K1 V1 ..
            uint32_t ph = 0;
            bool ok = wait_bar(bar(Y::kFull), 0);
            if (ok) {
                fence_after_sync();
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (cnt[i] > 0) issue_s(i, 0);
                if (el) mma_commit(bar(Y::kFree));
            }
            next(s, ph);
            for (int jj = 0; ok && jj < n; ++jj) {
                const int sv = s;  // V(jj), then K(jj + 1)
                ok = !stopped() && wait_bar(bar(Y::kFull + sv), ph);
                next(s, ph);
                bool have_k = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!ok || jj >= cnt[i]) continue;
                    ok = wait_bar(bar(Y::kP + i), jj & 1);
                    if (!ok) continue;
                    fence_after_sync();
                    issue_o(i, sv, 0, kFirst / 16, jj > 0);
                    ok = wait_bar(bar(Y::kP + 2 + i), jj & 1);
                    if (!ok) continue;
                    fence_after_sync();
                    issue_o(i, sv, kFirst / 16, kKeys / 16, true);
                    if (jj + 1 < cnt[i]) {
                        if (!have_k) ok = wait_bar(bar(Y::kFull + s), ph);
                        have_k = ok;
                        if (ok) {
                            fence_after_sync();
                            issue_s(i, s);
                        }
                    } else if (el) {
                        mma_commit(bar(Y::kO + i));
                    }
                }
                if (!ok) break;
                if (el) {
                    mma_commit(bar(Y::kFree + sv));
                    if (jj + 1 < n) mma_commit(bar(Y::kFree + s));
                }
                next(s, ph);
            }
            if (!ok && lane == 0) give_up();
            // every MMA and every arrival of theirs is done (bounded) before
            // the CTA gives up its shared memory and TMEM
            if (el) mma_commit(bar(Y::kDrain));
            wait_bar(bar(Y::kDrain), 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + tile * kKeys + lanes, tO = tmem + 2 * kKeys + tile * kKeys + lanes;
        // positions: rows past the sequence's last take its position (their
        // query is zero, their output not written)
        const int my_pos = job.first_pos + min(tok, job.L - 1);
        const int warp_pos = __shfl_sync(0xffffffffu, my_pos, 0);  // the warp's first
        const int cta_pos = job.first_pos + job.row0 / a.G;        // the CTA's first
        const bool pos_scale = a.scale_log2 > 0.f;
        const float mul = pos_scale ? a.scale_log2 : 1.f;
        const int my_cnt = cnt[tile];
        float m = neg_inf(), l = 0.f;
        bool ok = true;
        for (int jj = 0; jj < my_cnt; ++jj) {
            const int key0 = (js + jj) * kKeys;
            ok = !stopped() && wait_bar(bar(Y::kS + tile), jj & 1);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            fence_after_sync();
            float x[kKeys];
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + cc * 32, x + cc * 32);
            tmem_wait_ld();
            // with a positive scale the maximum is taken over raw scores and
            // the scale enters the exponent's FMA
            if (!pos_scale) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i) x[i] *= a.scale_log2;
            }
            if (key0 + kKeys - 1 > warp_pos) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i)
                    if (key0 + i > my_pos) x[i] = neg_inf();
            }
            float mq[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i + 7 < kKeys; i += 8) {
#pragma unroll
                for (int c = 0; c < 4; ++c) mq[c] = max3f(mq[c], x[i + c], x[i + 4 + c]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) mq[c] = fmaxf(mq[c], x[kKeys - 4 + c]);
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
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= alpha;
                    tmem_st32(tO + cc * 32, reinterpret_cast<const uint32_t*>(o));
                }
            }
            // a tile with keys that some row must not see: its V rows may hold
            // anything there; tile 0 looks, tile 1 once tile 0 is done
            if (key0 + kKeys - 1 > cta_pos && (tile == 0 || jj >= cnt[0])) {
                const int it = 2 * jj + 1;
                ok = wait_bar(bar(Y::kFull + slot(it)), phase(it));
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                uint8_t* vt = sm + Y::kOffRing + slot(it) * Y::kTile + (warp & 3) * 32 * 128;  // the warp's 32 rows
                typename Pair<T>::type acc[4];
                const uint32_t zero = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = *reinterpret_cast<const typename Pair<T>::type*>(&zero);
                auto at = [&](int c) {
                    return reinterpret_cast<uint4*>(vt + (c / 8) * (kRows * 128) + (c % 8) * 512 + lane * 16);
                };
#pragma unroll
                for (int c = 0; c < kCh; ++c) probe<T>(acc, *at(c));
                bool odd = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = make_float2(Half16<T>::to_float(acc[i].x), Half16<T>::to_float(acc[i].y));
                    odd |= f.x != f.x || f.y != f.y;
                }
                if (__any_sync(0xffffffffu, odd)) {
                    if (lane == 0) *odd_flag = 1;
                    constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
                    for (int c = 0; c < kCh; ++c) {
                        uint16_t* e = reinterpret_cast<uint16_t*>(at(c));
                        for (int i = 0; i < 8; ++i)
                            if ((e[i] & kExp) == kExp) e[i] = 0;
                    }
                    fence_async_shared();
                }
            }
            // P in steps of 32 keys; the first kFirst are handed over early
            const float mref = m == neg_inf() ? 0.f : m;
            const float2 mul2 = make_float2(mul, mul), ref2 = make_float2(-mref, -mref);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int cc = 0; cc < kKeys / 32; ++cc) {
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 e = fma2(make_float2(x[cc * 32 + 2 * i], x[cc * 32 + 2 * i + 1]), mul2, ref2);
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
                    if (lane == 0) mbar_arrive(bar(Y::kP + (cc + 1 == kKeys / 32 ? 2 : 0) + tile));
                }
            }
            const float2 s2 = add2(sum[0], sum[1]);
            l += s2.x + s2.y;
        }
        if (ok && my_cnt > 0) {
            ok = wait_bar(bar(Y::kO + tile), 0);
            fence_after_sync();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) give_up();
        // ---- epilogue.  Non-finite V values that were taken out come back for
        // the rows that see them (their weight is positive).
        const bool odd = my_cnt > 0 && *odd_flag != 0;
        const int odd0 = max((cta_pos + 1) / kKeys, js) * kKeys;
        auto put_back = [&](int d0, float (&o)[32]) {
            for (int t = max(odd0, 0); t <= my_pos && t < min(je * kKeys, job.S); ++t) {
                const T* vr = static_cast<const T*>(a.v) + (static_cast<int64_t>(job.k0) + t) * a.vs + kvh * D + d0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float f = Half16<T>::to_float(vr[i]);
                    if (!(fabsf(f) <= 3.4e38f)) o[i] += f;
                }
            }
        };
        const int64_t orow = (static_cast<int64_t>(job.q0) + tok) * a.hq + kvh * a.G + h;
        if (a.splits == 1) {
            // through the tile's Q (no longer read) so that rows go out in
            // whole 128-byte lines
            uint8_t* st = sm + Y::kOffQ + tile * Y::kTile + (warp & 3) * 32 * (D * 2);
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                if (my_cnt > 0) {
                    tmem_ld32(tO + cc * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (odd) put_back(cc * 32, o);
                if (l == 0.f) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 w;
                    w.x = Half16<T>::pack(o[8 * c] * inv, o[8 * c + 1] * inv);
                    w.y = Half16<T>::pack(o[8 * c + 2] * inv, o[8 * c + 3] * inv);
                    w.z = Half16<T>::pack(o[8 * c + 4] * inv, o[8 * c + 5] * inv);
                    w.w = Half16<T>::pack(o[8 * c + 6] * inv, o[8 * c + 7] * inv);
                    *reinterpret_cast<uint4*>(st + lane * (D * 2) + (((cc * 4 + c) ^ (lane & 7)) << 4)) = w;
                }
            }
            __syncwarp();
            constexpr int kStep = 32 / kCh;
            const int ch = lane % kCh;
            int rr = lane / kCh, orow_i = job.row0 + tile * kRows + (warp & 3) * 32 + rr;
            int t = orow_i / a.G, hh = orow_i - t * a.G;
            T* base = static_cast<T*>(a.out) + (static_cast<int64_t>(job.q0) * a.hq + kvh * a.G) * D + ch * 8;
#pragma unroll 4
            for (int x = 0; x < kCh; ++x) {
                const uint4 w = *reinterpret_cast<const uint4*>(st + rr * (D * 2) + ((ch ^ (rr & 7)) << 4));
                if (ok && orow_i < job.rows)
                    *reinterpret_cast<uint4*>(base + (static_cast<int64_t>(t) * a.hq + hh) * D) = w;
                rr += kStep;
                orow_i += kStep;
                hh += kStep;
                while (hh >= a.G) {
                    hh -= a.G;
                    ++t;
                }
            }
        } else {
            const int64_t prow = static_cast<int64_t>(split) * a.T * a.hq + orow;
            const bool put = valid && ok;
            if (put) *reinterpret_cast<float2*>(a.ws_ml + prow * 2) = make_float2(m, l);
            if (my_cnt > 0) {
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    float o[32];
                    tmem_ld32(tO + cc * 32, o);
                    tmem_wait_ld();
                    if (odd) put_back(cc * 32, o);
                    if (put) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<float4*>(a.ws_o + prow * D + cc * 32 + 4 * c) =
                                make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    }
                }
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Merge of the splits: out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
// One CTA per slot and KV head, a warp per row at a time.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) prompt_merge_kernel(const __grid_constant__ PromptArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int u = blockIdx.x / a.hkv, kvh = blockIdx.x % a.hkv;
    Job job;
    const bool any = find_job(a.q_start, a.kv_start, a.batch, a.T, a.S, a.G, u, job);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!any) return;
    const int end = min(job.row0 + kCtaRows, job.rows);
    for (int row = job.row0 + (threadIdx.x >> 5); row < end; row += kMergeWarps) {
        const int tok = row / a.G, h = row - tok * a.G;
        const int64_t orow = (static_cast<int64_t>(job.q0) + tok) * a.hq + kvh * a.G + h;
        const int64_t step = static_cast<int64_t>(a.T) * a.hq;
        float ms = neg_inf(), ls = 0.f;
        if (lane < a.splits) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.ws_ml + (lane * step + orow) * 2));
            ms = ml.x;
            ls = ml.y;
        }
        float M = ms;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float wt = ms == neg_inf() ? (ls == 0.f ? 0.f : ls) : ex2(ms - M);
        float Ls = ms == neg_inf() && ls == 0.f ? 0.f : wt * ls;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, off);
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int s = 0; s < a.splits; ++s) {
            const float w = __shfl_sync(0xffffffffu, wt, s);
            if (w == 0.f) continue;
            const float* p = a.ws_o + (s * step + orow) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += w * __ldcg(p + e);
        }
        const float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) w[e] = Half16<T>::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
        T* dst = static_cast<T*>(a.out) + orow * D + lane * E;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
}

// ---------------------------------------------------------------- host
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static std::once_flag once;
    static EncodeTiled fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
    });
    return fn;
}

// Rows [S, Hkv, D] (row stride in elements) as a 4-D tensor (64 dims; rows;
// halves of 64 dims; KV heads); a box is 128 rows of one head, landing as
// [half][row][64 dims] with 128-byte swizzle.
bool rows_map(CUtensorMap* map, const void* base, int64_t rows, int hkv, int D, int64_t stride, bool bf16) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(D / 64),
                                static_cast<cuuint64_t>(hkv)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride) * 2, 128, static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t box[4] = {64, kKeys, static_cast<cuuint32_t>(D / 64), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Slots of 256 rows (see Job).
int64_t num_slots(int64_t batch, int64_t T, int64_t G) { return T * G / kCtaRows + batch; }

// Splits of the key axis: 1 unless the slots leave SMs idle; then as many as
// fill them, each at least kMinTiles tiles of the average sequence long.
constexpr int kMaxSplits = 32;  // the merge holds one per lane
constexpr int kMinTiles = 4;
int num_splits(int64_t batch, int64_t T, int64_t S, int64_t hkv, int64_t G) {
    if (batch == 0 || T == 0) return 1;
    const int64_t ctas = num_slots(batch, T, G) * hkv;
    const int64_t tiles = (S / batch + kKeys - 1) / kKeys;
    int64_t n = num_sms() / ctas;
    if (n > tiles / kMinTiles) n = tiles / kMinTiles;
    if (n > kMaxSplits) n = kMaxSplits;
    return n < 1 ? 1 : static_cast<int>(n);
}

// Sets the kernel's shared memory limit once per device and checks that it
// was built with the registers its warpgroups' split needs.
template <auto kernel>
int prepare_kernel(int bytes) {
    static std::atomic<int> state[64];  // 0: not yet, 1: ready, 2: too few registers
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
    int s = state[dev].load(std::memory_order_acquire);
    if (s == 0) {
        cudaFuncAttributes fa;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
            cudaFuncGetAttributes(&fa, kernel) != cudaSuccess)
            return PKV_ERR_CUDA;
        s = fa.numRegs >= kLaunchRegs ? 1 : 2;
        state[dev].store(s, std::memory_order_release);
    }
    return s == 1 ? PKV_OK : PKV_ERR_UNSUPPORTED;
}

template <typename T, int D>
int launch_prompt(const CUtensorMap& km, const CUtensorMap& vm, const PromptArgs& a, cudaStream_t st) {
    const int rc = prepare_kernel<prompt_tc_kernel<T, D>>(Layout<D>::kBytes);
    if (rc != PKV_OK) return rc;
    const int64_t slots = num_slots(a.batch, a.T, a.G);
    const unsigned ctas = static_cast<unsigned>(slots * a.hkv);
    prompt_tc_kernel<T, D><<<ctas * a.splits, kThreads, Layout<D>::kBytes, st>>>(km, vm, a);
    if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
    if (a.splits == 1) return PKV_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prompt_merge_kernel<T, D>, a) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_prompt_attention_workspace_bytes(int32_t batch, int32_t num_tokens, int32_t num_kv_tokens,
                                                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                    size_t* out) {
    if (!out || batch < 0 || num_tokens < 0 || num_kv_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || num_q_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    const int n = pkv::num_splits(batch, num_tokens, num_kv_tokens, num_kv_heads, num_q_heads / num_kv_heads);
    *out = n == 1 ? 0
                  : static_cast<size_t>(n) * num_tokens * num_q_heads * (static_cast<size_t>(head_dim) + 2) *
                        sizeof(float);
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
    const int64_t G = num_q_heads / num_kv_heads;
    const int64_t dq = static_cast<int64_t>(num_q_heads) * head_dim, dk = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (q_stride < dq || k_stride < dk || v_stride < dk) return PKV_ERR_INVALID_ARG;
    // TMA strides are below 2^40 bytes; rows and CTAs are counted in 31 bits
    if ((head_dim != 64 && head_dim != 128) || G > 128 || k_stride >= (1LL << 38) || v_stride >= (1LL << 38) ||
        num_tokens * G > INT32_MAX - pkv::kCtaRows ||
        pkv::num_slots(batch, num_tokens, G) * num_kv_heads * pkv::kMaxSplits > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !q_start || !out || (num_kv_tokens > 0 && (!k || !v))) return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(q) || !pkv::aligned16(k) || !pkv::aligned16(v) || !pkv::aligned16(out) || q_stride % 8 != 0 ||
        k_stride % 8 != 0 || v_stride % 8 != 0 || (reinterpret_cast<uintptr_t>(q_start) & 3u) ||
        (reinterpret_cast<uintptr_t>(kv_start) & 3u))
        return PKV_ERR_MISALIGNED;
    pkv::PromptArgs a;
    a.splits = workspace ? pkv::num_splits(batch, num_tokens, num_kv_tokens, num_kv_heads, G) : 1;
    if (a.splits > 1) {
        const size_t rows = static_cast<size_t>(a.splits) * num_tokens * num_q_heads;
        if (workspace_bytes < rows * (head_dim + 2) * sizeof(float)) return PKV_ERR_WORKSPACE;
        if (!pkv::aligned16(workspace)) return PKV_ERR_MISALIGNED;
        a.ws_o = static_cast<float*>(workspace);
        a.ws_ml = a.ws_o + rows * head_dim;
    } else {
        a.ws_o = a.ws_ml = nullptr;
    }
    int* st = pkv::status_word();
    if (!st) return PKV_ERR_CUDA;
    const bool bf16 = dtype == PKV_DTYPE_BF16;
    // without K/V rows no tile is loaded; the maps still need an address
    const int64_t rows = num_kv_tokens > 0 ? num_kv_tokens : 1;
    CUtensorMap km, vm;
    if (!pkv::rows_map(&km, num_kv_tokens > 0 ? k : q, rows, num_kv_heads, head_dim, k_stride, bf16) ||
        !pkv::rows_map(&vm, num_kv_tokens > 0 ? v : q, rows, num_kv_heads, head_dim, v_stride, bf16))
        return PKV_ERR_CUDA;
    a.q = q;
    a.v = v;
    a.q_start = q_start;
    a.kv_start = kv_start ? kv_start : q_start;
    a.batch = batch;
    a.T = num_tokens;
    a.S = num_kv_tokens;
    a.hq = num_q_heads;
    a.hkv = num_kv_heads;
    a.G = static_cast<int>(G);
    a.qs = q_stride;
    a.vs = v_stride;
    a.scale_log2 = scale * pkv::kLog2e;
    a.out = out;
    a.status = st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (bf16)
        return head_dim == 128 ? pkv::launch_prompt<__nv_bfloat16, 128>(km, vm, a, cs)
                               : pkv::launch_prompt<__nv_bfloat16, 64>(km, vm, a, cs);
    return head_dim == 128 ? pkv::launch_prompt<__half, 128>(km, vm, a, cs)
                           : pkv::launch_prompt<__half, 64>(km, vm, a, cs);
}
