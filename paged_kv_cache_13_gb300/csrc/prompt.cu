// Attention of packed prompts over their own (unpaged) K/V rows:
// pkv_prompt_attention.
//
// What it computes: query row i of sequence b sits at position p = S_b - L_b
// + i of its S_b K/V rows, and
//   out[q_start[b] + i, h] = sum_{t <= p} softmax_t(scale <q, k_t>) v_t
// over KV head h / G ("The 8GB VRAM Breakthrough", §5: the prefill that
// precedes the decode loop).
//
// The tensor-core attention of attend_tc.cuh with K/V tiles copied by TMA, one
// box per tile.  Long K/V axes with few rows are gridded over splits of the
// key tiles too, fp32 partials (m, l, o) merged by a second kernel.
// Measured (32 query heads over 8, D 128, bf16): 8,192 tokens 354 us (1,550
// TFLOP/s), twelve prompts of 1 to 2,047 tokens 84 us; D 64, 578 rows behind
// 9,501 keys 66 us.  Bound by the chain of a tile (attend_tc.cuh); what a job
// adds is its masked tile and its output rows, ~4 us for 256 rows.

#include <cuda.h>
#include <math.h>

#include <mutex>

#include "attend_tc.cuh"
#include "balanced.cuh"

namespace pkv {
namespace {

using namespace tcattn;

constexpr int kThreads = 384;  // warps 0-3, 4-7: softmax of tiles 0, 1; 8: copies; 9: MMAs; 10, 11: V's non-finite values
constexpr int kWarpLoad = 8, kWarpMma = 9;
// Registers: launched at 168 a thread; the softmax warpgroups take 208 (128
// live scores), the third gives its own back down to 88.
constexpr int kLaunchRegs = 168;
static_assert(2 * 128 * 208 + 128 * 88 <= kThreads * kLaunchRegs, "register split exceeds the launch's registers");
// Ring items of a job still to be loaded when the next job is asked for: later,
// and the ring runs empty; earlier, and a CTA holds a job that another could
// have begun.
constexpr int kAhead = 8;

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

// The rows of one CTA.  The grid has num_slots = floor(T G / 256) + batch slots
// of 256 rows, counted from the last down: a sequence's later rows see more
// keys.  Up to 31 sequences each has exactly its tiles' slots, and those left
// over come last; of more, sequence b's start at off(b) = floor(q_start[b] G /
// 256) + b: off(b + 1) - off(b) is at least its tiles.
struct Job {
    int b, q0, L, k0, S, first_pos;
    int row0, rows;  // first row in the sequence, rows of the sequence (see Work)
};

// The y-th slot from the last.  Warp-collective; false when it has no rows.
__device__ __forceinline__ bool find_job(const int32_t* q_start, const int32_t* kv_start, int batch, int T, int S, int G,
                                         int y, Job& job) {
    const int lane = threadIdx.x & 31;
    auto start = [&](int b) { return min(max(q_start[b], 0), T); };
    int lo = 0;
    int qa, qe, ka, ke;
    int64_t row0;
    if (batch < 32) {  // every start in one round of loads
        const int qv = lane <= batch ? start(lane) : 0, kv = lane <= batch ? min(max(kv_start[lane], 0), S) : 0;
        const int qn = __shfl_down_sync(0xffffffffu, qv, 1);
        const int tiles = lane < batch && qn > qv
                              ? static_cast<int>((static_cast<int64_t>(qn - qv) * G + kCtaRows - 1) / kCtaRows)
                              : 0;
        int sum = tiles;  // of sequences 0 .. lane
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += x;
        }
        const int u = __shfl_sync(0xffffffffu, sum, 31) - 1 - y;
        if (u < 0) return false;
        lo = __popc(__ballot_sync(0xffffffffu, sum <= u));
        qa = __shfl_sync(0xffffffffu, qv, lo);
        qe = __shfl_sync(0xffffffffu, qv, lo + 1);
        ka = __shfl_sync(0xffffffffu, kv, lo);
        ke = __shfl_sync(0xffffffffu, kv, lo + 1);
        row0 = static_cast<int64_t>(u - __shfl_sync(0xffffffffu, sum - tiles, lo)) * kCtaRows;
    } else {
        const int64_t u = static_cast<int64_t>(T) * G / kCtaRows + batch - 1 - y;
        for (int n = batch;;) {
            const int step = (n + 31) / 32;
            const int b = lo + lane * step;
            const bool le = lane * step < n && static_cast<int64_t>(start(b)) * G / kCtaRows + b <= u;
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
        row0 = (u - (static_cast<int64_t>(qa) * G / kCtaRows + lo)) * kCtaRows;
    }
    job.b = lo;
    job.q0 = qa;
    job.L = qe - qa;
    job.k0 = ka;
    job.S = max(ke - ka, 0);
    if (job.L <= 0 || row0 < 0 || row0 >= static_cast<int64_t>(job.L) * G) return false;  // < 0: starts out of order
    job.row0 = static_cast<int>(row0);
    job.rows = job.L * G;
    job.first_pos = job.S - job.L;
    return true;
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

// Takes the non-finite values out of 64 rows of a V tile (a warp; any order
// will do, so the swizzle does not matter); true when there were any.
template <typename T, int D>
__device__ __forceinline__ bool clean_rows(uint8_t* p) {
    const int lane = threadIdx.x & 31;
    constexpr int kPer = kRows / 2 * 128 / 512;  // 512-byte pieces of a 64-column half
    auto piece = [&](int c) { return reinterpret_cast<uint4*>(p + c / kPer * (kRows * 128) + c % kPer * 512 + lane * 16); };
    typename Pair<T>::type acc[4];
    const uint32_t zero = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = *reinterpret_cast<const typename Pair<T>::type*>(&zero);
#pragma unroll 8
    for (int c = 0; c < D / 64 * kPer; ++c) probe<T>(acc, *piece(c));
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = make_float2(Half16<T>::to_float(acc[i].x), Half16<T>::to_float(acc[i].y));
        odd |= f.x != f.x || f.y != f.y;
    }
    if (!__any_sync(0xffffffffu, odd)) return false;
    constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
#pragma unroll 1
    for (int c = 0; c < D / 64 * kPer; ++c) {
        uint16_t* e = reinterpret_cast<uint16_t*>(piece(c));
        for (int i = 0; i < 8; ++i)
            if ((e[i] & kExp) == kExp) e[i] = 0;
    }
    fence_async_shared();
    return true;
}

// A job as the loading warp hands it to the others.
struct QueuedJob {
    int some;  // 0: no job is left
    int kvh, split;
    Job job;
    Work w;
};
static_assert(sizeof(QueuedJob) <= Layout<64, true>::kJobBytes, "queue entry");

// Asks for a CTA of the grid that has not started, to do its work in its
// place; the answer (16 bytes) lands at dst.  Not to be called again once it
// was no.
__device__ __forceinline__ void claim_cta(uint32_t dst, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}
// The claimed CTA's blockIdx.x, or -1.
__device__ __forceinline__ int claimed_cta(uint32_t src) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "mov.u32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=r"(x)
        : "r"(src)
        : "memory");
    return x;
}

// One CTA per (slot, KV head, split) is launched; those that fit run, and take
// over the work of the rest one by one.  A CTA's start, TMEM and first Q, K and
// V are then paid once, and between jobs the next one's K and V are already in
// the ring and its Q in registers when the last product of the one before is
// done (304 sequences of 64 rows: 177 us as a CTA per job, 119 us).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ PromptArgs a) {
    using Y = Layout<D, true>;
    constexpr int kCh = D / 8;  // 16-byte chunks per row
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Smem<D, true> sm(smem_raw);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tile = warp >> 2;  // softmax: 0 or 1
    auto find = [&](int x, QueuedJob& j) {  // CTA x's job
        const int per_slot = a.hkv * a.splits;
        j.kvh = x % per_slot / a.splits;
        j.split = x % a.splits;
        return find_job(a.q_start, a.kv_start, a.batch, a.T, a.S, a.G, x / per_slot, j.job);
    };
    auto entry = [&](int n) { return reinterpret_cast<QueuedJob*>(sm.p + Y::kOffJobs + n % Y::kQueue * Y::kJobBytes); };
    // job n (whole warp); false when there is none, or the wait ran out
    auto next_job = [&](int n) {
        const bool ok = __all_sync(0xffffffffu, wait_bar(sm.bar(Y::kJob + n % Y::kQueue), n / Y::kQueue & 1));
        if (!ok && lane == 0) sm.give_up(a.status);
        return ok && entry(n)->some != 0;
    };
    auto done_with = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.bar(Y::kJobDone + n % Y::kQueue));
    };
    // a softmax warp's 32 query rows, whole 128-byte lines at a time: lane l
    // takes chunk l % kCh of rows l / kCh, l / kCh + kStep, ..
    constexpr int kStep = 32 / kCh, kLoads = 32 / kStep;
    auto load_q = [&](const Job& job, int kvh, uint4 (&v)[kLoads]) {
        int row = job.row0 + tile * kRows + (warp & 3) * 32 + lane / kCh;
        int tok = row / a.G, h = row - tok * a.G;
        const T* base = static_cast<const T*>(a.q) + static_cast<int64_t>(job.q0) * a.qs + kvh * a.G * D + lane % kCh * 8;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            v[x] = make_uint4(0, 0, 0, 0);
            if (row < job.rows) v[x] = *reinterpret_cast<const uint4*>(base + tok * a.qs + h * D);
            row += kStep;
            h += kStep;
            while (h >= a.G) {
                h -= a.G;
                ++tok;
            }
        }
    };
    auto put_q = [&](const uint4 (&v)[kLoads]) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x)
            *reinterpret_cast<uint4*>(sm.p + Y::kOffQ + tile * Y::kTile +
                                      tile_off((warp & 3) * 32 + lane / kCh + x * kStep, lane % kCh)) = v[x];
        fence_async_shared();
    };
    auto q_written = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.bar(Y::kQ + tile));
    };

    // ---- the loading warp: jobs and their K and V
    int cta = blockIdx.x;  // the CTA whose job is next; -1: none
    QueuedJob job = {};
    Before before;
    int n = 0;  // jobs handed out
    bool asked = false, unchecked = cta == 0;
    uint32_t asked_phase = 0;
    auto load_item = [&](const QueuedJob& job, int i) {
        const int it = before.items + i;
        const uint32_t full = sm.bar(Y::kFull + sm.slot(it));
        mbar_arrive_expect_tx(full, Y::kTile);
        tma_load(sm.base + Y::kOffRing + sm.slot(it) * Y::kTile, i & 1 ? &vmap : &kmap,
                 job.job.k0 + (job.w.js + i / 2) * kKeys, job.kvh, full);
    };
    auto ask = [&]() {
        if (asked) return;
        asked = true;
        if (lane == 0) {
            fence_async_shared();  // the last answer has been read
            mbar_arrive_expect_tx(sm.bar(Y::kClaim), 16);
            claim_cta(sm.base + Y::kOffClaim, sm.bar(Y::kClaim));
        }
        __syncwarp();
    };
    auto answer = [&]() {  // false when it did not come
        if (!__all_sync(0xffffffffu, wait_bar(sm.bar(Y::kClaim), asked_phase))) return false;
        asked = false;
        asked_phase ^= 1u;
        cta = claimed_cta(sm.base + Y::kOffClaim);
        unchecked |= cta == 0;
        __syncwarp();
        return true;
    };
    auto check = [&]() {  // the ranges, once per call
        if (!unchecked) return;
        unchecked = false;
        bool bad = false;
        for (int j = lane; j < a.batch; j += 32) {
            const int q0 = a.q_start[j], q1 = a.q_start[j + 1], k0 = a.kv_start[j], k1 = a.kv_start[j + 1];
            bad |= q0 < 0 || q1 < q0 || q1 > a.T || k0 < 0 || k1 < k0 || k1 > a.S || k1 - k0 < q1 - q0;
        }
        if (bad) atomicOr(a.status, PKV_STATUS_BAD_CONTEXT);
    };
    // CTA `cta`'s job (or the next that has rows) to the others as job n; false
    // when a wait ran out
    auto hand_out = [&](QueuedJob& job) {
        bool ok = true;
        while (cta >= 0 && !find(cta, job)) {
            if (a.batch < 32) {  // nor has any CTA behind it
                cta = -1;
                break;
            }
            ask();
            if (!answer()) return false;
        }
        if (n >= Y::kQueue)
            ok = __all_sync(0xffffffffu, wait_bar(sm.bar(Y::kJobDone + n % Y::kQueue), (n / Y::kQueue - 1) & 1));
        if (!ok) return false;
        job.some = cta >= 0;
        if (cta >= 0) {
            job.w.row0 = job.job.row0;
            job.w.rows = job.job.rows;
            job.w.G = a.G;
            job.w.first_pos = job.job.first_pos;
            job.w.set_tiles(job.split, a.splits);
        }
        if (lane == 0) {
            *entry(n) = job;
            *sm.odd(n) = 0;
            mbar_arrive(sm.bar(Y::kJob + n % Y::kQueue));
        }
        __syncwarp();
        return true;
    };

    bool first = false;  // softmax: the CTA's own job has rows of the tile's, its Q is in place
    int early = 0;
    if (warp == kWarpLoad) {
        if (lane == 0) sm.init(1, 11);
        __syncwarp();
        if (hand_out(job) && cta >= 0) {
            early = min(2 * job.w.n, Y::kStages);  // items the empty ring takes, on their way while Q is fetched
            if (lane == 0)
                for (int i = 0; i < early; ++i) load_item(job, i);
        }
    } else if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sh_addr(sm.tmem_slot())),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (tile < 2) {
        first = find(blockIdx.x, job);
        if (first) {
            uint4 v[kLoads];
            load_q(job.job, job.kvh, v);
            put_q(v);
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *sm.tmem_slot();

    if (tile == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kWarpLoad) {
            bool ok = true;
            bool some = cta >= 0;
            while (ok && some) {
                // the next job is asked for and handed out in time for its
                // first items to follow this one's last, behind what the ring
                // holds
                const int items = 2 * job.w.n, at = max(min(items, Y::kStages), items - kAhead);
                QueuedJob after = {};
                int i = early;
                early = 0;
                some = false;
                for (;; ++i) {
                    if (i == at) {
                        check();
                        ask();
                        ok = answer();
                        if (ok) {
                            ++n;
                            ok = hand_out(after);
                            some = cta >= 0;
                        }
                    }
                    if (!ok || i >= items) break;
                    const int it = before.items + i;
                    if (it >= Y::kStages)
                        ok = !__any_sync(0xffffffffu, sm.stopped()) &&
                             __all_sync(0xffffffffu, wait_bar(sm.bar(Y::kFree + sm.slot(it)), sm.phase(it - Y::kStages)));
                    if (!ok) break;
                    if (lane == 0) load_item(job, i);
                    __syncwarp();
                }
                before.items += i;
                job = after;
            }
            check();
            if (!ok && lane == 0) sm.give_up(a.status);
            // stopping early: the copies and the answer in flight land
            // (bounded) before the shared memory is given up
            if (!ok) {
                for (int x = max(before.items - Y::kStages, 0); x < before.items; ++x)
                    wait_bar(sm.bar(Y::kFull + sm.slot(x)), sm.phase(x));
                if (asked) wait_bar(sm.bar(Y::kClaim), asked_phase);
            }
        } else if (warp == kWarpMma) {
            bool ok = true;
            for (; ok && next_job(n); ++n) {
                const Work w = entry(n)->w;
                done_with(n);
                ok = mma_job<T>(sm, tmem, w, before);
                before.add(w);
            }
            mma_end(sm, ok, a.status);
        } else {
            // The V tiles of every job before their products.  A tile with keys
            // that some row must not see may hold anything there (0 x NaN would
            // reach that row): its non-finite values are taken out.  By warps of
            // their own, ahead of the products: in the softmax warps it cost 3 us
            // a job.  Each takes half of the rows.
            bool ok = true;
            for (; ok && next_job(n); ++n) {
                const Work w = entry(n)->w;
                for (int jj = 0; jj < w.n && ok; ++jj) {
                    const int it = before.items + 2 * jj + 1;
                    ok = !__any_sync(0xffffffffu, sm.stopped()) &&
                         __all_sync(0xffffffffu, wait_bar(sm.bar(Y::kFull + sm.slot(it)), sm.phase(it)));
                    if (!ok) break;
                    if (w.masked(jj) && clean_rows<T, D>(sm.ring(it) + (warp & 1) * (kRows / 2) * 128) && lane == 0)
                        *sm.odd(n) = 1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sm.bar(Y::kClean + sm.slot(it)));
                }
                before.items += 2 * w.n;
                done_with(n);
            }
            if (!ok && lane == 0) sm.give_up(a.status);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        bool some = next_job(0);
        if (some && entry(0)->w.count(tile) > 0) {
            if (!first) {
                uint4 v[kLoads];
                load_q(entry(0)->job, entry(0)->kvh, v);
                put_q(v);
            }
            q_written();
        }
        while (some) {
            const Work w = entry(n)->w;
            float m, l;
            bool ok = softmax_tile<T>(sm, tmem, w, before, tile, a.scale_log2, m, l);
            // the next job's Q: fetched while the last product is computed,
            // written when that has read this one's
            const bool more = ok && next_job(n + 1);
            const bool has_q = more && entry(n + 1)->w.count(tile) > 0;
            uint4 v[kLoads];  // set either way: else live all through the loop
#pragma unroll
            for (int i = 0; i < kLoads; ++i) v[i] = make_uint4(0, 0, 0, 0);
            if (has_q) load_q(entry(n + 1)->job, entry(n + 1)->kvh, v);
            ok = wait_o(sm, w, before, tile, ok, a.status);
            if (has_q) {
                put_q(v);
                q_written();
            }
            const QueuedJob job = *entry(n);
            // non-finite V values that were taken out come back for the rows
            // that see them (their weight is positive)
            const int row = w.row0 + tile * kRows + (warp & 3) * 32 + lane;
            const bool odd = w.count(tile) > 0 && *sm.odd(n) != 0;
            const int my_pos = w.first_pos + min(row, w.rows - 1) / a.G;
            auto put_back = [&](int d0, float (&o)[32]) {
                if (!odd) return;
                for (int t = w.masked_from(); t <= my_pos && t < min((w.js + w.n) * kKeys, job.job.S); ++t) {
                    const T* vr = static_cast<const T*>(a.v) + (static_cast<int64_t>(job.job.k0) + t) * a.vs + job.kvh * D + d0;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float f = Half16<T>::to_float(vr[i]);
                        if (!(fabsf(f) <= 3.4e38f)) o[i] += f;
                    }
                }
            };
            auto o_read = [&]() {
                if (w.count(tile) == 0) return;
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.bar(Y::kORead + tile));
            };
            const int64_t head0 = static_cast<int64_t>(job.job.q0) * a.hq + job.kvh * a.G;  // row (token 0, head 0) of the output
            if (a.splits == 1) {
                store_tile<T, D, false>(sm, tmem, w, tile, l, ok, static_cast<T*>(a.out) + head0 * D, a.hq, put_back, o_read);
            } else {
                const int tok = row / a.G;
                const int64_t prow = static_cast<int64_t>(job.split) * a.T * a.hq + head0 +
                                     static_cast<int64_t>(tok) * a.hq + (row - tok * a.G);
                store_partial<D, false>(tmem, w, tile, m, l, ok && row < w.rows, a.ws_o, a.ws_ml, prow, put_back);
                o_read();
            }
            done_with(n);
            if (!ok) break;
            before.add(w);
            some = more;
            ++n;
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Merge of the splits: one CTA per slot and KV head, a warp per row at a time.
constexpr int kMergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) prompt_merge_kernel(const __grid_constant__ PromptArgs a) {
    const int kvh = blockIdx.x % a.hkv;
    Job job;
    const bool any = find_job(a.q_start, a.kv_start, a.batch, a.T, a.S, a.G, blockIdx.x / a.hkv, job);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!any) return;
    const int end = min(job.row0 + kCtaRows, job.rows);
    for (int row = job.row0 + (threadIdx.x >> 5); row < end; row += kMergeWarps) {
        const int tok = row / a.G;
        const int64_t orow = (static_cast<int64_t>(job.q0) + tok) * a.hq + kvh * a.G + (row - tok * a.G);
        merge_row<T, D>(a.ws_o, a.ws_ml, a.splits, static_cast<int64_t>(a.T) * a.hq, orow,
                        static_cast<T*>(a.out) + orow * D);
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

int prompt_splits(int64_t batch, int64_t T, int64_t S, int64_t hkv, int64_t G) {
    if (batch == 0 || T == 0) return 1;
    return num_splits(num_slots(batch, T, G) * hkv, (S / batch + kKeys - 1) / kKeys, num_sms());
}

template <typename T, int D>
int launch_prompt(const CUtensorMap& km, const CUtensorMap& vm, const PromptArgs& a, cudaStream_t st) {
    const int rc = prepare_kernel<prompt_tc_kernel<T, D>>(Layout<D, true>::kBytes, kLaunchRegs);
    if (rc != PKV_OK) return rc;
    const int64_t slots = num_slots(a.batch, a.T, a.G);
    const unsigned ctas = static_cast<unsigned>(slots * a.hkv);
    prompt_tc_kernel<T, D><<<ctas * a.splits, kThreads, Layout<D, true>::kBytes, st>>>(km, vm, a);
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
    const int n = pkv::prompt_splits(batch, num_tokens, num_kv_tokens, num_kv_heads, num_q_heads / num_kv_heads);
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
        num_tokens * G > INT32_MAX - pkv::tcattn::kCtaRows ||
        pkv::num_slots(batch, num_tokens, G) * num_kv_heads * pkv::tcattn::kMaxSplits > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !q_start || !out || (num_kv_tokens > 0 && (!k || !v))) return PKV_ERR_INVALID_ARG;
    if (!pkv::aligned16(q) || !pkv::aligned16(k) || !pkv::aligned16(v) || !pkv::aligned16(out) || q_stride % 8 != 0 ||
        k_stride % 8 != 0 || v_stride % 8 != 0 || (reinterpret_cast<uintptr_t>(q_start) & 3u) ||
        (reinterpret_cast<uintptr_t>(kv_start) & 3u))
        return PKV_ERR_MISALIGNED;
    pkv::PromptArgs a;
    a.splits = workspace ? pkv::prompt_splits(batch, num_tokens, num_kv_tokens, num_kv_heads, G) : 1;
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
    a.scale_log2 = scale * pkv::tcattn::kLog2e;
    a.out = out;
    a.status = st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (bf16)
        return head_dim == 128 ? pkv::launch_prompt<__nv_bfloat16, 128>(km, vm, a, cs)
                               : pkv::launch_prompt<__nv_bfloat16, 64>(km, vm, a, cs);
    return head_dim == 128 ? pkv::launch_prompt<__half, 128>(km, vm, a, cs)
                           : pkv::launch_prompt<__half, 64>(km, vm, a, cs);
}
