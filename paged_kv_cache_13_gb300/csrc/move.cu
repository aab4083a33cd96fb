// Row moves: the device side of a compaction (pkv_seq_compact).  For every
// pool, KV head and move i, the row at slot dst_i becomes a byte copy of the
// row at slot src_i.
//
// Bytes: 2 x moves x Hkv x row bytes per pool, plus 16 bytes of slots a move;
// no arithmetic.  HBM-bound once the rows exceed L2 (2.37 GB of 256-byte rows:
// 361 us, 6,576 GB/s), latency-bound (slot load, row load, row store, one after
// the other) for a single short sequence (16.8 MB: 4.5 us), and bound by the
// moves themselves for 2-byte scale rows beside 128-byte codes (45 us, 3,069
// GB/s).
//
// Layout: a CTA takes kMoves moves of one pool, translates their slots once
// into row offsets in shared memory (checked there), and copies their rows for
// its KV heads, head by head.  Within a head consecutive threads take the
// 16-byte vectors of a row, then the next move's row: the destinations of a
// compaction are consecutive rows, so a warp's stores are one contiguous run
// and its loads whole rows.  Each thread has kUnroll loads in flight.
// Sources and destinations are disjoint, so CTAs need no order.

#include "common.cuh"

namespace pkv {
namespace {

constexpr int kMoves = 64;      // moves per CTA
constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // vectors a thread has in flight
constexpr int kMaxPools = 256;
constexpr int64_t kMaxRow = 65536;  // bytes per row (the index arithmetic below)

struct MoveArgs {
    void* pool[kMaxPools];
    int32_t row[kMaxPools];  // bytes per row
};

// Quotient by a divisor d >= 2 through its reciprocal m = ceil(2^32 / d):
// exact while x (m d - 2^32) < 2^32, and m d - 2^32 < d.
__device__ __forceinline__ uint32_t div_by(uint32_t x, uint32_t m) { return __umulhi(x, m); }

// Copies the rows of n moves for heads [h0, h1).  V: the vector type, the
// widest whose size divides the row.  soff, doff: row index of head 0.
template <typename V>
__device__ __forceinline__ void copy_rows(void* pool, int row, const int64_t* soff, const int64_t* doff, int n,
                                          int h0, int h1, int bs) {
    V* base = static_cast<V*>(pool);
    const uint32_t cpr = static_cast<uint32_t>(row) / sizeof(V);  // vectors per row
    const uint32_t per_head = cpr * kMoves;
    // rows of fewer vectors than fill a CTA: several heads in one sweep
    const uint32_t heads = per_head >= kThreads ? 1u : kThreads / per_head;
    const uint32_t mc = cpr > 1 ? 0xffffffffu / cpr + 1 : 0, mh = 0xffffffffu / per_head + 1;
    for (int h = h0; h < h1; h += heads) {
        const uint32_t items = per_head * min(heads, static_cast<uint32_t>(h1 - h));
        for (uint32_t x0 = threadIdx.x; x0 < items; x0 += kThreads * kUnroll) {
            V v[kUnroll];
            int64_t d[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const uint32_t x = x0 + u * kThreads;
                d[u] = -1;
                if (x < items) {
                    const uint32_t hh = heads > 1 ? div_by(x, mh) : 0;
                    const uint32_t r = x - hh * per_head;
                    const uint32_t m = cpr > 1 ? div_by(r, mc) : r;
                    const uint32_t c = r - m * cpr;
                    if (static_cast<int>(m) < n && soff[m] >= 0) {
                        const int64_t head = static_cast<int64_t>(h + hh) * bs;
                        v[u] = base[(soff[m] + head) * cpr + c];
                        d[u] = (doff[m] + head) * cpr + c;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (d[u] >= 0) base[d[u]] = v[u];
        }
    }
}

__global__ void __launch_bounds__(kThreads)
    move_rows_kernel(const __grid_constant__ MoveArgs a, const int64_t* __restrict__ src,
                     const int64_t* __restrict__ dst, int n_moves, int num_blocks, int hkv, int bs,
                     int heads_per_cta, int* __restrict__ status) {
    __shared__ int64_t soff[kMoves], doff[kMoves];
    const int m0 = blockIdx.x * kMoves;
    const int n = min(kMoves, n_moves - m0);
    if (threadIdx.x < n) {
        const int64_t s = src[m0 + threadIdx.x], d = dst[m0 + threadIdx.x];
        const int64_t slots = static_cast<int64_t>(num_blocks) * bs;
        int64_t so = -1, dd = -1;
        if (s >= slots || d >= slots) {
            atomicOr(status, PKV_STATUS_BAD_SLOT);
        } else if (s >= 0 && d >= 0) {
            so = (s / bs) * hkv * bs + s % bs;
            dd = (d / bs) * hkv * bs + d % bs;
        }
        soff[threadIdx.x] = so;
        doff[threadIdx.x] = dd;
    }
    __syncthreads();
    const int p = blockIdx.y;
    const int h0 = blockIdx.z * heads_per_cta, h1 = min(h0 + heads_per_cta, hkv);
    const int row = a.row[p];
    if (row % 16 == 0) copy_rows<uint4>(a.pool[p], row, soff, doff, n, h0, h1, bs);
    else if (row % 8 == 0) copy_rows<uint2>(a.pool[p], row, soff, doff, n, h0, h1, bs);
    else if (row % 4 == 0) copy_rows<uint32_t>(a.pool[p], row, soff, doff, n, h0, h1, bs);
    else copy_rows<uint16_t>(a.pool[p], row, soff, doff, n, h0, h1, bs);
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_move_rows(void* const* pools, const int64_t* bytes_per_row, int32_t n_pools,
                             const int64_t* src_slots, const int64_t* dst_slots, int32_t n_moves,
                             int32_t num_blocks, int32_t num_kv_heads, int32_t block_size, void* stream) {
    if (n_moves < 0 || n_pools < 1 || n_pools > pkv::kMaxPools || num_blocks <= 0 || num_kv_heads <= 0 ||
        block_size <= 0 || !pools || !bytes_per_row)
        return PKV_ERR_INVALID_ARG;
    if (num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    pkv::MoveArgs a = {};
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i] || bytes_per_row[i] <= 0 || bytes_per_row[i] % 2 != 0) return PKV_ERR_INVALID_ARG;
        if (bytes_per_row[i] > pkv::kMaxRow) return PKV_ERR_UNSUPPORTED;
        if (!pkv::aligned16(pools[i])) return PKV_ERR_MISALIGNED;
        a.pool[i] = pools[i];
        a.row[i] = static_cast<int32_t>(bytes_per_row[i]);
    }
    if (n_moves == 0) return PKV_OK;
    if (!src_slots || !dst_slots) return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(src_slots) & 7u) || (reinterpret_cast<uintptr_t>(dst_slots) & 7u))
        return PKV_ERR_MISALIGNED;
    int* st = pkv::status_word();
    if (!st) return PKV_ERR_CUDA;
    const int heads = 1;
    const dim3 grid((n_moves + pkv::kMoves - 1) / pkv::kMoves, n_pools, (num_kv_heads + heads - 1) / heads);
    pkv::move_rows_kernel<<<grid, pkv::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        a, src_slots, dst_slots, n_moves, num_blocks, num_kv_heads, block_size, heads, st);
    return pkv::launch_status();
}
