// sorted_rows.cu -- the slots of a routed batch sorted by expert with their tokens' rows (coli_moe_sort_rows), the
// weighted sum of every token's expert rows (coli_moe_combine; without weights and addend the gradient of the sorted
// rows) and its gradient (coli_moe_combine_grad).
//
//   place[s] = #(slots of lower experts) + #(earlier slots of the same expert),  rows[place[t K + k]] = x[t]
//   out[t]   = add[t] + sum_k w[t][k] y[place[t K + k]]
//   dy[place[t K + k]] = w[t][k] dout[t],  dw[t][k] = sum_h dout[t][h] y[place[t K + k]][h]
//
// All three move rows and compute next to nothing: HBM bounds them (2048 tokens, 8 slots each of 6144 bf16 values: sorted in 42 us,
// 35 of them the copies at 6.4 TB/s; combined with a float32 addend in 49 us, 6.1 TB/s; 8192 tokens x 8 of 2048, the gradient in
// 98 us, 5.8 TB/s).  Every row is read once, by 16-byte pieces where
// its address allows it, else element by element; a token's rows are in flight together.  No atomics on data: the same
// call gives the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "pdl.h"
#include "sorted_rows.h"
#include "tc_ptx.h"

namespace coli {

namespace {

constexpr unsigned FULL = 0xffffffffu;

// ------------------------------------------------------------------ elements

// V elements of a row as they lie in memory, at a multiple of their bytes or of 16.  (No read-only loads: an addend may be the result
// itself.)  32 bytes go in two loads: one would want a multiple of 32, and is no faster (2048 tokens x 8 rows of 6144 with a float32
// addend 48 us either way, the gradient 82; at odd multiples of 16 bytes 48 and 82 too).
template <typename T, int V>
struct Raw {
    static constexpr int BYTES = sizeof(T) * V, WORDS = BYTES < 4 ? 1 : BYTES / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (BYTES == 32) {
            asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
            asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p + V / 2));
        } else if constexpr (BYTES == 16) {
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
        } else if constexpr (BYTES == 8) {
            asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};
template <typename T, int V>
__device__ __forceinline__ void store_row(T *p, const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = v[i];
        }
    } else if constexpr (V == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

constexpr int LOOSE = 8;  // elements of a thread, 32 apart, where rows go element by element and are many

// Threads and pieces of a row of n items: at most `most` threads, rows cut evenly.
struct Cut {
    int threads, pieces;
};
inline Cut cut(int n, int most) {
    Cut c;
    c.pieces = (n + most - 1) / most;
    c.threads = ((n + c.pieces - 1) / c.pieces + 31) / 32 * 32;
    return c;
}

// ------------------------------------------------------------------ sort

// Slots up to which every CTA counts them by itself (below 2^13): 64 experts, 8 slots to a token, 2048 bf16 columns: 3.1, 5.6
// and 7.2 us with 512, 2048 and 2560 slots against 6.2, 6.7 and 7.2 of the two kernels (1000 experts: 8.2 to 9.7).
constexpr int SMALL_N = 2560;
constexpr int SMALL_T = 256;    // threads

// A warp's LOOSE * 32 items of a row, from i on (lane 0's; i: this lane's first).
template <typename Item>
struct LooseRow {
    Item v[LOOSE];
    __device__ __forceinline__ LooseRow(const Item *x, int i, int items) {
        x += i;
        const int left = items - i;
#pragma unroll
        for (int u = 0; u < LOOSE; ++u)
            if (32 * u < left) v[u] = __ldg(x + 32 * u);
    }
    __device__ __forceinline__ void put(Item *row, int i, int items) const {
        row += i;
        const int left = items - i;
#pragma unroll
        for (int u = 0; u < LOOSE; ++u)
            if (32 * u < left) row[32 * u] = v[u];
    }
};

// Keys below `key` of n (padded to a multiple of 4), by a warp.
__device__ __forceinline__ int count_below(const uint32_t *keys, int n, uint32_t key, int lane) {
    int before = 0;
    for (int i = lane; i < (n + 3) / 4; i += 32) {
        const uint4 v = reinterpret_cast<const uint4 *>(keys)[i];
        before += (v.x < key) + (v.y < key) + (v.z < key) + (v.w < key);
    }
    return __reduce_add_sync(FULL, before);
}

// One kernel for few slots: CTA (token, piece of its row) counts where the token's slots go and copies the piece there.
// Slot s with id e has the key (e, s); its place is the number of lower keys.  An id that is no expert's sorts
// behind all experts; its slot is not placed.
template <typename Item>
__global__ void __launch_bounds__(SMALL_T) sort_small_kernel(const SortArgs a, int items, size_t px, size_t pr) {
    __shared__ __align__(16) uint32_t s_key[SMALL_N];
    __shared__ int s_place[32];
    wait_for_previous();
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int WARPS = SMALL_T / 32;
    const int n = a.T * a.K, i0 = blockIdx.y * SMALL_T + threadIdx.x;
    const Item *x = static_cast<const Item *>(a.x) + t * px;
    Item v;
    if (sizeof(Item) == 16 && a.x && i0 < items) v = __ldg(x + i0);  // on its way while the slots are counted
    for (int s = threadIdx.x; s < (n + 3 & ~3); s += SMALL_T) {
        uint32_t key = 0xffffffffu;
        if (s < n) {
            const int id = __ldg(a.ids + s);
            const bool ok = static_cast<unsigned>(id) < static_cast<unsigned>(a.E);
            if (!ok && id != -1 && t == 0 && blockIdx.y == 0) atomicOr(a.err, COLI_DEVERR_EXPERT_ID);
            key = static_cast<uint32_t>(ok ? id : a.E) << 13 | s;
        }
        s_key[s] = key;
    }
    __syncthreads();
    for (int k = warp; k < a.K; k += WARPS) {
        const int s = t * a.K + k;
        const uint32_t key = s_key[s];
        const int before = count_below(s_key, n, key, lane);
        if (lane == 0) {
            const bool ok = static_cast<int>(key >> 13) < a.E;
            s_place[k] = ok ? before : -1;
            if (blockIdx.y == 0) {
                a.place[s] = ok ? before : -1;
                a.perm[before] = ok ? s : -1;
            }
        }
    }
    if (blockIdx.y == 0) {
        if (n <= 64) {
            for (int e = t * SMALL_T + threadIdx.x; e <= a.E; e += a.T * SMALL_T) {
                int before = 0;
                for (int s = 0; s < n; ++s) before += s_key[s] < static_cast<uint32_t>(e) << 13;
                a.offsets[e] = before;
            }
        } else {
            for (int e = t * WARPS + warp; e <= a.E; e += a.T * WARPS) {
                const int before = count_below(s_key, n, static_cast<uint32_t>(e) << 13, lane);
                if (lane == 0) a.offsets[e] = before;
            }
        }
    }
    if (!a.x) return;
    __syncthreads();
    if constexpr (sizeof(Item) == 16) {
        for (int i = i0; i < items; i += gridDim.y * SMALL_T) {
            if (i != i0) v = __ldg(x + i);
            for (int k = 0; k < a.K; ++k) {
                const int to = s_place[k];
                if (to >= 0) static_cast<Item *>(a.rows)[to * pr + i] = v;
            }
        }
    } else {
        for (int i = (blockIdx.y * WARPS + warp) * 32 * LOOSE + lane; i < items + lane; i += gridDim.y * SMALL_T * LOOSE) {
            const LooseRow<Item> r(x, i, items);
            for (int k = 0; k < a.K; ++k) {
                const int to = s_place[k];
                if (to >= 0) r.put(static_cast<Item *>(a.rows) + to * pr, i, items);
            }
        }
    }
}

// Many slots: a cluster of SORT_CTAS CTAs sorts them (a share of the slots each, a warp its part of that, in order), then
// a second kernel copies the rows.  Pass 1 counts by warp and expert; the scans over warps, CTAs (through each
// other's shared memory) and experts turn the counts into first positions; pass 2 places the slots.  16,384 slots of 256 experts
// 6.8 us, 65,536 13, 262,144 36.  (Places of equal slots in a run by ballots over the bits of the id: 12 us where
// match.any took 17.)
constexpr int SORT_CTAS = 8, SORT_WARPS = 16, SORT_T = SORT_WARPS * 32;
constexpr int SORT_HOLD = 8;    // runs of 32 slots whose ids a warp keeps between the passes

// A word into the shared memory of CTA `rank` of the cluster, where this CTA has `p`.
__device__ __forceinline__ void put_peer(int *p, int rank, int v) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(r), "r"(v) : "memory");
}
__global__ void __launch_bounds__(SORT_T) sort_cluster_kernel(const SortArgs a) {  // one cluster of SORT_CTAS
    extern __shared__ int sm[];
    const int B = a.E + 1;              // the last for ids that are no expert's
    int *wc = sm;                       // [SORT_WARPS][B]: counts, then cursors
    int *tot = sm + SORT_WARPS * B;     // [SORT_CTAS][B]: every CTA's counts
    __shared__ int s_scan[SORT_WARPS];
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA has begun: its shared memory may be written to
    wait_for_previous();
    dependents_may_launch();            // the copies fetch their rows meanwhile
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
    const long n = static_cast<long>(a.T) * a.K;
    const int part = rank * SORT_WARPS + warp, parts = SORT_CTAS * SORT_WARPS;
    const int lo = static_cast<int>(n * part / parts), hi = static_cast<int>(n * (part + 1) / parts);
    const unsigned lt = (1u << lane) - 1u;
    int *mine = wc + warp * B;
    bool bad = false;
    // the buckets of a batch of runs of 32 slots: -1 behind the end
    int held[SORT_HOLD];
    auto fetch = [&](int base) {
#pragma unroll
        for (int h = 0; h < SORT_HOLD; ++h) {
            const int s = base + 32 * h + lane;
            held[h] = s < hi ? __ldg(a.ids + s) : -2;
        }
#pragma unroll
        for (int h = 0; h < SORT_HOLD; ++h) {
            const bool ok = static_cast<unsigned>(held[h]) < static_cast<unsigned>(a.E), in = base + 32 * h + lane < hi;
            bad = bad || (in && !ok && held[h] != -1);
            held[h] = ok ? held[h] : in ? a.E : -1;
        }
    };
    constexpr int BATCH = 32 * SORT_HOLD;
    fetch(lo);
    for (int i = tid; i < SORT_WARPS * B; i += SORT_T) wc[i] = 0;
    __syncthreads();
    for (int base = lo; base < hi; base += BATCH) {
        if (base != lo) fetch(base);
#pragma unroll
        for (int h = 0; h < SORT_HOLD; ++h)
            if (held[h] >= 0) atomicAdd(mine + held[h], 1);
    }
    if (bad) atomicOr(a.err, COLI_DEVERR_EXPERT_ID);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    for (int e = tid; e < B; e += SORT_T) {
        int c[SORT_WARPS], run = 0;
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) c[w] = wc[w * B + e];
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            wc[w * B + e] = run;
            run += c[w];
        }
#pragma unroll
        for (int c = 0; c < SORT_CTAS; ++c) put_peer(tot + rank * B + e, c, run);
    }
    // (nobody touches another CTA's memory behind this barrier: each may leave when it is done)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // a bucket per thread: what lower CTAs hold of it, and all CTAs; then the scan over the buckets
    int carry = 0;
    for (int base = 0; base < B; base += SORT_T) {
        const int e = base + tid;
        int below = 0, all = 0;
        if (e < B) {
#pragma unroll
            for (int c = 0; c < SORT_CTAS; ++c) {
                const int v = tot[c * B + e];
                below += c < rank ? v : 0;
                all += v;
            }
        }
        int inc = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int before = carry;
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            const int v = s_scan[w];
            before += w < warp ? v : 0;
            carry += v;
        }
        const int first = before + inc - all;
        if (e < B) {
            if (rank == 0) a.offsets[e] = first;
            int c[SORT_WARPS];
#pragma unroll
            for (int w = 0; w < SORT_WARPS; ++w) c[w] = wc[w * B + e];
#pragma unroll
            for (int w = 0; w < SORT_WARPS; ++w) wc[w * B + e] = c[w] + first + below;
        }
        __syncthreads();
    }
    for (int base = lo; base < hi; base += BATCH) {
        if (hi - lo > BATCH) fetch(base);
        unsigned peers[SORT_HOLD];  // the run's slots of the same bucket, from a ballot per bit of the bucket
#pragma unroll
        for (int h = 0; h < SORT_HOLD; ++h) peers[h] = FULL;
        for (int bit = 1; bit <= a.E; bit <<= 1) {
#pragma unroll
            for (int h = 0; h < SORT_HOLD; ++h) {
                const bool one = held[h] & bit;
                const unsigned ones = __ballot_sync(FULL, one);
                peers[h] &= one ? ones : ~ones;
            }
        }
#pragma unroll
        for (int h = 0; h < SORT_HOLD; ++h) {
            if (base + 32 * h >= hi) break;
            const int s = base + 32 * h + lane, id = held[h];
            const int first = id >= 0 ? mine[id] : 0, to = first + __popc(peers[h] & lt);
            __syncwarp();
            if (id >= 0) {
                if ((peers[h] & lt) == 0) mine[id] = first + __popc(peers[h]);
                a.place[s] = id < a.E ? to : -1;
                a.perm[to] = id < a.E ? s : -1;
            }
            __syncwarp();
        }
    }
}

// Row t of x to the places of its K slots, a piece of the row per CTA.  The piece is fetched before the sort has ended:
// x is older than the sort, which began when the kernels before it had ended.
template <typename Item>
__global__ void __launch_bounds__(SMALL_T) sort_copy_kernel(const SortArgs a, int items, size_t px, size_t pr) {
    const int t = blockIdx.x, lane = threadIdx.x & 31;
    const Item *x = static_cast<const Item *>(a.x) + t * px;
    auto place = [&] { return lane < a.K ? __ldcg(a.place + static_cast<size_t>(t) * a.K + lane) : -1; };
    if constexpr (sizeof(Item) == 16) {
        const int i = blockIdx.y * blockDim.x + threadIdx.x;
        Item v;
        if (i < items) v = __ldg(x + i);
        wait_for_previous();
        const int at = place();
        for (int k = 0; k < a.K; ++k) {
            const int to = __shfl_sync(FULL, at, k);
            if (to >= 0 && i < items) static_cast<Item *>(a.rows)[to * pr + i] = v;
        }
    } else {
        const int i = (blockIdx.y * blockDim.x + threadIdx.x - lane) * LOOSE + lane;
        const LooseRow<Item> r(x, i, items);
        wait_for_previous();
        const int at = place();
        for (int k = 0; k < a.K; ++k) {
            const int to = __shfl_sync(FULL, at, k);
            if (to >= 0) r.put(static_cast<Item *>(a.rows) + to * pr, i, items);
        }
    }
}

// The same by bulk copies through shared memory, a warp per CTA: pieces of rows come into a ring of BULK_SLOTS, lane k sends
// one on to the place of its token's slot k.  For long rows, where what is written is no more than BULK_ALL: 2048 tokens, 8 slots
// each, 2048 / 6144 / 8192 bf16 columns 17.7 / 40.5 / 53 us against 19.4 / 44 / 58 by sort_copy_kernel, 1024 columns the same; 8192 columns with
// 287 / 325 MiB written 61 / 70 against 64 / 72, 4096 tokens of 6144 (384 MiB) 85 against 83, 16,384 tokens of 4096 (1 GiB) 236 against 220.
constexpr int BULK_SLOTS = 4, BULK_PIECE = 16384, BULK_MIN = 4096;
constexpr long BULK_ALL = 288L << 20;

// (row, bytes: of a row and of its pieces, the last one shorter, multiples of 16; px, pr: from row to row.)
__global__ void __launch_bounds__(32) sort_bulk_kernel(const SortArgs a, int row, int bytes, int pieces, size_t px, size_t pr) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[BULK_SLOTS];
    __shared__ int s_abort;
    const int lane = threadIdx.x;
    volatile int *abort = &s_abort;
    if (lane == 0) {
        for (int i = 0; i < BULK_SLOTS; ++i) mbar_init(smem_u32(&bars[i]), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    const int all = a.T * pieces, mine = blockIdx.x < all ? (all - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1 : 0;
    auto load = [&](int i) {  // item i of this CTA into its slot of the ring
        const int w = blockIdx.x + i * gridDim.x, t = w / pieces, piece = w - t * pieces;
        const uint32_t bar = smem_u32(&bars[i % BULK_SLOTS]);
        if (elect_one()) {
            const uint32_t size = min(bytes, row - piece * bytes);
            mbar_expect_tx(bar, size);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         ::"r"(smem_u32(ring + static_cast<size_t>(i % BULK_SLOTS) * bytes)), "l"(static_cast<const unsigned char *>(a.x) + t * px + static_cast<size_t>(piece) * bytes),
                           "r"(size), "r"(bar) : "memory");
        }
        __syncwarp();
    };
    for (int i = 0; i < BULK_SLOTS && i < mine; ++i) load(i);
    wait_for_previous();
    auto place = [&](int i) {
        const int t = (blockIdx.x + i * gridDim.x) / pieces;
        return i < mine && lane < a.K ? __ldcg(a.place + static_cast<size_t>(t) * a.K + lane) : -1;
    };
    int next = place(0), i = 0;
    for (; i < mine; ++i) {
        const int at = next, w = blockIdx.x + i * gridDim.x, piece = w - w / pieces * pieces;
        next = place(i + 1);
        if (!__all_sync(FULL, mbar_wait(smem_u32(&bars[i % BULK_SLOTS]), (i / BULK_SLOTS) & 1, abort, a.err))) break;
        if (at >= 0)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                         ::"l"(static_cast<unsigned char *>(a.rows) + at * pr + static_cast<size_t>(piece) * bytes), "r"(smem_u32(ring + static_cast<size_t>(i % BULK_SLOTS) * bytes)),
                           "r"(min(bytes, row - piece * bytes)) : "memory");
        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        // the copies out of the slot before have read it: the next item may come there
        if (i > 0 && i - 1 + BULK_SLOTS < mine) load(i - 1 + BULK_SLOTS);
    }
    if (i < mine)  // given up: what was asked for lands before the ring is released
        for (int j = i; j < mine && j < max(i - 1, 0) + BULK_SLOTS; ++j) mbar_drain(smem_u32(&bars[j % BULK_SLOTS]), (j / BULK_SLOTS) & 1);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <typename Item>
cudaError_t sort_rows(const SortArgs &a, int item, cudaStream_t st) {
    const int ratio = sizeof(Item) / item, items = a.x ? a.hidden / ratio : 1;
    const size_t px = a.ldx / ratio, pr = a.ldr / ratio;
    constexpr int U = sizeof(Item) == 16 ? 1 : LOOSE;
    const Cut c = cut((items + U - 1) / U, SMALL_T);
    const int n = a.T * a.K;
    if (n <= SMALL_N) {
        const int pieces = a.T < device_sm_count() ? (items + SMALL_T * U - 1) / (SMALL_T * U) : 1;
        return launch_early(sort_small_kernel<Item>, dim3(a.T, pieces), SMALL_T, 0, st, 1, a, items, px, pr);
    }
    static std::atomic<uint64_t> ready{0}, ready_bulk{0};
    cudaError_t e = allow_smem(sort_cluster_kernel, (SORT_WARPS + SORT_CTAS) * (1024 + 1) * sizeof(int), ready);
    if (e != cudaSuccess) return e;
    const size_t smem = static_cast<size_t>(SORT_WARPS + SORT_CTAS) * (a.E + 1) * sizeof(int);
    if ((e = launch_early(sort_cluster_kernel, dim3(SORT_CTAS), SORT_T, smem, st, SORT_CTAS, a)) != cudaSuccess || !a.x) return e;
    const int row = a.hidden * item;
    if (sizeof(Item) == 16 && row >= BULK_MIN && static_cast<long>(n) * row <= BULK_ALL) {
        const int pieces = (row + BULK_PIECE - 1) / BULK_PIECE, bytes = ((row + pieces - 1) / pieces + 15) / 16 * 16;
        const long ring = static_cast<long>(BULK_SLOTS) * bytes, most = device_sm_count() * std::min(200 * 1024 / ring, 16L);
        if ((e = allow_smem(sort_bulk_kernel, BULK_SLOTS * BULK_PIECE, ready_bulk)) != cudaSuccess) return e;
        return launch_early(sort_bulk_kernel, dim3(static_cast<unsigned>(std::min(static_cast<long>(a.T) * pieces, most))), 32, ring, st, 1, a, row, bytes,
                            pieces, a.ldx * item, a.ldr * item);
    }
    return launch_early(sort_copy_kernel<Item>, dim3(a.T, c.pieces), c.threads, 0, st, 1, a, items, px, pr);
}

// ------------------------------------------------------------------ combine

constexpr int CT = 256;         // threads at most
constexpr int SM_T = 1024;      // threads of an SM with 64 registers each
// A thread takes V elements side by side, U times: rows with boundaries of 16 bytes once; others element by element, once where
// threads are over, LOOSE times where elements are many, fewer rows of a token in flight then and half the threads.
template <int U> constexpr int ROWS = U == 1 ? 8 : 4;
template <int U> constexpr int CTAS = U == 1 ? 4 : 2;   // resident per SM

// Rows place[k0 .. k0 + depth) of a token and their weights, one per lane; -1 where there is none.
struct Slots {
    int at;
    float f;
    __device__ __forceinline__ void load(const int32_t *place, const float *w, size_t t, int K, int k0, int depth, int lane) {
        const bool mine = lane < depth && k0 + lane < K;
        at = mine ? __ldg(place + t * K + k0 + lane) : -1;
        f = mine && w ? __ldg(w + t * K + k0 + lane) : 1.f;
    }
    __device__ __forceinline__ void check(int rows, int *err) {
        if (at < -1 || at >= rows) {
            at = -1;
            atomicOr(err, COLI_DEVERR_GROUPING);
        }
    }
};

// A CTA takes pieces of tokens' rows, one after another; the next one's places are on their way meanwhile.  Loads are
// behind predicates, not branches: those kept them apart (2048 tokens, 8 rows of 2047 bf16 elements: 31 us against 40).
template <typename Act, typename Out, int V, int U>
__global__ void __launch_bounds__(CT, CTAS<U>) combine_kernel(const CombineArgs a, int pieces) {
    constexpr int D = ROWS<U>, STEP = 32 * V;
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    int t = blockIdx.x / pieces, piece = blockIdx.x - t * pieces;
    const int dt = gridDim.x / pieces, dp = gridDim.x - dt * pieces;
    Slots next;
    if (t < a.T) next.load(a.place, a.w, t, a.K, 0, D, lane);
    while (t < a.T) {
        Slots s = next;
        const int c = (piece * blockDim.x + threadIdx.x - lane) * V * U + lane * V;
        const size_t t0 = t;
        t += dt;
        piece += dp;
        if (piece >= pieces) {
            piece -= pieces;
            ++t;
        }
        if (t < a.T) next.load(a.place, a.w, t, a.K, 0, D, lane);
        bool in[U];
        float acc[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = c + STEP * u < a.hidden;
            if (a.add && in[u]) {
                Raw<Out, V> r;
                r.load(static_cast<const Out *>(a.add) + t0 * a.ld_add + c + STEP * u);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[u][i] = r.at(i);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
            }
        }
        for (int k0 = 0; k0 < a.K; k0 += D) {
            if (k0) s.load(a.place, a.w, t0, a.K, k0, D, lane);
            s.check(a.rows, a.err);
            Raw<Act, V> v[D][U];
#pragma unroll
            for (int k = 0; k < D; ++k) {
                const int at = __shfl_sync(FULL, s.at, k);
                const Act *row = static_cast<const Act *>(a.y) + at * a.ldy + c;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (at >= 0 && in[u]) v[k][u].load(row + STEP * u);
            }
#pragma unroll
            for (int k = 0; k < D; ++k) {
                const float f = __shfl_sync(FULL, s.f, k);
                const bool have = __shfl_sync(FULL, s.at, k) >= 0;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (have && in[u]) {
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[u][i] = fmaf(f, v[k][u].at(i), acc[u][i]);
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (in[u]) store_row<Out, V>(static_cast<Out *>(a.out) + t0 * a.ldo + c + STEP * u, acc[u]);
    }
}

// ------------------------------------------------------------------ gradient

// A CTA takes tokens one after another, some of their rows at a time; the products with dout are summed over the CTA.
template <typename Act, typename Out, int V, int U>
__global__ void __launch_bounds__(U == 1 ? SM_T : CT, U == 1 ? 1 : CTAS<U>) combine_grad_kernel(const CombineGradArgs a) {
    constexpr int D = ROWS<U>, STEP = 32 * V;
    __shared__ float s_sum[2][SM_T / 32][D];
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int buf = 0;
    Slots next;
    if (blockIdx.x < a.T) next.load(a.place, a.w, blockIdx.x, a.K, 0, D, lane);
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        Slots s = next;
        if (t + static_cast<int>(gridDim.x) < a.T) next.load(a.place, a.w, t + gridDim.x, a.K, 0, D, lane);
        for (int k0 = 0; k0 < a.K; k0 += D, buf ^= 1) {
            if (k0) s.load(a.place, a.w, t, a.K, k0, D, lane);
            s.check(a.rows, a.err);
            float dot[D];
#pragma unroll
            for (int k = 0; k < D; ++k) dot[k] = 0.f;
            for (int c0 = 0; c0 < a.hidden; c0 += blockDim.x * V * U) {
                const int c = c0 + (threadIdx.x - lane) * V * U + lane * V;
                bool in[U];
                Raw<Out, V> d[U];
                Raw<Act, V> v[D][U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    in[u] = c + STEP * u < a.hidden;
                    if (in[u]) d[u].load(static_cast<const Out *>(a.dout) + t * a.ld_dout + c + STEP * u);
                }
                if (a.dw) {
#pragma unroll
                    for (int k = 0; k < D; ++k) {
                        const int at = __shfl_sync(FULL, s.at, k);
                        const Act *row = static_cast<const Act *>(a.y) + at * a.ldy + c;
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (at >= 0 && in[u]) v[k][u].load(row + STEP * u);
                    }
                }
                if (a.dy) {
#pragma unroll
                    for (int k = 0; k < D; ++k) {
                        const int at = __shfl_sync(FULL, s.at, k);
                        const float f = __shfl_sync(FULL, s.f, k);
                        Act *row = static_cast<Act *>(a.dy) + at * a.ld_dy + c;
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (at >= 0 && in[u]) {
                                float g[V];
#pragma unroll
                                for (int i = 0; i < V; ++i) g[i] = f * d[u].at(i);
                                store_row<Act, V>(row + STEP * u, g);
                            }
                    }
                }
                if (a.dw) {
#pragma unroll
                    for (int k = 0; k < D; ++k) {
                        const bool have = __shfl_sync(FULL, s.at, k) >= 0;
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (have && in[u]) {
#pragma unroll
                                for (int i = 0; i < V; ++i) dot[k] = fmaf(d[u].at(i), v[k][u].at(i), dot[k]);
                            }
                    }
                }
            }
            if (!a.dw) continue;
#pragma unroll
            for (int k = 0; k < D; ++k) {
#pragma unroll
                for (int o = 16; o; o >>= 1) dot[k] += __shfl_xor_sync(FULL, dot[k], o);
                if (lane == 0) s_sum[buf][warp][k] = dot[k];
            }
            __syncthreads();  // (the buffer is written again two rounds on: its readers have met the next round's barrier)
            if (threadIdx.x < D && k0 + threadIdx.x < a.K) {
                float sum = 0.f;
                for (int i = 0; i < warps; ++i) sum += s_sum[buf][i][threadIdx.x];
                a.dw[static_cast<size_t>(t) * a.K + k0 + threadIdx.x] = sum;
            }
        }
    }
}

// CTAs of so many threads for n pieces of work: those that are resident at once, `all` threads to an SM.
unsigned resident(long n, int threads, int all) {
    const long most = static_cast<long>(device_sm_count()) * std::min(all / threads, 32);
    return static_cast<unsigned>(n < most ? n : most);
}

// Whether single elements would keep all threads busy more than twice (149 rows of 2047 elements are many).  Eight elements to a thread
// against one, bf16 rows of 2047 elements, 8 to a token: 32 / 100 / 144 / 200 / 400 tokens combined in 3.2 / 3.2 / 3.4 / 3.8 / 5.4 us against 2.3 /
// 3.5 / 4.7 / 5.9 / 9.4, their gradient 4.9 / 4.9 / 4.9 / 6.2 / 9.4 against 6.1 / 6.2 / 6.3 / 9.7 / 13.2; rows of 33 elements, 148 / 9600 tokens, 3.0 /
// 10.5 against 2.2 / 8.0 and 3.7 / 16.1 against 2.6 / 14.1.
bool many(int T, int hidden) { return static_cast<long>(T) * hidden > 2L * device_sm_count() * SM_T; }

// Whether rows of `item`-byte elements can be taken `v` elements at a time, in accesses of at most 16 bytes.
bool whole(const void *p, size_t ld, size_t item, int v) {
    return !p || ((reinterpret_cast<uintptr_t>(p) | ld * item) & (item * v < 16 ? item * v - 1 : 15)) == 0;
}

template <typename Act, typename Out>
cudaError_t combine(const CombineArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(Act);
    auto run = [&](auto kernel, int n, int ctas) {
        const Cut c = cut(n, CT);
        return launch_early(kernel, dim3(resident(static_cast<long>(a.T) * c.pieces, c.threads, CT * ctas)), c.threads, 0, st, 1, a, c.pieces);
    };
    if (a.hidden % V == 0 && whole(a.y, a.ldy, sizeof(Act), V) && whole(a.add, a.ld_add, sizeof(Out), V) && whole(a.out, a.ldo, sizeof(Out), V))
        return run(combine_kernel<Act, Out, V, 1>, a.hidden / V, CTAS<1>);
    if (many(a.T, a.hidden)) return run(combine_kernel<Act, Out, 1, LOOSE>, (a.hidden + LOOSE - 1) / LOOSE, CTAS<LOOSE>);
    return run(combine_kernel<Act, Out, 1, 1>, a.hidden, CTAS<1>);
}

template <typename Act, typename Out>
cudaError_t combine_grad(const CombineGradArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(Act);
    auto run = [&](auto kernel, int n, int most, int ctas) {
        const int threads = cut(n, most).threads;
        return launch_early(kernel, dim3(resident(a.T, threads, CT * ctas)), threads, 0, st, 1, a);
    };
    const int most = a.T <= device_sm_count() ? SM_T : CT;  // (few tokens: all threads of an SM to each)
    if (a.hidden % V == 0 && whole(a.y, a.ldy, sizeof(Act), V) && whole(a.dout, a.ld_dout, sizeof(Out), V) && whole(a.dy, a.ld_dy, sizeof(Act), V))
        return run(combine_grad_kernel<Act, Out, V, 1>, a.hidden / V, most, CTAS<1>);
    if (many(a.T, a.hidden)) return run(combine_grad_kernel<Act, Out, 1, LOOSE>, (a.hidden + LOOSE - 1) / LOOSE, CT, CTAS<LOOSE>);
    return run(combine_grad_kernel<Act, Out, 1, 1>, a.hidden, most, CTAS<1>);
}

}  // namespace

cudaError_t launch_sort_rows(int act, const SortArgs &a, cudaStream_t st) {
    const int item = act == COLI_ACT_F32 ? 4 : 2;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.rows) | a.ldx * item | a.ldr * item | static_cast<size_t>(a.hidden) * item;
    if (!a.x || (at & 15) == 0) return sort_rows<uint4>(a, item, st);
    if ((at & 3) == 0) return sort_rows<uint32_t>(a, item, st);
    return sort_rows<uint16_t>(a, item, st);
}

cudaError_t launch_combine(int act, int out_type, const CombineArgs &a, cudaStream_t st) {
    if (act == COLI_ACT_F32)
        return out_type == COLI_ACT_F32 ? combine<float, float>(a, st) : combine<float, __nv_bfloat16>(a, st);
    return out_type == COLI_ACT_F32 ? combine<__nv_bfloat16, float>(a, st) : combine<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_combine_grad(int act, int out_type, const CombineGradArgs &a, cudaStream_t st) {
    if (act == COLI_ACT_F32)
        return out_type == COLI_ACT_F32 ? combine_grad<float, float>(a, st) : combine_grad<float, __nv_bfloat16>(a, st);
    return out_type == COLI_ACT_F32 ? combine_grad<__nv_bfloat16, float>(a, st) : combine_grad<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace coli
