// i8_gemm.cu -- products of 8-bit operands on the 5th-generation tensor cores (coli_moe_i8_product).
//
// out[i][j] = sa[i] * sw[j] * sum_k a[i][k] * w[j][k]
// The sums are whole numbers in 32 bits (exact); they become float32 and take the two scales in the epilogue.
//
// Swap-AB, tiles, groups and split k as in the product of 4-bit operands: weight rows of one matrix are the MMA's M side,
// rows of the matrix's group its N side; a k-block is 128 bytes of every row, 128 elements here.  Three
// tiles, chosen on the host:
//   at most 32 rows in all      128 weight rows x 32, k split over a cluster where tiles are few
//   few each (use_pairs)        128 weight rows x 128
//   more                        256 weight rows x 256 on a pair of CTAs
//
// One persistent CTA per SM, warp-specialised; tiles are taken round-robin:
//   warp 0      TMA producer: weight codes and the rows' codes (128-byte swizzle)
//   warp 1      MMA issuer: 4 MMAs of K = 32 a k-block
//   the others  epilogue, from two accumulators: one drains while the other fills
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "group_tiles.h"
#include "i8.h"
#include "internal.h"
#include "pdl.h"

namespace coli {

namespace {

constexpr int KB = 128;                  // elements (bytes) of a k-block's row
constexpr int A_BYTES = 128 * KB;        // weight codes of a k-block
constexpr int W_PROD = 0, W_MMA = 1, W_EPI0 = 2, N_EPI = 4;
constexpr int THREADS = (W_EPI0 + N_EPI) * 32;

template <int NT>
struct Plan {
    static constexpr int B_BYTES = NT * KB;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int PART = NT <= 32 ? (MAX_SPLIT - 1) * 32 * 128 * 4 : 0;  // split k: the other ranks' sums
    static constexpr int S = (216 * 1024 - PART) / STAGE;                       // ring stages
    static constexpr int ACC = NT <= 32 ? 32 : 128;                             // columns of an accumulator
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + PART + 1024;
};

// Instruction descriptor of kind::i8: D s32 (bits 4-5 = 2), A and B signed 8-bit (bits 7-9, 10-12 = 1),
// both K-major, M >> 4 in bits 24-28; N >> 3 goes to bits 17-22.
constexpr uint32_t idesc_i8(int m) { return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(m >> 4) << 24); }

template <int CTAS>
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (CTAS == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

struct GemmArgs : GroupArgs {
    const float *wscale;                 // [n] per matrix, or nullptr
    size_t wscale_stride;
    const float *xscale;                 // [rows], or nullptr
    int k;
    void *out;
    size_t ldo;
};
struct GemmMaps {
    CUtensorMap a;                       // weight codes {k bytes, n rows, matrices}
    CUtensorMap b[NBOX];                 // row codes {k bytes, rows}, boxes of 16 << i rows
};
__device__ __forceinline__ void prefetch_maps(const GemmMaps &m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&m.a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&m.b[0])) : "memory");
}

__device__ __forceinline__ int add_ints(int a, int b) { return a + b; }

// The sums of a run of 32 rows, as float32, times what of the scales' exponents does not go through their product.
// (The sum is rounded to 24 bits once, the product of the scales once, and theirs once.)
__device__ __forceinline__ void run_sums(int (&v)[32], float &rw, float &rx) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __float_as_int(__int2float_rn(v[j]));
    if (!__all_sync(0xffffffffu, ordinary(rw) && ordinary(rx))) {
        const float pw = halve_exponent(rw);
        split_scales(v, pw, rx);
    }
}

template <int NT, int OUT>
__global__ void __launch_bounds__(THREADS, 1) i8_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {
    using P = Plan<NT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES;
    constexpr bool SPLIT = NT <= 32;
    __shared__ __align__(8) uint64_t bars[2 * P::S + 7];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_tiles;
    __shared__ TileList list;
    __shared__ int s_scan[THREADS / 32];
    uint64_t *full = bars, *empty = full + P::S;
    uint64_t *dfull = empty + P::S, *dempty = dfull + 2, *drain = dempty + 2;
    uint64_t *pfull = drain + 1, *pfree = pfull + 1;  // split k: partial sums there; their place free again
    float *part = reinterpret_cast<float *>(sb + P::S * P::B_BYTES);
    // split k: the CTAs of a cluster take a share of the k-blocks each; rank 0 adds and stores
    const int C = SPLIT ? static_cast<int>(cluster_size()) : 1, rank = SPLIT ? static_cast<int>(cluster_rank()) : 0;
    const int first = blockIdx.x / C, stride = gridDim.x / C;
    volatile int *abort = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int MB = (p.n + 127) / 128, KALL = (p.k + KB - 1) / KB;
    const int kb0 = KALL * rank / C, KT = KALL * (rank + 1) / C - kb0;
    const int W = p.E;

    if (threadIdx.x == 0) {
        for (int i = 0; i < P::S; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&dfull[i]), 1);
            mbar_init(smem_u32(&dempty[i]), N_EPI * 32);
        }
        mbar_init(smem_u32(drain), 1);
        mbar_init(smem_u32(pfull), N_EPI);
        mbar_init(smem_u32(pfree), N_EPI);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) tmem_alloc(smem_u32(&s_tmem), 512);
    if (warp == W_PROD && elect_one()) prefetch_maps(maps);
    wait_for_previous();
    if (warp >= W_EPI0) {
        const int n = tile_list<NT, N_EPI * 32, W_EPI0>(p, W, MB, list, s_scan);
        if (threadIdx.x == W_EPI0 * 32) s_tiles = n;
    }
    tc_fence_before();
    __syncthreads();
    // the cluster's barriers are set up: waited for where another CTA's memory is first touched
    if (SPLIT && C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tbase = s_tmem;
    const int ntiles = s_tiles;

    if (warp == W_PROD) {
        // ------------------------------------------------------------------ TMA producer
        uint32_t it = 0, s = 0, phase = 1;
        for (int t = first; t < ntiles; t += stride) {
            const Tile x = tile_at<NT>(t, list, p, W);
            const int n16 = (x.nr + 15) / 16;
            for (int kb = 0; kb < KT; ++kb, ++it) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), phase, abort, p.err))) goto prod_done;
                const uint32_t fb = smem_u32(&full[s]);
                if (elect_one()) {
                    mbar_expect_tx(fb, A_BYTES + n16 * 16 * KB);
                    tma_load_3d(smem_u32(sa + s * A_BYTES), &maps.a, (kb0 + kb) * KB, x.m * 128, x.e, fb);
#pragma unroll
                    for (int bit = NT <= 32 ? 1 : NBOX - 1; bit >= 0; --bit) {
                        const int row0 = 16 * ((n16 >> (bit + 1)) << (bit + 1));  // rows of the larger boxes
                        if ((n16 >> bit) & 1) tma_load_2d(smem_u32(sb + s * P::B_BYTES + row0 * KB), &maps.b[bit], (kb0 + kb) * KB, x.n0 + row0, fb);
                    }
                }
                __syncwarp();
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
    prod_done:
        if (*abort && lane == 0) {
            // let the copies already issued land before the CTA's shared memory is released
            for (uint32_t i = it > static_cast<uint32_t>(P::S) ? it - P::S : 0; i < it; ++i)
                mbar_drain(smem_u32(&full[i % P::S]), (i / P::S) & 1);
        }
    } else if (warp == W_MMA) {
        // ------------------------------------------------------------------ MMA issuer
        uint32_t s = 0, phase = 0, tl = 0;
        const uint64_t adesc0 = smem_desc_sw128(smem_u32(sa)), bdesc0 = smem_desc_sw128(smem_u32(sb));
        for (int t = first; t < ntiles; t += stride, ++tl) {
            const Tile x = tile_at<NT>(t, list, p, W);
            const int n16 = (x.nr + 15) / 16;
            const uint32_t idesc = idesc_i8(128) | (static_cast<uint32_t>(2 * n16) << 17);
            const int acc = tl & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&dempty[acc]), ((tl >> 1) & 1) ^ 1, abort, p.err))) goto mma_done;
            tc_fence_after();
            const uint32_t dt = tbase + acc * P::ACC;
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), phase, abort, p.err))) goto mma_done;
                tc_fence_after();
                const int steps = min(4, (p.k - (kb0 + kb) * KB + 31) / 32);  // K = 32 steps that hold elements
                if (elect_one()) {
                    const uint64_t ad = adesc0 + static_cast<uint64_t>(s * (A_BYTES >> 4)), bd = bdesc0 + static_cast<uint64_t>(s * (P::B_BYTES >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < steps) mma_i8<1>(dt, ad + 2 * kk, bd + 2 * kk, idesc, (kb | kk) != 0);
                    mma_commit(smem_u32(&empty[s]));
                }
                __syncwarp();
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (elect_one()) mma_commit(smem_u32(&dfull[acc]));
            __syncwarp();
        }
    mma_done:
        // every MMA issued so far has completed once this commit arrives
        if (elect_one()) mma_commit(smem_u32(drain));
        __syncwarp();
        mbar_drain(smem_u32(drain), 0);
    } else {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3;  // TMEM lane quarter (warp % 4)
        uint32_t tl = 0;
        if (SPLIT && C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        for (int t = first; t < ntiles; t += stride, ++tl) {
            const Tile x = tile_at<NT>(t, list, p, W);
            const int acc = tl & 1;
            const int r = x.m * 128 + 32 * q + lane;
            const float rw = p.wscale && r < p.n ? __ldg(p.wscale + static_cast<size_t>(x.e) * p.wscale_stride + r) : 1.f;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&dfull[acc]), (tl >> 1) & 1, abort, p.err))) break;
            tc_fence_after();
            const uint32_t dt = tbase + acc * P::ACC + (static_cast<uint32_t>(32 * q) << 16);
            for (int g = 0; g < x.nr; g += 32) {
                int v[32];
                tmem_ld32(dt + g, v);
                if (SPLIT && C > 1) {
                    if (!split_sum(v, x.nr, C, rank, q, lane, tl, t + stride >= ntiles, part, pfull, pfree, abort, p.err, add_ints)) break;
                    if (rank != 0) break;
                }
                float rx = p.xscale && g + lane < x.nr ? __ldg(p.xscale + x.n0 + g + lane) : 1.f, rwg = rw;
                run_sums(v, rwg, rx);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (g + j >= x.nr) break;  // the same for the whole warp
                    const float y = __int_as_float(v[j]) * (rwg * __shfl_sync(0xffffffffu, rx, j));
                    if (r < p.n) {
                        const size_t at = static_cast<size_t>(x.n0 + g + j) * p.ldo + r;
                        if (OUT == COLI_ACT_F32) static_cast<float *>(p.out)[at] = y;
                        else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&dempty[acc]));
        }
    }

    dependents_may_launch();
    if (SPLIT && C > 1 && warp < W_EPI0) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (SPLIT && C > 1) cluster_sync_all();  // no CTA leaves while another may still write to it
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// ------------------------------------------------------------------ CTA pairs --------------
// Tiles of 256 weight rows x up to 256 rows on a pair of CTAs (cta_group::2): each CTA fetches its own 128 weight rows
// and half of the tile's rows, the tensor cores read both halves.  Two accumulators of 256 columns per CTA.
constexpr int P_THREADS = (W_EPI0 + P_EPI) * 32;
constexpr int P_OUT = 8192;              // bytes of an epilogue half's staging buffer

struct PairPlan {
    static constexpr int B_BYTES = P_NT / 2 * KB;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int S = (216 * 1024 - 2 * P_OUT) / STAGE;
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + 2 * P_OUT + 1024;
};

// A run of 32 rows x this CTA's 128 weight rows through shared memory: lanes hold a weight row each, out wants weight
// rows side by side.  `buf`: the half's P_OUT bytes; vec: 16-byte stores are aligned.
template <int OUT>
__device__ __forceinline__ void staged_run(const GemmArgs &p, const Tile &x, const int *v, int g, int row0, float rw, float rx,
                                           unsigned char *buf, int half, int q, int lane, bool vec) {
    constexpr int ITEM = OUT == COLI_ACT_F32 ? 4 : 2;
    constexpr int RUN = OUT == COLI_ACT_F32 ? 16 : 32;    // rows at a time
    constexpr int COLS = 128;
    constexpr int VPR = COLS * ITEM / 16;                 // 16-byte pieces of a row
    const int tid = 32 * q + lane;
#pragma unroll
    for (int h = 0; h < 32 / RUN; ++h) {
        if (g + RUN * h >= x.nr) return;                  // the same for all four warps
        half_sync(half);                                  // the buffer's last run has been read
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
            const float y = __int_as_float(v[RUN * h + j]) * (rw * __shfl_sync(0xffffffffu, rx, RUN * h + j));
            if (OUT == COLI_ACT_F32) reinterpret_cast<float *>(buf)[j * COLS + tid] = y;
            else reinterpret_cast<__nv_bfloat16 *>(buf)[j * COLS + tid] = __float2bfloat16_rn(y);
        }
        half_sync(half);
#pragma unroll
        for (int i = 0; i < RUN * VPR / 128; ++i) {
            const int at = i * 128 + tid, j = at / VPR, c = row0 + (at % VPR) * (16 / ITEM);
            const int row = g + RUN * h + j;
            if (row >= x.nr || c >= p.n) continue;
            unsigned char *dst = static_cast<unsigned char *>(p.out) + (static_cast<size_t>(x.n0 + row) * p.ldo + c) * ITEM;
            const uint4 w = *reinterpret_cast<const uint4 *>(buf + 16 * at);
            if (vec && c + 16 / ITEM <= p.n) {
                *reinterpret_cast<uint4 *>(dst) = w;
            } else {
                const int n = min(16 / ITEM, p.n - c);
                for (int e = 0; e < n; ++e) {
                    if (ITEM == 4) reinterpret_cast<float *>(dst)[e] = reinterpret_cast<const float *>(buf + 16 * at)[e];
                    else reinterpret_cast<uint16_t *>(dst)[e] = reinterpret_cast<const uint16_t *>(buf + 16 * at)[e];
                }
            }
        }
    }
}

template <int OUT>
__global__ void __launch_bounds__(P_THREADS, 1) i8_pair_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {  // clusters of 2
    using P = PairPlan;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // the same offset in both CTAs: the dynamic array starts at the same address in each
    unsigned char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES, *sout = sb + P::S * P::B_BYTES;
    __shared__ __align__(8) uint64_t bars[2 * P::S + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_tiles;
    __shared__ TileList list;
    __shared__ int s_scan[P_THREADS / 32];
    // full: the leader's, of both CTAs' copies; empty, dfull: in each CTA; dempty: the leader's
    uint64_t *full = bars, *empty = full + P::S, *dfull = empty + P::S, *dempty = dfull + 2, *drain = dempty + 2;
    volatile int *abort = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int MB = (p.n + 255) / 256, KT = (p.k + KB - 1) / KB;
    const int W = p.E;

    if (threadIdx.x == 0) {
        for (int i = 0; i < P::S; ++i) {
            mbar_init(smem_u32(&full[i]), 2);  // each CTA's producer
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&dfull[i]), 1);
            mbar_init(smem_u32(&dempty[i]), 2 * P_EPI);
        }
        mbar_init(smem_u32(drain), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == W_PROD && elect_one()) prefetch_maps(maps);
    wait_for_previous();
    if (warp >= W_EPI0) {
        const int n = tile_list<P_NT, P_EPI * 32, W_EPI0>(p, W, MB, list, s_scan);
        if (threadIdx.x == W_EPI0 * 32) s_tiles = n;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tbase = s_tmem;
    const int ntiles = s_tiles;

    if (warp == W_PROD) {
        // ------------------------------------------------------------------ TMA producer
        uint32_t s = 0, phase = 1;
        for (int t = pair; t < ntiles; t += pairs) {
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int n32 = (x.nr + 31) / 32;                        // N / 32; this CTA's share is 16 * n32 rows
            const int row_lo = x.n0 + static_cast<int>(rank) * 16 * n32;
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), phase, abort, p.err))) goto prod_done;
                const uint32_t fb = map_rank(smem_u32(&full[s]), 0);
                if (elect_one()) {
                    remote_expect_tx(fb, A_BYTES + n32 * 16 * KB);
                    pair_load_3d(smem_u32(sa + s * A_BYTES), &maps.a, kb * KB, x.m * 256 + static_cast<int>(rank) * 128, x.e, fb);
#pragma unroll
                    for (int bit = NBOX - 1; bit >= 0; --bit) {
                        const int row0 = 16 * ((n32 >> (bit + 1)) << (bit + 1));
                        if ((n32 >> bit) & 1) pair_load_2d(smem_u32(sb + s * P::B_BYTES + row0 * KB), &maps.b[bit], kb * KB, row_lo + row0, fb);
                    }
                }
                __syncwarp();
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
    prod_done:
        // a producer that gives up leaves its copies to land: the pair's barrier below waits for the
        // leader, whose MMA warp waits for them (bounded)
        ;
    } else if (warp == W_MMA && rank == 0) {
        // ------------------------------------------------------------------ MMA issuer (the pair's)
        uint32_t s = 0, phase = 0, tl = 0;
        const uint64_t adesc0 = smem_desc_sw128(smem_u32(sa)), bdesc0 = smem_desc_sw128(smem_u32(sb));
        for (int t = pair; t < ntiles; t += pairs, ++tl) {
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int n32 = (x.nr + 31) / 32, acc = tl & 1;
            const uint32_t idesc = idesc_i8(256) | (static_cast<uint32_t>(4 * n32) << 17);
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&dempty[acc]), ((tl >> 1) & 1) ^ 1, abort, p.err))) goto mma_done;
            tc_fence_after();
            const uint32_t dt = tbase + acc * P_NT;
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&full[s]), phase, abort, p.err))) goto mma_done;
                tc_fence_after();
                const int steps = min(4, (p.k - kb * KB + 31) / 32);
                if (elect_one()) {
                    const uint64_t ad = adesc0 + static_cast<uint64_t>(s * (A_BYTES >> 4)), bd = bdesc0 + static_cast<uint64_t>(s * (P::B_BYTES >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < steps) mma_i8<2>(dt, ad + 2 * kk, bd + 2 * kk, idesc, (kb | kk) != 0);
                    pair_commit(smem_u32(&empty[s]));
                }
                __syncwarp();
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (elect_one()) pair_commit(smem_u32(&dfull[acc]));
            __syncwarp();
        }
    mma_done:
        if (elect_one())
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(drain)) : "memory");
        __syncwarp();
        mbar_drain(smem_u32(drain), 0);
        if (*abort) {  // copies that are still in flight land before shared memory is released
            for (int i = 0; i < P::S; ++i) {
                mbar_drain(smem_u32(&full[s]), phase);
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= W_EPI0) {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - W_EPI0) >> 2;  // TMEM lane quarter, 128-column half
        unsigned char *obuf = sout + half * P_OUT;
        constexpr int ITEM = OUT == COLI_ACT_F32 ? 4 : 2;
        const bool vec = ((reinterpret_cast<uintptr_t>(p.out) | (p.ldo * ITEM)) & 15) == 0;
        uint32_t tl = 0;
        for (int t = pair; t < ntiles; t += pairs, ++tl) {
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int acc = tl & 1, row0 = x.m * 256 + static_cast<int>(rank) * 128;
            const int r = row0 + 32 * q + lane;
            const float rw = p.wscale && r < p.n ? __ldg(p.wscale + static_cast<size_t>(x.e) * p.wscale_stride + r) : 1.f;
            // (all eight warps meet in the staging barriers: they give up together, or not at all)
            if (epi_or(!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&dfull[acc]), (tl >> 1) & 1, abort, p.err)))) break;
            tc_fence_after();
            const uint32_t dt = tbase + acc * P_NT + (static_cast<uint32_t>(32 * q) << 16);
            for (int g = 128 * half; g < min(x.nr, 128 * half + 128); g += 32) {
                float rx = p.xscale && g + lane < x.nr ? __ldg(p.xscale + x.n0 + g + lane) : 1.f, rwg = rw;
                int v[32];
                tmem_ld32(dt + g, v);
                run_sums(v, rwg, rx);
                staged_run<OUT>(p, x, v, g, row0, rwg, rx, obuf, half, q, lane, vec);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive(map_rank(smem_u32(&dempty[acc]), 0));
        }
    }

    dependents_may_launch();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == W_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512u) : "memory");
    }
}

// Weight codes of `count` matrices, boxes of 128 rows of a k-block.
bool mats_map(CUtensorMap *m, const coli_i8_mats &w, int k) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(w.n), static_cast<cuuint64_t>(w.count)};
    const cuuint64_t strides[2] = {w.ld, w.count > 1 ? w.codes_stride : static_cast<cuuint64_t>(w.n) * w.ld};
    const cuuint32_t box[3] = {KB, 128, 1};
    return encode_u8(m, w.codes, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Row codes, boxes of 16 << i rows, as far as the rows reach.
bool rows_maps(CUtensorMap *m, const coli_i8_rows &a, int k) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t strides[1] = {a.ld};
    for (int i = 0; i < NBOX; ++i) {
        if (i && (8 << i) >= a.rows) {  // no group is that high: the box is never used
            m[i] = m[i - 1];
            continue;
        }
        const cuuint32_t box[2] = {KB, static_cast<cuuint32_t>(16 << i)};
        if (!encode_u8(m + i, a.codes, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
    }
    return true;
}

// Groups that have rows, at most.
long groups_of(const GemmArgs &g) { return g.rows < g.E ? g.rows : g.E; }

template <int OUT>
cudaError_t launch_gemm(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<128>;
    auto kernel = i8_gemm_kernel<128, OUT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const long tiles = (g.rows / 128 + groups_of(g)) * ((g.n + 127) / 128);
    const int sms = device_sm_count();
    return launch_early(kernel, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), THREADS, P::SMEM, st, 1, maps, g);
}

// At most 32 rows: tiles of 128 weight rows x all rows of a matrix, their k-blocks split over clusters of 1, 2
// or 4 CTAs, whichever leaves the busiest CTA the least (the matrices that have rows are at most as many as rows).
template <int OUT>
cudaError_t launch_split(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<32>;
    auto kernel = i8_gemm_kernel<32, OUT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count(), kt = (g.k + KB - 1) / KB;
    const int tiles = static_cast<int>(groups_of(g)) * ((g.n + 127) / 128);
    int C = 1;
    long best = 0;
    for (int c = 1; c <= MAX_SPLIT && c <= kt; c *= 2) {
        const int clusters = cluster_count(c, sms);
        const long cost = static_cast<long>((tiles + clusters - 1) / clusters) * ((kt + c - 1) / c);  // k-blocks of the busiest CTA
        if (c == 1 || 16 * cost < 15 * best) {
            best = cost;
            C = c;
        }
    }
    const int clusters = cluster_count(C, sms);
    return launch_early(kernel, dim3(C * (tiles < clusters ? tiles : clusters)), THREADS, P::SMEM, st, C, maps, g);
}

template <int OUT>
cudaError_t launch_pair(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = PairPlan;
    auto kernel = i8_pair_kernel<OUT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const long tiles = (g.rows / P_NT + groups_of(g)) * ((g.n + 255) / 256);
    const int pairs = device_sm_count() / 2;
    return launch_early(kernel, dim3(2 * static_cast<unsigned>(tiles < pairs ? tiles : pairs)), P_THREADS, P::SMEM, st, 2, maps, g);
}

template <int OUT>
cudaError_t launch_out(const GemmMaps &maps, const GemmArgs &g, bool pairs, cudaStream_t st) {
    if (pairs) return launch_pair<OUT>(maps, g, st);
    return g.rows <= 32 ? launch_split<OUT>(maps, g, st) : launch_gemm<OUT>(maps, g, st);
}

}  // namespace

constexpr int PAIR_ROWS = 112;

static bool use_pairs(const I8ProductArgs &p) {
    const int avg = p.a.rows / p.w.count;
    return avg >= PAIR_ROWS || (avg > 32 && static_cast<long>(p.w.count) * ((avg + 127) / 128) * ((p.w.n + 127) / 128) < device_sm_count());
}

cudaError_t launch_i8_product(const I8ProductArgs &p, cudaStream_t st) {
    GemmMaps maps;
    if (!mats_map(&maps.a, p.w, p.k) || !rows_maps(maps.b, p.a, p.k)) return cudaErrorInvalidValue;
    GemmArgs g;
    g.offsets = p.offsets;
    g.E = p.w.count;
    g.S = 0;
    g.rows = p.a.rows;
    g.n = p.w.n;
    g.err = p.err;
    g.wscale = p.w.scale;
    g.wscale_stride = p.w.scale_stride;
    g.xscale = p.a.scale;
    g.k = p.k;
    g.out = p.out;
    g.ldo = p.ldo;
    const bool pairs = use_pairs(p);
    return p.out_type == COLI_ACT_F32 ? launch_out<COLI_ACT_F32>(maps, g, pairs, st) : launch_out<COLI_ACT_BF16>(maps, g, pairs, st);
}

}  // namespace coli
