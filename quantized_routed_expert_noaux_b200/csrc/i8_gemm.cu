// i8_gemm.cu -- products of 8-bit operands on the 5th-generation tensor cores (coli_moe_i8_product).
//
// out[i][j] = sa[i] * sw[j] * sum_k a[i][k] * w[j][k]
// The sums are whole numbers in 32 bits (exact); they become float32 and take the two scales in the epilogue.
//
// Swap-AB, tiles, groups and split k as in the product of 4-bit operands: weight rows of one matrix are the MMA's M side,
// rows of the matrix's group its N side; a k-block is 128 bytes of every row, 128 elements here.  Tiles, chosen on the host
// (launch_out):
//   128 weight rows x 32 or 128    k split over a cluster of CTAs where tiles are few
//   128 weight rows x 128          few rows to a matrix, many matrices
//   256 weight rows x 256          on a pair of CTAs, from 32 rows to a matrix; k split over two pairs where tiles are few
//
// Few rows to a matrix make it a stream of weights: 64 matrices of 4096 x 6144 with 4 / 16 / 32 / 64 / 128 rows each take 240 / 245 /
// 253 / 261 / 285 us (6.7 to 6.1 TB/s; copy peak 6.5); of 6144 x 2048 127 / 131 / 137 / 143 / 159.  From 64 rows on the operands'
// way from L2 counts (64 matrices 6144 x 2048, 4096 rows: 1.65 GB in 144 us, 40 bytes per cycle and SM), which is why
// pairs, whose CTAs share a tile's rows, take over at 32.  Many rows are bound by the power cap: 8192 rows, 4096 x 6144 in
// 125 us at 1594 MHz (3.3 POPS, tensor pipe active in 85% of the cycles), 145 us in long runs.
//
// One persistent CTA per SM, warp-specialised; tiles are taken round-robin:
//   warp 0      TMA producer: weight codes and the rows' codes (128-byte swizzle)
//   warp 1      MMA issuer: 4 MMAs of K = 32 a k-block
//   the others  epilogue, from two accumulators: one drains while the other fills
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

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
constexpr int STAGED = 2048, WARP_BUF = STAGED + 128;  // an epilogue warp's shared memory: values on their way out, scales

template <int NT, bool SPLIT>
struct Plan {
    static constexpr int B_BYTES = NT * KB;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int PART = SPLIT ? (MAX_SPLIT - 1) * NT / MAX_SPLIT * 128 * 4 : 0;  // split k: the other CTAs' sums (most with MAX_SPLIT of them)
    static constexpr int S = (216 * 1024 - PART - N_EPI * WARP_BUF) / STAGE;    // ring stages
    static constexpr int ACC = NT <= 32 ? 32 : 128;                             // columns of an accumulator
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + PART + N_EPI * WARP_BUF + 1024;
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

// The sums of a run of N rows, as float32, times what of the scales' exponents does not go through their product.
// (The sum is rounded to 24 bits once, the product of the scales once, and theirs once.)
template <int N>
__device__ __forceinline__ void run_sums(int (&v)[N], float &rw, float &rx) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __float_as_int(__int2float_rn(v[j]));
    if (!__all_sync(0xffffffffu, ordinary(rw) && ordinary(rx))) {
        const float pw = halve_exponent(rw);
        split_scales(v, pw, rx);
    }
}
// Rows g .. g + N - 1 of a tile x this warp's 32 weight rows (from r0 on, one per lane).  out wants weight rows side by side:
// where its rows start at multiples of 16 bytes (vec) the values go through the warp's shared memory and out in
// 16-byte pieces, else straight from the lanes.
template <int OUT, int N>
__device__ __forceinline__ void store_run(const GemmArgs &p, const Tile &x, int (&v)[N], int g, int r0, float rw, unsigned char *buf, bool vec) {
    constexpr int ITEM = OUT == COLI_ACT_F32 ? 4 : 2;
    using Item = typename std::conditional<OUT == COLI_ACT_F32, float, __nv_bfloat16>::type;
    const int lane = threadIdx.x & 31;
    float rx = p.xscale && lane < N && g + lane < x.nr ? __ldg(p.xscale + x.n0 + g + lane) : 1.f;
    run_sums(v, rw, rx);
    float *s_rx = reinterpret_cast<float *>(buf + STAGED);
    __syncwarp();                                          // what was there has been read
    if (lane < N) s_rx[lane] = rx;
    __syncwarp();
    auto item = [](float y) {
        if constexpr (OUT == COLI_ACT_F32) return y;
        else return __float2bfloat16_rn(y);
    };
    if (vec) {
        constexpr int FIT = STAGED / (32 * ITEM), RUN = N < FIT ? N : FIT;  // rows at a time
        constexpr int PIECES = 32 * ITEM / 16, ROWS = 32 / PIECES;          // 16-byte pieces of a row, rows of a step
        const int c = r0 + lane % PIECES * (16 / ITEM);
        unsigned char *dst = static_cast<unsigned char *>(p.out) + (static_cast<size_t>(x.n0 + g + lane / PIECES) * p.ldo + c) * ITEM;
        const size_t step = ROWS * p.ldo * ITEM;
        const int left = c < p.n ? x.nr - g - lane / PIECES : 0;            // rows from this lane's first on
#pragma unroll
        for (int h = 0; h < N; h += RUN) {
            if (g + h >= x.nr) return;                                      // the same for the whole warp
            if (h) __syncwarp();
#pragma unroll
            for (int j = 0; j < RUN; j += 4) {
                const float4 s = *reinterpret_cast<const float4 *>(s_rx + h + j);
                Item *to = reinterpret_cast<Item *>(buf) + j * 32 + lane;
                to[0] = item(__int_as_float(v[h + j]) * (rw * s.x));
                to[32] = item(__int_as_float(v[h + j + 1]) * (rw * s.y));
                to[64] = item(__int_as_float(v[h + j + 2]) * (rw * s.z));
                to[96] = item(__int_as_float(v[h + j + 3]) * (rw * s.w));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < RUN; i += ROWS, dst += step) {
                if (h + i >= left) continue;
                const uint4 w = *reinterpret_cast<const uint4 *>(buf + 16 * lane + i * 32 * ITEM);
                if (c + 16 / ITEM <= p.n) {
                    *reinterpret_cast<uint4 *>(dst) = w;
                } else {
                    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 16 / ITEM; ++e)
                        if (c + e < p.n) {
                            if (ITEM == 4) reinterpret_cast<uint32_t *>(dst)[e] = words[e];
                            else reinterpret_cast<uint16_t *>(dst)[e] = static_cast<uint16_t>(words[e / 2] >> 16 * (e & 1));
                        }
                }
            }
        }
    } else {
        Item *dst = static_cast<Item *>(p.out) + static_cast<size_t>(x.n0 + g) * p.ldo + r0 + lane;
        const int rows = r0 + lane < p.n ? x.nr - g : 0;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 s = *reinterpret_cast<const float4 *>(s_rx + j);
            const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i, dst += p.ldo)
                if (j + i < rows) *dst = item(__int_as_float(v[j + i]) * (rw * f[i]));
        }
    }
}
template <int OUT>
__device__ __forceinline__ bool out_in_pieces(const GemmArgs &p) {
    return ((reinterpret_cast<uintptr_t>(p.out) | p.ldo * (OUT == COLI_ACT_F32 ? 4 : 2)) & 15) == 0;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, int (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "r"(taddr) : "memory");
}
// Split k over the C CTAs of a cluster.  A tile's columns go in pieces of 8, `per` of them to each CTA in turn: every CTA
// sends its sums of the others' pieces by stores that count on the owner's barrier as they land (no fence), adds
// what comes in for its own, and stores those.  `part`: [C - 1 senders][2 per halves of a piece][128 weight rows] of 16 bytes.
// pfull waits for every warp of the cluster, a CTA that owns nothing included: one that ran ahead could complete another's
// pfree twice before that looked at it.  tl counts the tiles; `last`: none follows.  One epilogue warp's 32 weight rows; false
// when a wait gave up.
template <int OUT>
__device__ __forceinline__ bool split_tile(const GemmArgs &p, const Tile &x, uint32_t dt, int C, int rank, int q, float rw, uint32_t tl, bool last,
                                           unsigned char *buf, bool vec, unsigned char *part, uint64_t *pfull, uint64_t *pfree, volatile int *abort) {
    const int lane = threadIdx.x & 31, row = 32 * q + lane;
    const int pieces = (x.nr + 7) / 8, per = (pieces + C - 1) / C;
    const int lo = min(rank * per, pieces), own = min(pieces - lo, per);
    if (lane == 0) mbar_expect_tx(smem_u32(pfull), (C - 1) * 32 * 32 * own);  // this warp's rows
    if (tl > 0 && !__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(pfree), (tl & 1) ^ 1, abort, p.err))) return false;
    for (int i = 0; i < pieces; ++i) {
        const int to = i / per;
        if (to == rank) continue;
        int v[8];
        tmem_ld8(dt + 8 * i, v);
        const int unit = (rank < to ? rank : rank - 1) * 2 * per + 2 * (i - to * per);
        const uint32_t dst = map_rank(smem_u32(part) + (unit * 128 + row) * 16, to), bar = map_rank(smem_u32(pfull), to);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                         ::"r"(dst + h * 2048), "r"(v[4 * h]), "r"(v[4 * h + 1]), "r"(v[4 * h + 2]), "r"(v[4 * h + 3]), "r"(bar) : "memory");
    }
    if (lane < C && lane != rank) remote_arrive(map_rank(smem_u32(pfull), lane));
    if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(pfull), tl & 1, abort, p.err))) return false;
    for (int i = 0; i < own; ++i) {
        int v[8];
        tmem_ld8(dt + 8 * (lo + i), v);
        for (int c = 0; c < C - 1; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int4 f = *reinterpret_cast<const int4 *>(part + ((c * 2 * per + 2 * i + h) * 128 + row) * 16);
                v[4 * h] += f.x;
                v[4 * h + 1] += f.y;
                v[4 * h + 2] += f.z;
                v[4 * h + 3] += f.w;
            }
        store_run<OUT>(p, x, v, 8 * (lo + i), x.m * 128 + 32 * q, rw, buf, vec);
    }
    __syncwarp();
    if (lane < C && lane != rank && !last) remote_arrive(map_rank(smem_u32(pfree), lane));
    return true;
}

template <int NT, int OUT, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) i8_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {
    using P = Plan<NT, SPLIT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES;
    __shared__ __align__(8) uint64_t bars[2 * P::S + 7];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_tiles;
    __shared__ TileList list;
    __shared__ int s_scan[THREADS / 32];
    uint64_t *full = bars, *empty = full + P::S;
    uint64_t *dfull = empty + P::S, *dempty = dfull + 2, *drain = dempty + 2;
    uint64_t *pfull = drain + 1, *pfree = pfull + 1;  // split k: partial sums there; their place free again
    unsigned char *part = sb + P::S * P::B_BYTES;
    // split k: the CTAs of a cluster take a share of the k-blocks each
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
        mbar_init(smem_u32(pfull), C * N_EPI);
        mbar_init(smem_u32(pfree), (C > 1 ? C - 1 : 1) * N_EPI);
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
        unsigned char *buf = part + P::PART + q * WARP_BUF;
        const bool vec = out_in_pieces<OUT>(p);
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
            if (SPLIT && C > 1) {
                if (!split_tile<OUT>(p, x, dt, C, rank, q, rw, tl, t + stride >= ntiles, buf, vec, part, pfull, pfree, abort)) break;
            } else {
                int g = 0;
                for (; x.nr - g > 8; g += 32) {
                    int v[32];
                    tmem_ld32(dt + g, v);
                    store_run<OUT>(p, x, v, g, x.m * 128 + 32 * q, rw, buf, vec);
                }
                if (g < x.nr) {
                    int v[8];
                    tmem_ld8(dt + g, v);
                    store_run<OUT>(p, x, v, g, x.m * 128 + 32 * q, rw, buf, vec);
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
//
// Split k (SPLIT): the C pairs of a cluster share a tile's k-blocks.  Columns go in runs of 32, run g to pair g % C: every
// CTA sends its sums of the others' runs to the CTA there that has the same weight rows, adds what comes in for its
// own, and stores those.  The ring takes them in: nothing else uses it any more when a CTA says that it may be written to.
constexpr int P_THREADS = (W_EPI0 + P_EPI) * 32;
constexpr int RUN_BYTES = 128 * 32 * 4;  // a run's sums of a CTA's weight rows

struct PairPlan {
    static constexpr int B_BYTES = P_NT / 2 * KB;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int S = (216 * 1024 - P_EPI * WARP_BUF) / STAGE;
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + P_EPI * WARP_BUF + 1024;
    static_assert((MAX_SPLIT - 1) * (P_NT / 32 / MAX_SPLIT) * RUN_BYTES <= S * STAGE && P_NT / 32 / 2 * RUN_BYTES <= S * STAGE, "a split's sums fit the ring");
};

template <int OUT, bool SPLIT>
__global__ void __launch_bounds__(P_THREADS, 1) i8_pair_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {  // clusters of 2 C CTAs
    using P = PairPlan;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // the same offset in all CTAs of the cluster: the dynamic array starts at the same address in each
    unsigned char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES, *sout = sb + P::S * P::B_BYTES;
    __shared__ __align__(8) uint64_t bars[2 * P::S + 7];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_tiles;
    __shared__ TileList list;
    __shared__ int s_scan[P_THREADS / 32];
    // full: the leader's, of both CTAs' copies; empty, dfull: in each CTA; dempty: the leader's
    uint64_t *full = bars, *empty = full + P::S, *dfull = empty + P::S, *dempty = dfull + 2, *drain = dempty + 2;
    uint64_t *pready = drain + 1, *pfull = pready + 1;  // split k: the others may be written to; their sums are here
    volatile int *abort = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = static_cast<int>(cluster_rank()), rank = crank & 1, leader = crank & ~1;
    const int C = SPLIT ? static_cast<int>(cluster_size()) >> 1 : 1, part = SPLIT ? crank >> 1 : 0;
    const int first = blockIdx.x / (2 * C), stride = gridDim.x / (2 * C);
    const int MB = (p.n + 255) / 256, KALL = (p.k + KB - 1) / KB;
    const int kb0 = KALL * part / C, KT = KALL * (part + 1) / C - kb0;
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
        mbar_init(smem_u32(pready), C > 1 ? C - 1 : 1);
        mbar_init(smem_u32(pfull), 1);
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
    // A cluster that splits k has one tile; should groups that overlap make more of them than the host counted, all its
    // warps meet before the next one, whose copies need the ring.  A warp that gives up at tile t leaves its loop by way of
    // give_up(): it meets the others as often as they will (the tiles are the same for the whole cluster), so that nobody waits
    // for it at a barrier without a bound; their own waits for what it no longer does run out.
    auto next_tile = [&](int t) {
        if (SPLIT && t != first) cluster_sync_all();
    };
    auto give_up = [&](int t) {
        for (t += stride; SPLIT && t < ntiles; t += stride) next_tile(t);
    };

    if (warp == W_PROD) {
        // ------------------------------------------------------------------ TMA producer
        uint32_t s = 0, phase = 1;
        for (int t = first; t < ntiles; t += stride) {
            next_tile(t);
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int n32 = (x.nr + 31) / 32;                        // N / 32; this CTA's share is 16 * n32 rows
            const int row_lo = x.n0 + rank * 16 * n32;
            for (int kb = kb0; kb < kb0 + KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), phase, abort, p.err))) {
                    give_up(t);
                    goto prod_done;
                }
                const uint32_t fb = map_rank(smem_u32(&full[s]), leader);
                if (elect_one()) {
                    remote_expect_tx(fb, A_BYTES + n32 * 16 * KB);
                    pair_load_3d(smem_u32(sa + s * A_BYTES), &maps.a, kb * KB, x.m * 256 + rank * 128, x.e, fb);
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
        const uint16_t both = static_cast<uint16_t>(3 << leader);
        for (int t = first; t < ntiles; t += stride, ++tl) {
            next_tile(t);
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int n32 = (x.nr + 31) / 32, acc = tl & 1;
            const uint32_t idesc = idesc_i8(256) | (static_cast<uint32_t>(4 * n32) << 17);
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&dempty[acc]), ((tl >> 1) & 1) ^ 1, abort, p.err))) {
                give_up(t);
                goto mma_done;
            }
            tc_fence_after();
            const uint32_t dt = tbase + acc * P_NT;
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&full[s]), phase, abort, p.err))) {
                    give_up(t);
                    goto mma_done;
                }
                tc_fence_after();
                const int steps = min(4, (p.k - (kb0 + kb) * KB + 31) / 32);
                if (elect_one()) {
                    const uint64_t ad = adesc0 + static_cast<uint64_t>(s * (A_BYTES >> 4)), bd = bdesc0 + static_cast<uint64_t>(s * (P::B_BYTES >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < steps) mma_i8<2>(dt, ad + 2 * kk, bd + 2 * kk, idesc, (kb | kk) != 0);
                    pair_commit(smem_u32(&empty[s]), both);
                }
                __syncwarp();
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (elect_one()) pair_commit(smem_u32(&dfull[acc]), both);
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
    } else if (warp == W_MMA) {
        if (SPLIT)
            for (int t = first; t < ntiles; t += stride) next_tile(t);
    } else {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - W_EPI0) >> 2;  // TMEM lane quarter; every other of this CTA's runs
        unsigned char *buf = sout + (warp - W_EPI0) * WARP_BUF;
        const bool vec = out_in_pieces<OUT>(p);
        uint32_t tl = 0;
        for (int t = first; t < ntiles; t += stride, ++tl) {
            next_tile(t);
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int acc = tl & 1, row0 = x.m * 256 + rank * 128;
            const int r = row0 + 32 * q + lane, runs = (x.nr + 31) / 32;
            const float rw = p.wscale && r < p.n ? __ldg(p.wscale + static_cast<size_t>(x.e) * p.wscale_stride + r) : 1.f;
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&dfull[acc]), (tl >> 1) & 1, abort, p.err))) {
                give_up(t);
                break;
            }
            tc_fence_after();
            const uint32_t dt = tbase + acc * P_NT + (static_cast<uint32_t>(32 * q) << 16);
            const int own = runs > part ? (runs - part + C - 1) / C : 0;  // this CTA's runs
            if (SPLIT) {
                if (warp == W_EPI0) {
                    // nothing reads or writes this CTA's ring any more: the products have been made, the copies came before them
                    if (lane == 0) mbar_expect_tx(smem_u32(pfull), (C - 1) * own * RUN_BYTES);
                    __syncwarp();
                    if (lane < C && lane != part) remote_arrive(map_rank(smem_u32(pready), 2 * lane + rank));
                    __syncwarp();
                }
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(pready), tl & 1, abort, p.err))) {
                    give_up(t);
                    break;
                }
                for (int g = half; g < runs; g += 2) {
                    const int to = g % C;
                    if (to == part) continue;
                    int v[32];
                    tmem_ld32(dt + 32 * g, v);
                    const int slot = (part < to ? part : part - 1) * ((runs - to + C - 1) / C) + g / C;
                    const uint32_t dst = map_rank(smem_u32(sm) + slot * RUN_BYTES + (32 * q + lane) * 128, 2 * to + rank), bar = map_rank(smem_u32(pfull), 2 * to + rank);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                                     ::"r"(dst + ((i ^ (lane & 7)) << 4)), "r"(v[4 * i]), "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3]), "r"(bar) : "memory");
                }
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(pfull), tl & 1, abort, p.err))) {
                    give_up(t);
                    break;
                }
            }
            for (int i = half; i < own; i += 2) {
                const int g = 32 * (part + i * C);
                int v[32];
                tmem_ld32(dt + g, v);
                if (SPLIT)
                    for (int c = 0; c < C - 1; ++c) {
                        const int4 *from = reinterpret_cast<const int4 *>(sm + (c * own + i) * RUN_BYTES + (32 * q + lane) * 128);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int4 f = from[j ^ (lane & 7)];
                            v[4 * j] += f.x;
                            v[4 * j + 1] += f.y;
                            v[4 * j + 2] += f.z;
                            v[4 * j + 3] += f.w;
                        }
                    }
                store_run<OUT>(p, x, v, g, row0 + 32 * q, rw, buf, vec);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive(map_rank(smem_u32(&dempty[acc]), leader));
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

// Groups that have rows, and chunks of at most nt rows of one group, at most.
long groups_of(const GemmArgs &g) { return g.rows < g.E ? g.rows : g.E; }
long chunks_of(const GemmArgs &g, int nt) { return (g.rows - groups_of(g)) / nt + groups_of(g); }

template <int OUT>
cudaError_t launch_gemm(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<128, false>;
    auto kernel = i8_gemm_kernel<128, OUT, false>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const long tiles = chunks_of(g, 128) * ((g.n + 127) / 128);
    const int sms = device_sm_count();
    return launch_early(kernel, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), THREADS, P::SMEM, st, 1, maps, g);
}

// Tiles of 128 weight rows x at most NT rows, their k-blocks split over clusters of 1, 2 or 4 CTAs, whichever leaves the busiest
// CTA the least.
template <int OUT, int NT>
cudaError_t launch_split(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<NT, true>;
    auto kernel = i8_gemm_kernel<NT, OUT, true>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count(), kt = (g.k + KB - 1) / KB;
    const int tiles = static_cast<int>(chunks_of(g, NT) * ((g.n + 127) / 128));
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

template <int OUT, bool SPLIT>
cudaError_t launch_pair(const GemmMaps &maps, const GemmArgs &g, int C, cudaStream_t st) {
    using P = PairPlan;
    auto kernel = i8_pair_kernel<OUT, SPLIT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const long tiles = chunks_of(g, P_NT) * ((g.n + 255) / 256), clusters = SPLIT ? tiles : device_sm_count() / 2;
    return launch_early(kernel, dim3(2 * C * static_cast<unsigned>(tiles < clusters ? tiles : clusters)), P_THREADS, P::SMEM, st, 2 * C, maps, g);
}

// Which tiles.  Split k costs 2 to 3 us and pays from SPLIT_KT k-blocks on: 40 / 64 / 128 rows, 4096 x 6144, in 9.6 / 10.2 / 12.8 us on
// single CTAs against 15.0 / 15.2 / 16.4 on pairs unsplit; 256 / 512 rows, two pairs to a tile, 18 / 20 us against 21 / 22;
// but 40 rows, 6144 x 2048, 8.9 against 8.2.  (Four pairs to a tile: clusters of 8 do not all fit at once, 30 us against 21.)
// Pairs against single CTAs with 64 matrices of 6144 x 2048, 16 / 32 / 64 / 128 rows each: 137 / 140 / 148 / 163 us against 134 /
// 139 / 154 / 243; 2048 x 1024, 8 / 32 rows: 26.7 / 28.1 against 26.0 / 31.0.
constexpr int PAIR_ROWS = 32, SPLIT_KT = 20;

template <int OUT>
cudaError_t launch_out(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    if (g.rows <= 32) return launch_split<OUT, 32>(maps, g, st);
    const int sms = device_sm_count(), kt = (g.k + KB - 1) / KB;
    const long small = chunks_of(g, 128) * ((g.n + 127) / 128), tiles = chunks_of(g, P_NT) * ((g.n + 255) / 256);
    if (kt >= SPLIT_KT && small <= cluster_count(4, sms)) return launch_split<OUT, 128>(maps, g, st);
    if (kt >= SPLIT_KT && tiles <= cluster_count(4, sms)) return launch_pair<OUT, true>(maps, g, 2, st);
    if (g.rows / groups_of(g) < PAIR_ROWS && small >= sms) return launch_gemm<OUT>(maps, g, st);
    return launch_pair<OUT, false>(maps, g, 1, st);
}

}  // namespace

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
    return p.out_type == COLI_ACT_F32 ? launch_out<COLI_ACT_F32>(maps, g, st) : launch_out<COLI_ACT_BF16>(maps, g, st);
}

}  // namespace coli
