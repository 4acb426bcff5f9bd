// fp4_gemm.cu -- products of microscaled 4-bit operands on the 5th-generation tensor cores
// (coli_moe_fp4_product, and the expert products of the layer over 4-bit records).
//
// out[i][j] = rx[i] * rw[j] * sum_b sx[i][b] * sw[j][b] * sum_{k in block b} x[i][k] * w[j][k]
// The block scales are applied by the tensor core (tcgen05.mma with block scales from tensor
// memory), the row scales by the epilogue; sums are float32.
//
// Swap-AB: 128 weight rows of one matrix are the MMA's M side, up to NT rows of the matrix's group
// its N side, so a weight tile is fetched once per NT rows.  Few rows per matrix are the rule (a
// batch spread over many experts): the kernel is then a stream of weights from HBM, and the ring of
// k-blocks (128 x 128 bytes of codes and their scales) is what keeps it full.
//
// One persistent CTA per SM, warp-specialised; tiles (matrix, 128 weight rows, chunk of rows; the
// chunk fastest, so that a weight tile's second use comes from L2) are taken round-robin:
//   warp 0      TMA producer: weight codes (128-byte swizzle), their scale tiles (one bulk copy: the
//               tiles of a k-block are adjacent), and the rows' codes.
//   warp 1      MMA issuer: copies the k-block's scales from shared to tensor memory
//               (tcgen05.cp, 128 rows x 4 scales each) and issues 4 MMAs of K = 64.
//   warp 2      scales of the rows: 4 bytes at a time from their rows into the tile order that
//               tcgen05.cp reads, asynchronously, LAG k-blocks ahead of the fence that publishes them.
//   warps 4-7   epilogue, from two accumulators: one drains while the other fills.
// Tensor memory: accumulators at columns [0, 256), scale stage s at 256 + s * SF_COLS.  A scale
// stage goes with a ring stage, so it is written again only after the MMAs that read it have
// completed (the ring's empty barrier).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"
#include "internal.h"
#include "tc_ptx.h"

namespace coli {

namespace {

constexpr int A_BYTES = 128 * 128;       // weight codes of a k-block
constexpr int MAX_MATS = 1025;           // 1024 and a shared one
constexpr int NBOX = 5;                  // box heights 16 << i rows
constexpr int W_PROD = 0, W_MMA = 1, W_SF = 2, W_EPI0 = 4, N_EPI = 4;
constexpr int THREADS = 8 * 32;
constexpr int LAG = 2;                   // k-blocks between a row-scale copy and its publication

template <int FMT> struct Sf;            // scales of a k-block
template <> struct Sf<COLI_FP4_NV> { static constexpr int ATOMS = 4; };  // 64 elements per 4 scales
template <> struct Sf<COLI_FP4_MX> { static constexpr int ATOMS = 2; };  // 128 elements per 4 scales

template <int FMT, int NT>
struct Plan {
    static constexpr int ATOMS = Sf<FMT>::ATOMS;
    static constexpr int B_BYTES = NT * 128;
    static constexpr int SFA_BYTES = ATOMS * 512;
    static constexpr int HALVES = (NT + 127) / 128;           // 128-row pieces of the N side
    static constexpr int SFB_BYTES = ATOMS * 512 * HALVES;
    static constexpr int STAGE = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int SF_COLS = ATOMS * 4 * (1 + HALVES);
    static constexpr int FIT = (220 * 1024) / STAGE, TFIT = 256 / SF_COLS;
    static constexpr int S = FIT < TFIT ? FIT : TFIT;         // ring stages
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + 1024;
    static_assert(S > LAG, "the publication lags behind the copies by less than the ring");
};

// Instruction descriptor of block-scaled e2m1 products: A and B e2m1 (bits 7-9, 10-11 = 1), both
// K-major, scales ue4m3 (bit 23 = 0) or ue8m0 (1), M = 128 (bits 27-28 = M >> 7); N >> 3 goes to
// bits 17-22, which scale byte of a 32-bit word comes first to bits 4-5 (B) and 29-30 (A).
template <int FMT>
__device__ __forceinline__ constexpr uint32_t idesc_fp4() {
    return (1u << 7) | (1u << 10) | (FMT == COLI_FP4_MX ? 1u << 23 : 0u) | (1u << 27);
}

template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (FMT == COLI_FP4_NV)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// 128 rows x 4 scales (512 bytes in shared memory: row r at (r % 32) * 16 + (r / 32) * 4) to 4 columns
// of tensor memory, the same in all four lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// 32 rows of 16 bytes without swizzle: 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sf(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// 4 bytes, or 4 zero bytes
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

struct GemmArgs {
    const uint8_t *wsf, *wsf_shared;         // scale tiles
    size_t wsf_stride;
    const float *wrow, *wrow_shared;
    size_t wrow_stride;
    const uint8_t *xsf;
    const float *xrow;
    const int32_t *offsets;
    int E, S;                                // matrices; 1: a shared one for the rows behind the groups
    int rows, n, k;
    void *out;
    size_t ldo;
    int *err;
};
struct GemmMaps {
    CUtensorMap a, as;     // weight codes {k / 2 bytes, n rows, matrices}
    CUtensorMap b[NBOX];   // row codes {k / 2 bytes, rows}
};

struct Tile {
    int e, m, n0, nr;      // matrix, block of 128 weight rows, first row, rows
};

// First row and row count of matrix e's group; count -1 when the offsets are not ascending in range.
__device__ __forceinline__ void group_rows(const GemmArgs &p, int e, int &lo, int &cnt) {
    lo = 0;
    cnt = p.rows;
    if (p.offsets) {
        lo = __ldg(p.offsets + e);
        const int hi = e < p.E ? __ldg(p.offsets + e + 1) : p.rows;
        cnt = lo < 0 || hi < lo || hi > p.rows ? -1 : hi - lo;
    }
}

// Tile t of the list; s_first[e]: tiles before matrix e.
template <int NT>
__device__ __forceinline__ Tile tile_at(int t, const int *s_first, const GemmArgs &p, int W) {
    int lo = 0, hi = W;  // the last e with s_first[e] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= t) lo = mid;
        else hi = mid;
    }
    Tile x;
    x.e = lo;
    int row0, cnt;
    group_rows(p, lo, row0, cnt);
    const int nch = (cnt + NT - 1) / NT;
    const int per = ((cnt + nch - 1) / nch + 15) & ~15;  // rows of a chunk: even shares
    const int i = t - s_first[lo];
    x.m = i / nch;
    const int c = i - x.m * nch;
    x.n0 = row0 + c * per;
    x.nr = min(per, cnt - c * per);
    return x;
}

template <int FMT, int NT, int OUT>
__global__ void __launch_bounds__(THREADS, 1) fp4_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {
    using P = Plan<FMT, NT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES, *ssa = sb + P::S * P::B_BYTES, *ssb = ssa + P::S * P::SFA_BYTES;
    __shared__ __align__(8) uint64_t bars[3 * P::S + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_first[MAX_MATS], s_scan[THREADS / 32];
    uint64_t *full = bars, *sfull = full + P::S, *empty = sfull + P::S;
    uint64_t *dfull = empty + P::S, *dempty = dfull + 2, *drain = dempty + 2;
    volatile int *abort = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int MB = (p.n + 127) / 128, KT = (p.k + FP4_KB - 1) / FP4_KB;
    const int W = p.E + p.S;

    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), 512);
    if (threadIdx.x == 32) {
        for (int i = 0; i < P::S; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&sfull[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&dfull[i]), 1);
            mbar_init(smem_u32(&dempty[i]), N_EPI * 32);
        }
        mbar_init(smem_u32(drain), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // the tile list: an exclusive scan of the matrices' tiles
    int carry = 0;
    for (int base = 0; base < W; base += THREADS) {
        const int e = base + threadIdx.x;
        int lo = 0, cnt = 0;
        if (e < W) group_rows(p, e, lo, cnt);
        if (cnt < 0) {
            cnt = 0;
            if (blockIdx.x == 0) atomicOr(p.err, COLI_DEVERR_GROUPING);
        }
        const int tiles = (cnt + NT - 1) / NT * MB;
        int inc = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < THREADS / 32; ++w) {
            const int v = s_scan[w];
            if (w < warp) before += v;
            carry += v;
        }
        if (e < W) s_first[e] = before + inc - tiles;
        __syncthreads();
    }
    const int ntiles = carry;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = s_tmem;

    if (warp == W_PROD) {
        // ------------------------------------------------------------------ TMA producer
        // lane 0: weight codes and their scales; lane i < NBOX: the box of 16 << (NBOX - 1 - i) rows
        // when that bit of the row count is set
        const size_t mtile = 128 * fp4_pitch(FMT, p.k);  // scale bytes of 128 weight rows
        uint32_t it = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
            const Tile x = tile_at<NT>(t, s_first, p, W);
            const bool shared = x.e >= p.E;
            const CUtensorMap *ta = shared ? &maps.as : &maps.a;
            const int ez = shared ? 0 : x.e;
            const uint8_t *wsf = (shared ? p.wsf_shared : p.wsf + static_cast<size_t>(x.e) * p.wsf_stride) + static_cast<size_t>(x.m) * mtile;
            const int n16 = (x.nr + 15) / 16;
            for (int kb = 0; kb < KT; ++kb, ++it) {
                const int s = it % P::S;
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), ((it / P::S) & 1) ^ 1, abort, p.err))) goto prod_done;
                const uint32_t fb = smem_u32(&full[s]);
                if (lane == 0) mbar_expect_tx(fb, A_BYTES + P::SFA_BYTES + n16 * 16 * 128);
                __syncwarp();
                if (lane == 0) {
                    tma_load_3d(smem_u32(sa + s * A_BYTES), ta, kb * 128, x.m * 128, ez, fb);
                    bulk_load(smem_u32(ssa + s * P::SFA_BYTES), wsf + static_cast<size_t>(kb) * P::SFA_BYTES, P::SFA_BYTES, fb);
                }
                if (lane < NBOX) {
                    const int bit = NBOX - 1 - lane;
                    if ((n16 >> bit) & 1) {
                        const int row0 = 16 * ((n16 >> (bit + 1)) << (bit + 1));  // rows of the larger boxes
                        tma_load_2d(smem_u32(sb + s * P::B_BYTES + row0 * 128), &maps.b[bit], kb * 128, x.n0 + row0, fb);
                    }
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
        uint32_t it = 0, tl = 0;
        const uint64_t adesc0 = smem_desc_sw128(smem_u32(sa)), bdesc0 = smem_desc_sw128(smem_u32(sb));
        const uint64_t sadesc0 = smem_desc_sf(smem_u32(ssa)), sbdesc0 = smem_desc_sf(smem_u32(ssb));
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x, ++tl) {
            const Tile x = tile_at<NT>(t, s_first, p, W);
            const int n16 = (x.nr + 15) / 16;
            const uint32_t idesc = idesc_fp4<FMT>() | (static_cast<uint32_t>(2 * n16) << 17);
            const int acc = tl & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&dempty[acc]), ((tl >> 1) & 1) ^ 1, abort, p.err))) goto mma_done;
            tc_fence_after();
            const uint32_t dt = tbase + acc * 128;
            for (int kb = 0; kb < KT; ++kb, ++it) {
                const int s = it % P::S;
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), (it / P::S) & 1, abort, p.err))) goto mma_done;
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sfull[s]), (it / P::S) & 1, abort, p.err))) goto mma_done;
                tc_fence_after();
                const int steps = min(4, (p.k - kb * FP4_KB + 63) / 64);  // K = 64 steps that hold elements
                if (elect_one()) {
                    const uint32_t sfa = tbase + 256 + s * P::SF_COLS, sfb = sfa + 4 * P::ATOMS;
                    const uint64_t ad = adesc0 + static_cast<uint64_t>(s * (A_BYTES >> 4)), bd = bdesc0 + static_cast<uint64_t>(s * (P::B_BYTES >> 4));
                    const uint64_t sad = sadesc0 + static_cast<uint64_t>(s * (P::SFA_BYTES >> 4)), sbd = sbdesc0 + static_cast<uint64_t>(s * (P::SFB_BYTES >> 4));
#pragma unroll
                    for (int i = 0; i < P::ATOMS; ++i) {
                        sf_copy(sfa + 4 * i, sad + 32 * i);
#pragma unroll
                        for (int h = 0; h < P::HALVES; ++h)
                            sf_copy(sfb + 4 * (i * P::HALVES + h), sbd + 32 * (i * P::HALVES + h));
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk < steps) {
                            const int atom = FMT == COLI_FP4_NV ? kk : kk >> 1;
                            const uint32_t id = FMT == COLI_FP4_NV ? 0u : 2u * (kk & 1);
                            mma_fp4<FMT>(dt, ad + 2 * kk, bd + 2 * kk, idesc | (id << 4) | (id << 29), sfa + 4 * atom, sfb + 4 * P::HALVES * atom, (kb | kk) != 0);
                        }
                    }
                    mma_commit(smem_u32(&empty[s]));
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit(smem_u32(&dfull[acc]));
            __syncwarp();
        }
    mma_done:
        // every MMA issued so far has completed once this commit arrives
        if (elect_one()) mma_commit(smem_u32(drain));
        __syncwarp();
        mbar_drain(smem_u32(drain), 0);
    } else if (warp == W_SF) {
        // ------------------------------------------------------------------ scales of the rows
        const size_t pitch = fp4_pitch(FMT, p.k);
        uint32_t it = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
            const Tile x = tile_at<NT>(t, s_first, p, W);
            const int nr16 = (x.nr + 15) & ~15;
            for (int kb = 0; kb < KT; ++kb, ++it) {
                const int s = it % P::S;
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), ((it / P::S) & 1) ^ 1, abort, p.err))) goto sf_done;
                const uint32_t dst = smem_u32(ssb + s * P::SFB_BYTES);
                for (int r = lane; r < nr16; r += 32) {
                    const bool real = x.n0 + r < p.rows;
                    const uint8_t *src = p.xsf + static_cast<size_t>(real ? x.n0 + r : 0) * pitch + kb * (4 * P::ATOMS);
                    const uint32_t at = dst + (r >> 7) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
#pragma unroll
                    for (int i = 0; i < P::ATOMS; ++i) copy4(at + i * 512 * P::HALVES, src + 4 * i, real);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (it >= LAG) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(LAG) : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sfull[(it - LAG) % P::S]));
                }
            }
        }
    sf_done:
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && !*abort)
            for (uint32_t i = it > static_cast<uint32_t>(LAG) ? it - LAG : 0; i < it; ++i) mbar_arrive(smem_u32(&sfull[i % P::S]));
    } else if (warp >= W_EPI0) {
        // ------------------------------------------------------------------ epilogue
        const int q = warp - W_EPI0;  // TMEM lane quarter (warp % 4)
        uint32_t tl = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x, ++tl) {
            const Tile x = tile_at<NT>(t, s_first, p, W);
            const int acc = tl & 1;
            const int r = x.m * 128 + 32 * q + lane;
            const float *wrow = x.e >= p.E ? p.wrow_shared : (p.wrow ? p.wrow + static_cast<size_t>(x.e) * p.wrow_stride : nullptr);
            const float rw = wrow && r < p.n ? __ldg(wrow + r) : 1.f;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&dfull[acc]), (tl >> 1) & 1, abort, p.err))) break;
            tc_fence_after();
            const uint32_t dt = tbase + acc * 128 + (static_cast<uint32_t>(32 * q) << 16);
            for (int g = 0; g < x.nr; g += 32) {
                int v[32];
                tmem_ld32(dt + g, v);
                const float rx = p.xrow && g + lane < x.nr ? __ldg(p.xrow + x.n0 + g + lane) : 1.f;
                if (OUT == FP4_OUT_SWIGLU) {
                    const bool gate = lane < 16;
                    const int col = (x.m * 128 + 32 * q) / 2 + (lane & 15);
                    float d[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) d[j] = __int_as_float(v[j]) * (rw * __shfl_sync(0xffffffffu, rx, j));
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        // gate lanes take rows 0-15 of the run, up lanes rows 16-31
                        const float other = __shfl_xor_sync(0xffffffffu, gate ? d[16 + i] : d[i], 16);
                        const float gv = gate ? d[i] : other, uv = gate ? other : d[16 + i];
                        const int j = g + (gate ? i : 16 + i);
                        if (j < x.nr && r < p.n)
                            static_cast<__nv_bfloat16 *>(p.out)[static_cast<size_t>(x.n0 + j) * p.ldo + col] = __float2bfloat16_rn(gv / (1.0f + expf(-gv)) * uv);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float y = __int_as_float(v[j]) * (rw * __shfl_sync(0xffffffffu, rx, j));
                        if (g + j < x.nr && r < p.n) {
                            const size_t at = static_cast<size_t>(x.n0 + g + j) * p.ldo + r;
                            if (OUT == FP4_OUT_F32) static_cast<float *>(p.out)[at] = y;
                            else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
                        }
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&dempty[acc]));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Weight codes of `count` matrices, boxes of 128 rows of a k-block.
bool mats_map(CUtensorMap *m, const coli_fp4_mats &w, int k) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k) / 2, static_cast<cuuint64_t>(w.n), static_cast<cuuint64_t>(w.count)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(k) / 2, w.count > 1 ? w.codes_stride : static_cast<cuuint64_t>(w.n) * (k / 2)};
    const cuuint32_t box[3] = {128, 128, 1};
    return encode_u8(m, w.codes, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool rows_maps(CUtensorMap *m, const coli_fp4_rows &a, int k) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k) / 2, static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k) / 2};
    for (int i = 0; i < NBOX; ++i) {
        const cuuint32_t box[2] = {128, 16u << i};
        if (!encode_u8(m + i, a.codes, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
    }
    return true;
}

template <int FMT, int NT, int OUT>
cudaError_t launch_gemm(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<FMT, NT>;
    auto kernel = fp4_gemm_kernel<FMT, NT, OUT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(P::SMEM));
    if (e != cudaSuccess) return e;
    const long chunks = g.rows / NT + (g.rows < g.E + g.S ? g.rows : g.E + g.S);  // at most
    const long tiles = (chunks < 1 ? 1 : chunks) * ((g.n + 127) / 128);
    const int sms = device_sm_count();
    kernel<<<static_cast<int>(tiles < sms ? tiles : sms), THREADS, P::SMEM, st>>>(maps, g);
    return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_fmt(const GemmMaps &maps, const GemmArgs &g, int out_kind, cudaStream_t st) {
    if (out_kind == FP4_OUT_F32) return launch_gemm<FMT, 128, FP4_OUT_F32>(maps, g, st);
    if (out_kind == FP4_OUT_BF16) return launch_gemm<FMT, 128, FP4_OUT_BF16>(maps, g, st);
    return launch_gemm<FMT, 128, FP4_OUT_SWIGLU>(maps, g, st);
}

}  // namespace

cudaError_t launch_fp4_product(int fmt, const Fp4ProductArgs &p, cudaStream_t st) {
    GemmMaps maps;
    bool ok = mats_map(&maps.a, p.w, p.k) && rows_maps(maps.b, p.a, p.k);
    if (ok && p.shared) ok = mats_map(&maps.as, *p.shared, p.k);
    else maps.as = maps.a;
    if (!ok) return cudaErrorInvalidValue;
    GemmArgs g;
    g.wsf = p.w.scales;
    g.wsf_stride = p.w.scales_stride;
    g.wrow = p.w.row_scale;
    g.wrow_stride = p.w.row_scale_stride;
    g.wsf_shared = p.shared ? p.shared->scales : nullptr;
    g.wrow_shared = p.shared ? p.shared->row_scale : nullptr;
    g.xsf = p.a.scales;
    g.xrow = p.a.row_scale;
    g.offsets = p.offsets;
    g.E = p.w.count;
    g.S = p.shared ? 1 : 0;
    g.rows = p.a.rows;
    g.n = p.w.n;
    g.k = p.k;
    g.out = p.out;
    g.ldo = p.ldo;
    g.err = p.err;
    return fmt == COLI_FP4_MX ? launch_fmt<COLI_FP4_MX>(maps, g, p.out_kind, st) : launch_fmt<COLI_FP4_NV>(maps, g, p.out_kind, st);
}

}  // namespace coli
