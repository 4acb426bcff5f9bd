// fp4_gemm.cu -- products of microscaled 4-bit operands on the 5th-generation tensor cores
// (coli_moe_fp4_product, and the expert products of the layer over 4-bit records).
//
// out[i][j] = rx[i] * rw[j] * sum_b sx[i][b] * sw[j][b] * sum_{k in block b} x[i][k] * w[j][k]
// The block scales are applied by the tensor core (tcgen05.mma with block scales from tensor
// memory), the row scales by the epilogue; sums are float32.
//
// Swap-AB: weight rows of one matrix are the MMA's M side, rows of the matrix's group its N side, so a
// weight tile is fetched once for as many rows as a tile has.  Few rows per matrix are the rule (a batch
// spread over many experts): the kernel is then a stream of weights from HBM, and the ring of k-blocks
// (128 x 128 bytes of codes and their scales) is what keeps it full.  Three tiles, chosen on the host:
//   at most 32 rows in all      128 weight rows x 32, k split over a cluster where tiles are few
//   few each (use_pairs)        128 weight rows x 128
//   more                        256 weight rows x 256 on a pair of CTAs
// 64 matrices of 4096 x 6144 (NV) with 1 to 32 rows each stream at 6.4 to 6.9 TB/s (copy peak 6.5); 8192
// rows of one run at 4.4 PFLOP/s (94 us at 1965 MHz; 109 us at 1580 MHz, under the power cap, in long runs).  That is
// 1030 to 1100 cycles per k-block, of which the products need 512; a CTA takes 41 KB from L2 in that time, 37 to
// 40 bytes per cycle.  Which of the operands, the row scales and the single accumulator it waits for is not measured.
//
// One persistent CTA per SM, warp-specialised; tiles are taken round-robin:
//   warp 0      TMA producer: weight codes (128-byte swizzle), their scale tiles (one bulk copy: the
//               tiles of a k-block are adjacent), and the rows' codes.
//   warp 1      MMA issuer: copies the k-block's scales from shared to tensor memory
//               (tcgen05.cp, 128 rows x 4 scales each) and issues 4 MMAs of K = 64.
//   warps 2-3   scales of the rows, every other k-block each: from their rows through registers (the
//               next k-blocks' loads in flight meanwhile) into the tile order that tcgen05.cp reads.
//   warps 4-7   epilogue, from two accumulators: one drains while the other fills (pairs: below).
// Tensor memory: accumulators at columns [0, 256), scale stage s at 256 + s * SF_COLS.  A scale
// stage goes with a ring stage, so it is written again only after the MMAs that read it have
// completed (the ring's empty barrier).
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"
#include "group_tiles.h"
#include "internal.h"
#include "pdl.h"
#include "tc_ptx.h"

namespace coli {

namespace {

constexpr int A_BYTES = 128 * 128;       // weight codes of a k-block
constexpr int W_PROD = 0, W_MMA = 1, W_SF = 2, N_SF = 2, W_EPI0 = 4, N_EPI = 4;
constexpr int THREADS = 8 * 32;

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
    static constexpr int PART = NT <= 32 ? (MAX_SPLIT - 1) * 32 * 128 * 4 : 0;  // split k: the other ranks' sums
    static constexpr int FIT = (216 * 1024 - PART) / STAGE, TFIT = 256 / SF_COLS;
    static constexpr int S = FIT < TFIT ? FIT : TFIT;         // ring stages
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + PART + 1024;
    static_assert(S >= 3, "the ring covers the copies' latency");
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
struct GemmArgs : GroupArgs {
    const uint8_t *wsf, *wsf_shared;         // scale tiles
    size_t wsf_stride;
    const float *wrow, *wrow_shared;
    size_t wrow_stride;
    const uint8_t *xsf;
    const float *xrow;
    int k;
    void *out;
    size_t ldo;
};
struct GemmMaps {
    CUtensorMap a, as;     // weight codes {k / 2 bytes, n rows, matrices}
    CUtensorMap b[NBOX];   // row codes {k / 2 bytes, rows}, boxes of 16 << i rows
    CUtensorMap sf, sfs;   // scale tiles {512 bytes, tiles, matrices} (pairs)
};

// The tensor maps the kernel starts with, on their way before their first use.
__device__ __forceinline__ void prefetch_maps(const GemmMaps &m, int shared) {
    auto one = [](const CUtensorMap *t) { asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(t)) : "memory"); };
    one(&m.a);
    one(&m.b[0]);
    if (shared) one(&m.as);
}

// The same in tensor memory, 8 columns at a time.
__device__ __forceinline__ void split_scales(uint32_t taddr, float pw, float &rx) {
    const float px = halve_exponent(rx);
#pragma unroll 1
    for (int c = 0; c < 32; c += 8) {
        uint32_t v[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "r"(taddr + c) : "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = static_cast<uint32_t>(scaled_sum(static_cast<int>(v[j]), pw, __shfl_sync(0xffffffffu, px, c + j)));
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\ttcgen05.wait::st.sync.aligned;"
                     ::"r"(taddr + c), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    }
}

// SiLU(gate) * up for rows i (gate lanes, 0-15) and 16 + i (up lanes) of a run of 32 rows: the lane
// exchanges the sum it does not use with its partner's.  Rounded to bf16: h is quantised to 4 bits next,
// whose steps are 32 times as wide at least.
__device__ __forceinline__ __nv_bfloat16 swiglu_pair(const int *v, int i, bool gate, float rw, float rx) {
    const float lo = __int_as_float(v[i]) * (rw * __shfl_sync(0xffffffffu, rx, i));
    const float hi = __int_as_float(v[16 + i]) * (rw * __shfl_sync(0xffffffffu, rx, 16 + i));
    const float other = __shfl_xor_sync(0xffffffffu, gate ? hi : lo, 16);
    const float gv = gate ? lo : other, uv = gate ? other : hi;
    return __float2bfloat16_rn(gv / (1.0f + expf(-gv)) * uv);
}

// A run of 32 rows x this warp's 32 weight rows: v holds the sums of weight row r, rx the row scale
// of the run's row `lane`.
template <int OUT>
__device__ __forceinline__ void store_run(const GemmArgs &p, const Tile &x, const int *v, int g, int r, float rw, float rx, int lane) {
    if (OUT == FP4_OUT_SWIGLU) {
        const bool gate = lane < 16;
        const int col = (r >> 5) * 16 + (lane & 15);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __nv_bfloat16 h = swiglu_pair(v, i, gate, rw, rx);
            const int j = g + (gate ? i : 16 + i);
            if (j < x.nr && r < p.n) static_cast<__nv_bfloat16 *>(p.out)[static_cast<size_t>(x.n0 + j) * p.ldo + col] = h;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (g + j >= x.nr) break;  // the same for the whole warp
            const float y = __int_as_float(v[j]) * (rw * __shfl_sync(0xffffffffu, rx, j));
            if (r < p.n) {
                const size_t at = static_cast<size_t>(x.n0 + g + j) * p.ldo + r;
                if (OUT == FP4_OUT_F32) static_cast<float *>(p.out)[at] = y;
                else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y);
            }
        }
    }
}

// Row-scale warp `w` of N_SF: its k-blocks' scales of up to NT rows, from their rows (4 * ATOMS bytes
// each) to the tile order of tcgen05.cp.  A lane takes rows lane + 32 c of each 128: word j of its four rows is
// one 16-byte piece of tile j, so a k-block of 128 rows is ATOMS stores of 16 bytes per lane (shared memory is
// nearly used up by the products' operands: 4-byte stores, four times as many, kept a warp busy for 780 cycles per
// k-block of 256 rows, longer than the products then took).  Rows behind the tile's last repeat a row
// that exists: what they give is not stored by the epilogue.  publish(stage) tells the MMA warp.
template <int FMT, int NT, typename Publish>
__device__ __forceinline__ void row_scales(const GemmArgs &p, int w, int first, int stride, int ntiles, int KT, const TileList &list, int W,
                                           unsigned char *ssb, uint64_t *empty, int S, int kb0, volatile int *abort, Publish publish) {
    constexpr int ATOMS = Sf<FMT>::ATOMS, HALVES = (NT + 127) / 128, SLOTS = NT <= 32 ? 1 : 4 * HALVES;
    const int lane = threadIdx.x & 31;
    const size_t pitch = fp4_pitch(FMT, p.k);
    const uint32_t dst0 = smem_u32(ssb) + lane * 16;
    // DEPTH k-blocks of this warp in registers: a buffer is loaded again, for the k-block DEPTH turns on,
    // as soon as it has been stored (buffers are named by the unrolled loop: a copy from one to another
    // would wait for its loads)
    constexpr int DEPTH = 3;
    uint32_t v[DEPTH][SLOTS][ATOMS];
    // the cursor of the loads: tile, k-block, the slots' addresses
    int t = first, kb = w;
    const uint8_t *src[SLOTS];
    bool upper = false;  // the tile has more than 128 rows
    auto tile = [&]() {
        if (t >= ntiles) return;
        const Tile x = tile_at<NT>(t, list, p, W);
        upper = x.nr > 128;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) src[i] = p.xsf + static_cast<size_t>(x.n0 + min(32 * i + lane, x.nr - 1)) * pitch;
    };
    auto step = [&]() {  // to the tile that holds k-block kb
        if (kb < KT) return;
        do {
            kb -= KT;
            t += stride;
        } while (kb >= KT && t < ntiles);
        tile();
    };
    auto load = [&](uint32_t (&d)[SLOTS][ATOMS]) {
        if (t < ntiles) {
            const int off = (kb0 + kb) * (4 * ATOMS);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                if (i < 4 || upper) {
                    if (ATOMS == 4) {
                        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(src[i] + off));
                        d[i][0] = q.x; d[i][1] = q.y; d[i][ATOMS - 2] = q.z; d[i][ATOMS - 1] = q.w;
                    } else {
                        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(src[i] + off));
                        d[i][0] = q.x; d[i][1] = q.y;
                    }
                }
            }
        }
        kb += N_SF;
        step();
    };
    tile();
    step();
    // k-blocks of this warp: every N_SF-th of the CTA's
    const uint32_t all = first < ntiles ? static_cast<uint32_t>((ntiles - first + stride - 1) / stride) * KT : 0u;
#pragma unroll
    for (int b = 0; b < DEPTH; ++b) load(v[b]);
    uint32_t s = w, phase = 1;
    for (uint32_t it = w; it < all;) {
#pragma unroll
        for (int b = 0; b < DEPTH; ++b) {
            if (it >= all) return;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), phase, abort, p.err))) return;
            const uint32_t dst = dst0 + s * (ATOMS * 512 * HALVES);
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
#pragma unroll
                for (int j = 0; j < ATOMS; ++j)
                    if (SLOTS == 1) asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + j * 512), "r"(v[b][0][j]) : "memory");
                    else asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                                 ::"r"(dst + (j * HALVES + h) * 512), "r"(v[b][4 * h][j]), "r"(v[b][(4 * h + 1) % SLOTS][j]), "r"(v[b][(4 * h + 2) % SLOTS][j]), "r"(v[b][(4 * h + 3) % SLOTS][j]) : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) publish(s);
            load(v[b]);
            it += N_SF;
            s += N_SF;
            if (s >= static_cast<uint32_t>(S)) {
                s -= S;
                phase ^= 1;
            }
        }
    }
}

__device__ __forceinline__ int add_floats(int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }

template <int FMT, int NT, int OUT>
__global__ void __launch_bounds__(THREADS, 1) fp4_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {
    using P = Plan<FMT, NT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES, *ssa = sb + P::S * P::B_BYTES, *ssb = ssa + P::S * P::SFA_BYTES;
    constexpr bool SPLIT = NT <= 32;
    __shared__ __align__(8) uint64_t bars[2 * P::S + 7];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_tiles;
    __shared__ TileList list;
    __shared__ int s_scan[THREADS / 32];
    uint64_t *full = bars, *empty = full + P::S;
    uint64_t *dfull = empty + P::S, *dempty = dfull + 2, *drain = dempty + 2;
    uint64_t *pfull = drain + 1, *pfree = pfull + 1;  // split k: partial sums there; their place free again
    float *part = reinterpret_cast<float *>(ssb + P::S * P::SFB_BYTES);
    // split k: the CTAs of a cluster take a share of the k-blocks each; rank 0 adds and stores
    const int C = SPLIT ? static_cast<int>(cluster_size()) : 1, rank = SPLIT ? static_cast<int>(cluster_rank()) : 0;
    const int first = blockIdx.x / C, stride = gridDim.x / C;
    volatile int *abort = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int MB = (p.n + 127) / 128, KALL = (p.k + FP4_KB - 1) / FP4_KB;
    const int kb0 = KALL * rank / C, KT = KALL * (rank + 1) / C - kb0;
    const int W = p.E + p.S;

    if (threadIdx.x == 32) {
        for (int i = 0; i < P::S; ++i) {
            mbar_init(smem_u32(&full[i]), 2);  // the producer and a row-scale warp
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
    if (warp == W_SF) tmem_alloc(smem_u32(&s_tmem), 512);
    if (warp == W_PROD && elect_one()) prefetch_maps(maps, p.S);
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
        // one elected lane issues with warp-uniform operands: weight codes, their scales, and a box of
        // 16 << i rows for every bit i of the row count (from lanes that differ, or behind a test of the
        // lane, a copy took the compiler's loop over lanes and 200 cycles)
        const size_t mtile = 128 * fp4_pitch(FMT, p.k);  // scale bytes of 128 weight rows
        uint32_t it = 0, s = 0, phase = 1;
        for (int t = first; t < ntiles; t += stride) {
            const Tile x = tile_at<NT>(t, list, p, W);
            const bool shared = x.e >= p.E;
            const CUtensorMap *ta = shared ? &maps.as : &maps.a;
            const int ez = shared ? 0 : x.e;
            const uint8_t *wsf = (shared ? p.wsf_shared : p.wsf + static_cast<size_t>(x.e) * p.wsf_stride) + static_cast<size_t>(x.m) * mtile;
            const int n16 = (x.nr + 15) / 16;
            for (int kb = 0; kb < KT; ++kb, ++it) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), phase, abort, p.err))) goto prod_done;
                const uint32_t fb = smem_u32(&full[s]);
                if (elect_one()) {
                    mbar_expect_tx(fb, A_BYTES + P::SFA_BYTES + n16 * 16 * 128);
                    tma_load_3d(smem_u32(sa + s * A_BYTES), ta, (kb0 + kb) * 128, x.m * 128, ez, fb);
                    bulk_load(smem_u32(ssa + s * P::SFA_BYTES), wsf + static_cast<size_t>(kb0 + kb) * P::SFA_BYTES, P::SFA_BYTES, fb);
#pragma unroll
                    for (int bit = NT <= 32 ? 1 : NBOX - 1; bit >= 0; --bit) {
                        const int row0 = 16 * ((n16 >> (bit + 1)) << (bit + 1));  // rows of the larger boxes
                        if ((n16 >> bit) & 1) tma_load_2d(smem_u32(sb + s * P::B_BYTES + row0 * 128), &maps.b[bit], (kb0 + kb) * 128, x.n0 + row0, fb);
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
        const uint64_t sadesc0 = smem_desc_sf(smem_u32(ssa)), sbdesc0 = smem_desc_sf(smem_u32(ssb));
        for (int t = first; t < ntiles; t += stride, ++tl) {
            const Tile x = tile_at<NT>(t, list, p, W);
            const int n16 = (x.nr + 15) / 16;
            const uint32_t idesc = idesc_fp4<FMT>() | (static_cast<uint32_t>(2 * n16) << 17);
            const int acc = tl & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&dempty[acc]), ((tl >> 1) & 1) ^ 1, abort, p.err))) goto mma_done;
            tc_fence_after();
            const uint32_t dt = tbase + acc * 128;
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), phase, abort, p.err))) goto mma_done;
                tc_fence_after();
                const int steps = min(4, (p.k - (kb0 + kb) * FP4_KB + 63) / 64);  // K = 64 steps that hold elements
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
    } else if (warp < W_EPI0) {
        // ------------------------------------------------------------------ scales of the rows
        row_scales<FMT, NT>(p, warp - W_SF, first, stride, ntiles, KT, list, W, ssb, empty, P::S, kb0, abort,
                            [&](int st) { mbar_arrive(smem_u32(&full[st])); });
    } else {
        // ------------------------------------------------------------------ epilogue
        const int q = warp - W_EPI0;  // TMEM lane quarter (warp % 4)
        uint32_t tl = 0;
        if (SPLIT && C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        for (int t = first; t < ntiles; t += stride, ++tl) {
            const Tile x = tile_at<NT>(t, list, p, W);
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
                if (SPLIT && C > 1) {
                    if (!split_sum(v, x.nr, C, rank, q, lane, tl, t + stride >= ntiles, part, pfull, pfree, abort, p.err, add_floats)) break;
                    if (rank != 0) break;
                }
                float rx = p.xrow && g + lane < x.nr ? __ldg(p.xrow + x.n0 + g + lane) : 1.f, rwg = rw;
                if (!__all_sync(0xffffffffu, ordinary(rw) && ordinary(rx))) {
                    const float pw = halve_exponent(rwg);
                    split_scales(v, pw, rx);
                }
                store_run<OUT>(p, x, v, g, r, rwg, rx, lane);
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
    if (warp == W_SF) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// ------------------------------------------------------------------ CTA pairs --------------
// The same product with tiles of 256 weight rows x up to 256 rows on a pair of CTAs
// (cta_group::2): each CTA fetches its own 128 weight rows and half of the tile's rows, the tensor
// cores read both halves, so a byte of shared memory feeds twice the products of a 128 x 128 tile.
// Both CTAs hold the scales of all rows of the tile.  One accumulator of 256 columns per CTA; the
// epilogue's eight warps take it whole into registers before they store, so that the next
// tile's products wait for the reads alone.
constexpr int P_THREADS = (4 + P_EPI) * 32;

constexpr int P_OUT = 8192;              // bytes of an epilogue half's staging buffer

template <int FMT>
struct PairPlan {
    static constexpr int ATOMS = Sf<FMT>::ATOMS;
    static constexpr int B_BYTES = P_NT / 2 * 128;
    static constexpr int SFA_BYTES = ATOMS * 512, SFB_BYTES = ATOMS * 1024;
    static constexpr int STAGE = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int SF_COLS = ATOMS * 12;
    static constexpr int FIT = (216 * 1024 - 2 * P_OUT) / STAGE, TFIT = 256 / SF_COLS;
    static constexpr int S = FIT < TFIT ? FIT : TFIT;
    static constexpr size_t SMEM = static_cast<size_t>(S) * STAGE + 2 * P_OUT + 1024;
    static_assert(S >= 3, "the ring covers the copies' latency");
};

// A run of RUN rows x this CTA's 128 weight rows (64 columns of h with SwiGLU) through shared memory:
// lanes hold a weight row each, out wants weight rows side by side.  Stored straight from the lanes, 2
// bytes each, a tile's epilogue took 21,000 cycles against 12,000 of its products at k = 6144.
// `buf`: the half's P_OUT bytes; vec: 16-byte stores are aligned.
template <int OUT>
__device__ __forceinline__ void staged_run(const GemmArgs &p, const Tile &x, const int *v, int g, int row0, float rw, float rx,
                                           unsigned char *buf, int half, int q, int lane, bool vec) {
    constexpr int ITEM = OUT == FP4_OUT_F32 ? 4 : 2;
    constexpr int RUN = OUT == FP4_OUT_F32 ? 16 : 32;     // rows at a time
    constexpr int COLS = OUT == FP4_OUT_SWIGLU ? 64 : 128;
    constexpr int VPR = COLS * ITEM / 16;                 // 16-byte pieces of a row
    const int tid = 32 * q + lane;
#pragma unroll
    for (int h = 0; h < 32 / RUN; ++h) {
        if (g + RUN * h >= x.nr) return;                  // the same for all four warps
        half_sync(half);                                  // the buffer's last run has been read
        if (OUT == FP4_OUT_SWIGLU) {
            const bool gate = lane < 16;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                reinterpret_cast<__nv_bfloat16 *>(buf)[(gate ? i : 16 + i) * COLS + 16 * q + (lane & 15)] = swiglu_pair(v, i, gate, rw, rx);
        } else {
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                const float y = __int_as_float(v[RUN * h + j]) * (rw * __shfl_sync(0xffffffffu, rx, RUN * h + j));
                if (OUT == FP4_OUT_F32) reinterpret_cast<float *>(buf)[j * COLS + tid] = y;
                else reinterpret_cast<__nv_bfloat16 *>(buf)[j * COLS + tid] = __float2bfloat16_rn(y);
            }
        }
        half_sync(half);
        const int ncols = OUT == FP4_OUT_SWIGLU ? p.n / 2 : p.n, col0 = OUT == FP4_OUT_SWIGLU ? row0 / 2 : row0;
#pragma unroll
        for (int i = 0; i < RUN * VPR / 128; ++i) {
            const int at = i * 128 + tid, j = at / VPR, c = col0 + (at % VPR) * (16 / ITEM);
            const int row = g + RUN * h + j;
            if (row >= x.nr || c >= ncols) continue;
            unsigned char *dst = static_cast<unsigned char *>(p.out) + (static_cast<size_t>(x.n0 + row) * p.ldo + c) * ITEM;
            const uint4 w = *reinterpret_cast<const uint4 *>(buf + 16 * at);
            if (vec && c + 16 / ITEM <= ncols) {
                *reinterpret_cast<uint4 *>(dst) = w;
            } else {
                const int n = min(16 / ITEM, ncols - c);
                for (int e = 0; e < n; ++e) {
                    if (ITEM == 4) reinterpret_cast<float *>(dst)[e] = reinterpret_cast<const float *>(buf + 16 * at)[e];
                    else reinterpret_cast<uint16_t *>(dst)[e] = reinterpret_cast<const uint16_t *>(buf + 16 * at)[e];
                }
            }
        }
    }
}

template <int FMT>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (FMT == COLI_FP4_NV)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void pair_sf_copy(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
template <int FMT, int OUT>
__global__ void __launch_bounds__(P_THREADS, 1) fp4_pair_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {  // clusters of 2
    using P = PairPlan<FMT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // the same offset in both CTAs: the dynamic array starts at the same address in each
    unsigned char *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sa = sm, *sb = sa + P::S * A_BYTES, *ssa = sb + P::S * P::B_BYTES, *ssb = ssa + P::S * P::SFA_BYTES;
    __shared__ __align__(8) uint64_t bars[2 * P::S + 3];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_tiles;
    __shared__ TileList list;
    __shared__ int s_scan[P_THREADS / 32];
    // full: the leader's, of both CTAs' copies; empty, dfull: in each CTA; dempty: the leader's
    uint64_t *full = bars, *empty = full + P::S, *dfull = empty + P::S, *dempty = dfull + 1, *drain = dempty + 1;
    volatile int *abort = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int MB = (p.n + 255) / 256, KT = (p.k + FP4_KB - 1) / FP4_KB;
    const int W = p.E + p.S;

    if (threadIdx.x == 32) {
        for (int i = 0; i < P::S; ++i) {
            mbar_init(smem_u32(&full[i]), 4);  // each CTA's producer and row-scale warp
            mbar_init(smem_u32(&empty[i]), 1);
        }
        mbar_init(smem_u32(dfull), 1);
        mbar_init(smem_u32(dempty), 2 * P_EPI);
        mbar_init(smem_u32(drain), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_SF) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == W_PROD && elect_one()) prefetch_maps(maps, p.S);
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
        const int atoms = static_cast<int>(fp4_pitch(FMT, p.k) / 4);  // scale tiles of 128 weight rows
        uint32_t s = 0, phase = 1;
        for (int t = pair; t < ntiles; t += pairs) {
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const bool shared = x.e >= p.E;
            const CUtensorMap *ta = shared ? &maps.as : &maps.a, *tsf = shared ? &maps.sfs : &maps.sf;
            const int ez = shared ? 0 : x.e;
            const int n32 = (x.nr + 31) / 32;                        // N / 32; this CTA's share is 16 * n32 rows
            const int row_lo = x.n0 + static_cast<int>(rank) * 16 * n32;
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), phase, abort, p.err))) goto prod_done;
                const uint32_t fb = map_rank(smem_u32(&full[s]), 0);
                if (elect_one()) {
                    remote_expect_tx(fb, A_BYTES + P::SFA_BYTES + n32 * 16 * 128);
                    pair_load_3d(smem_u32(sa + s * A_BYTES), ta, kb * 128, x.m * 256 + static_cast<int>(rank) * 128, ez, fb);
                    pair_load_3d(smem_u32(ssa + s * P::SFA_BYTES), tsf, 0, (x.m * 2 + static_cast<int>(rank)) * atoms + kb * P::ATOMS, ez, fb);
#pragma unroll
                    for (int bit = NBOX - 1; bit >= 0; --bit) {
                        const int row0 = 16 * ((n32 >> (bit + 1)) << (bit + 1));
                        if ((n32 >> bit) & 1) pair_load_2d(smem_u32(sb + s * P::B_BYTES + row0 * 128), &maps.b[bit], kb * 128, row_lo + row0, fb);
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
        const uint64_t sadesc0 = smem_desc_sf(smem_u32(ssa)), sbdesc0 = smem_desc_sf(smem_u32(ssb));
        for (int t = pair; t < ntiles; t += pairs, ++tl) {
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int n32 = (x.nr + 31) / 32;
            const uint32_t idesc = (idesc_fp4<FMT>() & ~(3u << 27)) | (2u << 27) | (static_cast<uint32_t>(4 * n32) << 17);
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(dempty), (tl & 1) ^ 1, abort, p.err))) goto mma_done;
            tc_fence_after();
            for (int kb = 0; kb < KT; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&full[s]), phase, abort, p.err))) goto mma_done;
                tc_fence_after();
                const int steps = min(4, (p.k - kb * FP4_KB + 63) / 64);
                if (elect_one()) {
                    const uint32_t sfa = tbase + 256 + s * P::SF_COLS, sfb = sfa + 4 * P::ATOMS;
                    const uint64_t ad = adesc0 + static_cast<uint64_t>(s * (A_BYTES >> 4)), bd = bdesc0 + static_cast<uint64_t>(s * (P::B_BYTES >> 4));
                    const uint64_t sad = sadesc0 + static_cast<uint64_t>(s * (P::SFA_BYTES >> 4)), sbd = sbdesc0 + static_cast<uint64_t>(s * (P::SFB_BYTES >> 4));
#pragma unroll
                    for (int i = 0; i < P::ATOMS; ++i) {
                        pair_sf_copy(sfa + 4 * i, sad + 32 * i);
                        pair_sf_copy(sfb + 8 * i, sbd + 64 * i);
                        pair_sf_copy(sfb + 8 * i + 4, sbd + 64 * i + 32);
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk < steps) {
                            const int atom = FMT == COLI_FP4_NV ? kk : kk >> 1;
                            const uint32_t id = FMT == COLI_FP4_NV ? 0u : 2u * (kk & 1);
                            pair_mma<FMT>(tbase, ad + 2 * kk, bd + 2 * kk, idesc | (id << 4) | (id << 29), sfa + 4 * atom, sfb + 8 * atom, (kb | kk) != 0);
                        }
                    }
                    pair_commit(smem_u32(&empty[s]));
                }
                __syncwarp();
                if (++s == P::S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (elect_one()) pair_commit(smem_u32(dfull));
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
    } else if (warp == W_SF || warp == W_SF + 1) {
        // ------------------------------------------------------------------ scales of the rows
        row_scales<FMT, P_NT>(p, warp - W_SF, pair, pairs, ntiles, KT, list, W, ssb, empty, P::S, 0, abort,
                              [&](int st) { remote_arrive(map_rank(smem_u32(&full[st]), 0)); });
    } else if (warp >= W_EPI0) {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - W_EPI0) >> 2;  // TMEM lane quarter, 128-column half
        unsigned char *obuf = ssb + P::S * P::SFB_BYTES + half * P_OUT;
        constexpr int ITEM = OUT == FP4_OUT_F32 ? 4 : 2;
        const bool vec = ((reinterpret_cast<uintptr_t>(p.out) | (p.ldo * ITEM)) & 15) == 0;
        uint32_t tl = 0;
        for (int t = pair; t < ntiles; t += pairs, ++tl) {
            const Tile x = tile_at<P_NT>(t, list, p, W);
            const int r = x.m * 256 + static_cast<int>(rank) * 128 + 32 * q + lane;
            const float *wrow = x.e >= p.E ? p.wrow_shared : (p.wrow ? p.wrow + static_cast<size_t>(x.e) * p.wrow_stride : nullptr);
            float rw = wrow && r < p.n ? __ldg(wrow + r) : 1.f;
            float rx[4];
            bool usual = ordinary(rw);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int j = 128 * half + 32 * g + lane;
                rx[g] = p.xrow && j < x.nr ? __ldg(p.xrow + x.n0 + j) : 1.f;
                usual = usual && ordinary(rx[g]);
            }
            // (all eight warps meet in the staging barriers: they give up together, or not at all)
            if (epi_or(!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(dfull), tl & 1, abort, p.err)))) break;
            tc_fence_after();
            if (!__all_sync(0xffffffffu, usual)) {
                // in tensor memory, before the sums fill the registers (8 at a time: more took registers from the
                // ordinary tiles, 8192 rows, k 512, 57 us against 49)
                const float pw = halve_exponent(rw);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (128 * half + 32 * g < x.nr) split_scales(tbase + (static_cast<uint32_t>(32 * q) << 16) + 128 * half + 32 * g, pw, rx[g]);
            }
            int v[4][32];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (128 * half + 32 * g < x.nr) tmem_ld32(tbase + (static_cast<uint32_t>(32 * q) << 16) + 128 * half + 32 * g, v[g]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive(map_rank(smem_u32(dempty), 0));
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (128 * half + 32 * g < x.nr)
                    staged_run<OUT>(p, x, v[g], 128 * half + 32 * g, x.m * 256 + static_cast<int>(rank) * 128, rw, rx[g], obuf, half, q, lane, vec);
        }
    }

    dependents_may_launch();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == W_SF) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512u) : "memory");
    }
}

// Weight codes of `count` matrices, boxes of 128 rows of a k-block.
bool mats_map(CUtensorMap *m, const coli_fp4_mats &w, int k) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k) / 2, static_cast<cuuint64_t>(w.n), static_cast<cuuint64_t>(w.count)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(k) / 2, w.count > 1 ? w.codes_stride : static_cast<cuuint64_t>(w.n) * (k / 2)};
    const cuuint32_t box[3] = {128, 128, 1};
    return encode_u8(m, w.codes, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scale tiles of `count` matrices, boxes of a k-block's tiles.
bool tiles_map(CUtensorMap *m, const coli_fp4_mats &w, int fmt, int k) {
    const cuuint64_t bytes = fp4_scale_bytes(fmt, COLI_FP4_TILES, w.n, k);
    const cuuint64_t dims[3] = {128, bytes / 512, static_cast<cuuint64_t>(w.count)};
    const cuuint64_t strides[2] = {512, w.count > 1 ? w.scales_stride : bytes};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(FP4_KB / fp4_block(fmt) / 4), 1}, es[3] = {1, 1, 1};
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(w.scales), dims, strides, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Row codes, boxes of 16 << i rows, as far as the rows reach.
bool rows_maps(CUtensorMap *m, const coli_fp4_rows &a, int k) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k) / 2, static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k) / 2};
    for (int i = 0; i < NBOX; ++i) {
        if (i && (8 << i) >= a.rows) {  // no group is that high: the box is never used
            m[i] = m[i - 1];
            continue;
        }
        const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(16 << i)};
        if (!encode_u8(m + i, a.codes, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return false;
    }
    return true;
}

template <int FMT, int OUT>
cudaError_t launch_gemm(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<FMT, 128>;
    auto kernel = fp4_gemm_kernel<FMT, 128, OUT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const long chunks = g.rows / 128 + (g.rows < g.E + g.S ? g.rows : g.E + g.S);  // at most
    const long tiles = (chunks < 1 ? 1 : chunks) * ((g.n + 127) / 128);
    const int sms = device_sm_count();
    return launch_early(kernel, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), THREADS, P::SMEM, st, 1, maps, g);
}

// At most 32 rows: tiles of 128 weight rows x all rows of a matrix, their k-blocks split over clusters of 1, 2
// or 4 CTAs, whichever leaves the busiest CTA the least (the matrices that have rows are at most as many as
// rows).  One row, 4096 x 6144: 8.5 us against 11.3 unsplit.
template <int FMT, int OUT>
cudaError_t launch_split(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = Plan<FMT, 32>;
    auto kernel = fp4_gemm_kernel<FMT, 32, OUT>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count(), kt = (g.k + FP4_KB - 1) / FP4_KB;
    const int tiles = (g.rows < g.E + g.S ? g.rows : g.E + g.S) * ((g.n + 127) / 128);
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

template <int FMT, int OUT>
cudaError_t launch_pair(const GemmMaps &maps, const GemmArgs &g, cudaStream_t st) {
    using P = PairPlan<FMT>;
    auto kernel = fp4_pair_kernel<FMT, OUT>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, P::SMEM, ready);
    if (e != cudaSuccess) return e;
    const long chunks = g.rows / P_NT + (g.rows < g.E + g.S ? g.rows : g.E + g.S);
    const long tiles = (chunks < 1 ? 1 : chunks) * ((g.n + 255) / 256);
    const int pairs = device_sm_count() / 2;
    return launch_early(kernel, dim3(2 * static_cast<unsigned>(tiles < pairs ? tiles : pairs)), P_THREADS, P::SMEM, st, 2, maps, g);
}

template <int FMT, int OUT>
cudaError_t launch_out(const GemmMaps &maps, const GemmArgs &g, bool pairs, cudaStream_t st) {
    if (pairs) return launch_pair<FMT, OUT>(maps, g, st);
    return g.rows <= 32 ? launch_split<FMT, OUT>(maps, g, st) : launch_gemm<FMT, OUT>(maps, g, st);
}

template <int FMT>
cudaError_t launch_fmt(const GemmMaps &maps, const GemmArgs &g, int out_kind, bool pairs, cudaStream_t st) {
    if (out_kind == FP4_OUT_F32) return launch_out<FMT, FP4_OUT_F32>(maps, g, pairs, st);
    if (out_kind == FP4_OUT_BF16) return launch_out<FMT, FP4_OUT_BF16>(maps, g, pairs, st);
    return launch_out<FMT, FP4_OUT_SWIGLU>(maps, g, pairs, st);
}

}  // namespace

// Tiles of 256 x 256 on CTA pairs, or of 128 x 128 on single CTAs: pairs from PAIR_ROWS rows per matrix on
// average, and from 33 where tiles of 128 x 128 do not fill the GPU (the pair kernel's epilogue is the
// faster one).  Measured (4096 x 6144 matrices, NV, bf16 out; pairs against single CTAs, us): 64 matrices
// with 32 / 64 / 96 rows each 142 / 150 / 158 against 142 / 148 / 156, with 128 rows 167 against 211; one
// matrix with 64 / 256 / 2048 / 8192 rows 12 / 16 / 31 / 95 against 14 / 19 / 49 / 146.  A shared expert's many
// rows ask for pairs too: expert half of a layer with 512 / 1024 / 2048 tokens (256 experts, Zipf, 8 and the
// shared one per token) 639 / 819 / 1141 us against 637 / 831 / 1272.
constexpr int PAIR_ROWS = 112, PAIR_SHARED = 768;

static bool use_pairs(const Fp4ProductArgs &p) {
    const int mats = p.w.count + (p.shared ? 1 : 0), avg = p.a.rows / mats;
    return avg >= PAIR_ROWS || p.shared_rows >= PAIR_SHARED || (avg > 32 && static_cast<long>(mats) * ((avg + 127) / 128) * ((p.w.n + 127) / 128) < device_sm_count());
}

cudaError_t launch_fp4_product(int fmt, const Fp4ProductArgs &p, cudaStream_t st) {
    GemmMaps maps;
    const bool pairs = use_pairs(p);
    bool ok = mats_map(&maps.a, p.w, p.k) && (!p.shared || mats_map(&maps.as, *p.shared, p.k));
    ok = ok && rows_maps(maps.b, p.a, p.k);
    if (pairs) ok = ok && tiles_map(&maps.sf, p.w, fmt, p.k) && (!p.shared || tiles_map(&maps.sfs, *p.shared, fmt, p.k));
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
    return fmt == COLI_FP4_MX ? launch_fmt<COLI_FP4_MX>(maps, g, p.out_kind, pairs, st) : launch_fmt<COLI_FP4_NV>(maps, g, p.out_kind, pairs, st);
}

}  // namespace coli
