// group_tiles.h -- what the grouped products of 4-bit and 8-bit operands share: the list of tiles of a
// batch's groups, split k over clusters, CTA pairs, and the scaling of their sums.  Included by one .cu per kernel
// family; all names stay local to it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "coli_moe.h"
#include "pdl.h"
#include "tc_ptx.h"

namespace coli {
namespace {

constexpr int P_NT = 256;                // rows of a CTA pair's tile
constexpr int P_EPI = 8;                 // epilogue warps of a pair's CTA
constexpr int BAND = 8;                  // weight blocks side by side in the order of the tiles
constexpr int MAX_MATS = 1025;           // 1024 and a shared one
constexpr int NBOX = 4;                  // box heights 16 << i rows
constexpr int MAX_SPLIT = 4;             // CTAs that share a tile's k-blocks at most

struct GroupArgs {
    const int32_t *offsets;
    int E, S;                            // matrices; 1: a shared one for the rows behind the groups
    int rows, n;
    int *err;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t a) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ void remote_expect_tx(uint32_t a, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(a), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try_cluster(uint32_t a, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(a), "r"(parity), "r"(20000u) : "memory");
    return ok != 0;
}
// mbar_wait for a phase that the other CTA of the pair takes part in
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t a, uint32_t parity, volatile int *abort, int *err) {
    if (mbar_try_cluster(a, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_cluster(a, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > WAIT_CYCLES) {
            *abort = 1;
            atomicOr(err, COLI_DEVERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
struct Tile {
    int e, m, n0, nr;      // matrix, block of 128 weight rows, first row, rows
};

// What every role looks tiles up in, in shared memory: tiles before each matrix, and the offsets.
struct TileList {
    int first[MAX_MATS + 31 & ~31];
    int off[MAX_MATS];
};

// First row and row count of matrix e's group; count -1 when the offsets are not ascending in range.
__device__ __forceinline__ void group_rows(const GroupArgs &p, const TileList &l, int e, int &lo, int &cnt) {
    lo = 0;
    cnt = p.rows;
    if (p.offsets) {
        lo = l.off[e];
        const int hi = e < p.E ? l.off[e + 1] : p.rows;
        cnt = lo < 0 || hi < lo || hi > p.rows ? -1 : hi - lo;
    }
}

// Tile t of the list, by a whole warp: two ballots find the last matrix whose first tile is not behind t.
template <int NT>
__device__ __forceinline__ Tile tile_at(int t, const TileList &l, const GroupArgs &p, int W) {
    const int MB = (p.n + (NT == P_NT ? 255 : 127)) / (NT == P_NT ? 256 : 128);
    const int lane = threadIdx.x & 31;
    const int most = min(W, 1024), blocks = (most + 31) / 32;
    const int run = 31 - __clz(__ballot_sync(0xffffffffu, lane < blocks && l.first[min(32 * lane, MAX_MATS - 1)] <= t) | 1u);
    int e = 32 * run + 31 - __clz(__ballot_sync(0xffffffffu, 32 * run + lane < most && l.first[32 * run + lane] <= t) | 1u);
    if (W > 1024 && l.first[1024] <= t) e = 1024;
    Tile x;
    x.e = e;
    int row0, cnt;
    group_rows(p, l, e, row0, cnt);
    const int i = t - l.first[e];
    x.m = i;
    x.n0 = row0;
    x.nr = cnt;
    if (cnt > NT) {
        const int nch = (cnt + NT - 1) / NT;
        const int per = ((cnt + nch - 1) / nch + 31) & ~31;  // rows of a chunk: even shares
        // bands of BAND weight blocks: a wave of tiles is BAND blocks times several chunks (against all chunks
        // of one block after another: 2048 rows, 6144 x 2048, 25 us against 29)
        const int band = i / (BAND * nch), j = i - band * (BAND * nch), high = min(BAND, MB - band * BAND);
        const int c = j / high;
        x.m = band * BAND + (j - c * high);
        x.n0 = row0 + c * per;
        x.nr = min(per, cnt - c * per);
    }
    return x;
}

// Fills the tile list, by the N threads from warp W0 on, the epilogue's (named barrier 1), while the others set up the
// rest: the offsets, and an exclusive scan of the matrices' tiles.  The number of tiles.
template <int NT, int N, int W0>
__device__ __forceinline__ int tile_list(const GroupArgs &p, int W, int MB, TileList &l, int *s_scan) {
    const int tid = threadIdx.x - W0 * 32, warp = tid >> 5, lane = tid & 31;
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); };
    if (p.offsets) {
        for (int e = tid; e <= p.E; e += N) l.off[e] = __ldg(p.offsets + e);
        sync();
    }
    int carry = 0;
    for (int base = 0; base < W; base += N) {
        const int e = base + tid;
        int lo = 0, cnt = 0;
        if (e < W) group_rows(p, l, e, lo, cnt);
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
        sync();
        int before = carry;
        for (int w = 0; w < N / 32; ++w) {
            const int v = s_scan[w];
            if (w < warp) before += v;
            carry += v;
        }
        if (e < W) l.first[e] = before + inc - tiles;
        sync();
    }
    return carry;
}

// The row scales.  A sum is multiplied with rw * rx, which can leave float32's range before the result does: the
// quantiser itself hands out scales of 2^-126 to 2^117.  Of scales within [2^-63, 2^64) every product is a
// normal float32 and nothing more is done.  Otherwise half of each scale's exponent, a power of two, goes out of
// rw and rx and into the sums: rw rx is then in range for all pairs; it and the power have exponents of the same
// sign, so neither overflows or underflows a result that does not; and a normal result whose rw rx was in range
// has the same bits as without.
__device__ __forceinline__ bool ordinary(float s) { return (__float_as_uint(s) >> 23 & 0xffu) - 64u <= 126u; }
// s = the returned power of two * s afterwards.
__device__ __forceinline__ float halve_exponent(float &s) {
    const int e = static_cast<int>(__float_as_uint(s) >> 23 & 0xffu), k = e ? (e - 126) >> 1 : -74;
    s *= __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}
// A sum times the parts of the exponent (2^64 twice would be infinite).
__device__ __forceinline__ int scaled_sum(int v, float pw, float px) {
    const float s = __int_as_float(v);
    return __float_as_int((px < 1.f) == (pw < 1.f) ? s * px * pw : s * (px * pw));
}
// A run of N rows (rx: row `lane`'s) x a weight row per lane, whose part of the exponent is `pw`.
template <int N>
__device__ __forceinline__ void split_scales(int (&v)[N], float pw, float &rx) {
    const float px = halve_exponent(rx);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = scaled_sum(v[j], pw, __shfl_sync(0xffffffffu, px, j));
}

// Split k, one epilogue warp's 32 weight rows: ranks above 0 send their sums to rank 0's shared memory by
// stores that count on its barrier as they land (no fence: with one, and whole-cluster barriers in the
// kernel's way, a split took 3.5 us), rank 0 adds them in the order of the ranks.  A weight row's 32 sums
// are 8 pieces of 16 bytes, piece i at i ^ (row % 8).  tl counts the tiles; `last`: no tile follows.
// False when a wait gave up.
template <typename Add>
__device__ __forceinline__ bool split_sum(int (&v)[32], int nr, int C, int rank, int q, int lane, uint32_t tl, bool last, float *part,
                                          uint64_t *pfull, uint64_t *pfree, volatile int *abort, int *err, Add add) {
    const int row = 32 * q + lane, pieces = (nr + 3) / 4;
    if (rank != 0) {
        if (tl > 0 && !__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(pfree), (tl & 1) ^ 1, abort, err))) return false;
        const uint32_t to = map_rank(smem_u32(part) + ((rank - 1) * 128 + row) * 128, 0), bar = map_rank(smem_u32(pfull), 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < pieces)
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                             ::"r"(to + ((i ^ (lane & 7)) << 4)), "r"(v[4 * i]), "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3]), "r"(bar) : "memory");
    } else {
        if (lane == 0) mbar_expect_tx(smem_u32(pfull), (C - 1) * 32 * pieces * 16);  // this warp's rows
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(pfull), tl & 1, abort, err))) return false;
        for (int c = 1; c < C; ++c) {
            const int4 *from = reinterpret_cast<const int4 *>(part + ((c - 1) * 128 + row) * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < pieces) {
                    const int4 f = from[i ^ (lane & 7)];
                    v[4 * i] = add(v[4 * i], f.x);
                    v[4 * i + 1] = add(v[4 * i + 1], f.y);
                    v[4 * i + 2] = add(v[4 * i + 2], f.z);
                    v[4 * i + 3] = add(v[4 * i + 3], f.w);
                }
        }
        __syncwarp();
        if (lane == 0 && !last)
            for (int c = 1; c < C; ++c) remote_arrive(map_rank(smem_u32(pfree), c));
    }
    return true;
}

__device__ __forceinline__ void half_sync(int half) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}
// A predicate OR-ed over the eight epilogue warps.
__device__ __forceinline__ bool epi_or(bool pred) {
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, 3, %2, p; selp.u32 %0, 1, 0, q; }"
                 : "=r"(r) : "r"(static_cast<uint32_t>(pred)), "n"(P_EPI * 32) : "memory");
    return r != 0;
}
// TMA loads of a pair's CTA: into its own shared memory, the barrier in the leader's.
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *m, int c0, int c1, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
// arrive on the barrier at this address in both CTAs (`both`: the ranks' bits) once the MMAs issued so far have completed
__device__ __forceinline__ void pair_commit(uint32_t mbar, uint16_t both = 3) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(mbar), "h"(both) : "memory");
}

// Clusters of c CTAs, one CTA per SM, that run at once: with c = 4 some SMs of a GPC are left over (33
// clusters on B200's 148 SMs, by cudaOccupancyMaxActiveClusters).
int cluster_count(int c, int sms) { return c <= 2 ? sms / c : (sms - 16) / 4; }

}  // namespace
}  // namespace coli
