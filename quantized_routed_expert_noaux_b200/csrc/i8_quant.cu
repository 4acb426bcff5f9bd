// i8_quant.cu -- rows to 8-bit integers with one scale each (coli_moe_i8_quantize), SwiGLU of gate and up rows first
// where asked for, every row written to the places of its copies.
//
// scale = m / 127, m = the row's largest |x| (at least 127 * 2^-126); code = the whole number nearest to x / (m / 127) of
// the real numbers, ties to even.  With v within 2^-22 of 127 / m, the real quotient lies between x v (1 - 2^-21)
// and x v (1 + 2^-21), and so does its nearest whole number between theirs (an FMA that adds 1.5 * 2^23 rounds each
// once, to a whole number).  Where those two differ, once in 10^5 float32 elements, the quotient is next to a half i + 1/2, and
// 127 |x| is compared with (i + 1/2) m: with p = fl((i + 1/2) m) and e = (i + 1/2) m - p (an FMA gives it exactly), 127 |x| - p is
// a float32 too, since the two are within 2^-13 of each other and 127 |x| has 31 bits; it is compared with e.  (Both
// sides over 128, and times 2^64 where m is below 1, so that nothing overflows or underflows.)
//
// A thread takes chunks of 16 elements; the row's chunks stay in registers between the pass that finds m
// and the one that writes, HOLD to a thread (what is done once a row and thread, 60 instructions, counts beside the 90 of a
// chunk); what rows beyond HOLD * MOST_T chunks have more is read again, from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "chunk.h"
#include "i8.h"
#include "internal.h"
#include "pdl.h"
#include "tc_ptx.h"

namespace coli {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int HOLD = 2;       // chunks a thread keeps in registers
constexpr int MOST_T = 384;   // threads of a row at most
constexpr int WARP_ROWS = 4;  // rows of a CTA where a warp takes a row

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The first n (<= 16) of 16 elements at any address, zeros behind them.
template <typename In>
__device__ __forceinline__ void load_some(Chunk<In> &c, const In *p, int n) {
    c.zero();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i >= n) continue;
        if constexpr (sizeof(In) == 4) c.v[i] = __ldg(p + i);
        else c.w[i >> 1] |= static_cast<uint32_t>(__ldg(p + i)) << (16 * (i & 1));
    }
}
// align: what every row's address is a multiple of, in bytes (32, 16 or less)
template <typename In, bool SHARED>
__device__ __forceinline__ void load_chunk(Chunk<In> &c, const In *p, int n, int align) {
    if constexpr (SHARED) {  // whole 16-byte pieces
        uint32_t w[sizeof(In) * 4] = {};
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(In)); ++i)
            if (n > i * static_cast<int>(16 / sizeof(In))) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
            }
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(In)) * 4; ++i) {
            if constexpr (sizeof(In) == 4) c.v[i] = __uint_as_float(w[i]);
            else c.w[i] = w[i];
        }
        return;
    }
    if (n >= 16 && align >= 16) c.load(p, align >= 32);
    else load_some(c, p, n);
}

// The largest magnitude so far as bits of a float32 (of two bf16 values side by side): a NaN stays.  (The signs
// of the results mean nothing.)
__device__ __forceinline__ void largest(uint32_t &top, const Chunk<float> &c) {
#pragma unroll
    for (int i = 0; i < 16; ++i) asm("max.NaN.xorsign.abs.f32 %0, %0, %1;" : "+r"(top) : "r"(__float_as_uint(c.v[i])));
}
__device__ __forceinline__ void largest(uint32_t &top, const Chunk<uint16_t> &c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(c.w[i]));
}
template <typename Held>
__device__ __forceinline__ uint32_t magnitude(uint32_t top) {
    if constexpr (sizeof(Held) == sizeof(Chunk<float>)) return top & 0x7fffffffu;
    else return max(top & 0x7fff0000u, top << 16 & 0x7fff0000u);
}

constexpr float FAR = -80.0f;
// SiLU(gate) * up.  Of a divisor above 2^126 (gates below -87.3) the fast quotient is 0, and e^-gate is infinite below -88.7.  Below FAR the
// divisor is e^-gate but for 2^-115 of it; e^gate, which float32 does not hold further down, comes in as its fourth root four times:
// magnitudes fall from product to product behind the one with `up`, so each is a normal number where the result is, and
// |gate| e^(gate / 4) < 1 keeps that one finite.  (Four times expf's unit of 2^-23 and five roundings: within 7 * 2^-23.)
__device__ __forceinline__ float swiglu(float gate, float up) { return __fdividef(gate, 1.0f + expf(-gate)) * up; }
__device__ __forceinline__ float swiglu_far(float gate, float up) {
    const float e = expf(0.25f * gate);
    return gate * e * up * e * e * e;
}

// What is quantised: the row's own elements, or SiLU(gate) * up in float32.
template <typename In, bool GLU> struct Source { using Held = Chunk<In>; };
template <typename In> struct Source<In, true> { using Held = Chunk<float>; };

// Chunk i of a row; `low`: the lowest gate so far.  far_gates() below goes over the chunk again where that is below FAR.
template <typename In, bool GLU, bool SHARED = false>
__device__ __forceinline__ void fetch(typename Source<In, GLU>::Held &h, float &low, const In *row, int k, int up, int i, int align) {  // up: where up values begin
    const int n = k - 16 * i;
    if constexpr (GLU) {
        Chunk<In> g, u;
        load_chunk<In, SHARED>(g, row + 16 * static_cast<size_t>(i), n, align);
        load_chunk<In, SHARED>(u, row + up + 16 * static_cast<size_t>(i), n, align);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            low = fminf(low, g.at(j));
            h.v[j] = swiglu(g.at(j), u.at(j));
        }
    } else {
        load_chunk<In, SHARED>(h, row + 16 * static_cast<size_t>(i), n, align);
    }
}
__device__ __forceinline__ float value(const float *p) { return *p; }
__device__ __forceinline__ float value(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
// (Element by element from memory, behind all chunks of a thread: 4096 bf16 / 2048 float32 rows of k = 2048 take 10.9 / 8.4 us, 10.5 / 8.4
// without this, and 11.2 / 9.6 where fetch() does it with gates and up values held until then.)
template <typename In, typename Held>
__device__ __forceinline__ void far_gates(Held &h, const In *row, int k, int up, int i) {
    if constexpr (sizeof(Held) == sizeof(Chunk<float>)) {
        row += 16 * static_cast<size_t>(i);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < k - 16 * i && value(row + j) < FAR) h.v[j] = swiglu_far(value(row + j), value(row + up + j));
    }
}

constexpr float ROUND = 12582912.0f;  // 1.5 * 2^23: added, the whole number is in the low bits

__device__ __forceinline__ uint32_t pack4(const float *f) {  // the low bytes of four words
    return __byte_perm(__byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040), __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040), 0x5410);
}

// Codes of a chunk; `lo`, `hi`: v (1 - 2^-21) and v (1 + 2^-21), twice each.
template <typename Held>
__device__ __forceinline__ uint4 encode(const Held &h, float m, uint64_t lo, uint64_t hi) {
    const uint64_t up = pack2(ROUND, ROUND);
    uint32_t word[4], differ = 0u;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t x = pack2(h.at(4 * w + 2 * i), h.at(4 * w + 2 * i + 1));
            unpack2(fma2(x, lo, up), a[2 * i], a[2 * i + 1]);
            unpack2(fma2(x, hi, up), b[2 * i], b[2 * i + 1]);
        }
        word[w] = pack4(a);
        differ |= word[w] ^ pack4(b);
    }
    if (differ) {
        float vl, vh;
        unpack2(lo, vl, vh);
        const float up64 = m < 1.f ? 0x1p64f : 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = h.at(i), f = floorf(fabsf(x * vl)), r = rintf(fabsf(x * vl));
            // (f: the half's i, or one more where x vl comes that close to the next whole number, which is no border then)
            const float g = (f + 0.5f) * 0x1p-7f, ms = m * up64, p = g * ms;
            const float e = fmaf(g, ms, -p), d = fmaf(127.0f * 0x1p-7f, fabsf(x) * up64, -p);
            const bool near = fabsf(fabsf(x * vl) - f - 0.5f) < 1.0f / 8192.0f;
            int c = static_cast<int>(f);
            c += d > e || (d == e && (c & 1));
            if (!near) c = static_cast<int>(r);
            const uint32_t byte = static_cast<uint32_t>(x < 0.f ? -c : c) & 0xffu;
            word[i >> 2] = (word[i >> 2] & ~(0xffu << 8 * (i & 3))) | byte << 8 * (i & 3);
        }
    }
    return make_uint4(word[0], word[1], word[2], word[3]);
}

// What a row's codes are made with: from the bits of its largest magnitude.
struct Scale {
    bool finite;
    float m;
    uint64_t lo, hi;
    __device__ __forceinline__ explicit Scale(uint32_t top) {
        finite = top < INF_BITS;
        m = fmaxf(__uint_as_float(top), 127.0f * 0x1p-126f);
        float v;  // (of m / 16, whose inverse is a normal number)
        asm("rcp.approx.f32 %0, %1;" : "=f"(v) : "f"(m * 0.0625f));
        v *= 127.0f * 0.0625f;
        const float vlo = v * (1.0f - 0x1p-21f), vhi = v * (1.0f + 0x1p-21f);
        lo = pack2(vlo, vlo);
        hi = pack2(vhi, vhi);
    }
    __device__ __forceinline__ float value() const { return finite ? __fdiv_rn(m, 127.0f) : __uint_as_float(0x7fffffffu); }
    template <typename Held>
    __device__ __forceinline__ uint4 codes(const Held &h) const {
        return finite ? encode(h, m, lo, hi) : make_uint4(0u, 0u, 0u, 0u);
    }
};

// Where row r goes.  With PLACE: the places of its first 32 copies are in `first`, one per lane.
template <bool PLACE>
struct Target {
    const I8QuantArgs &a;
    const int r, lane;
    int first;
    __device__ __forceinline__ Target(const I8QuantArgs &a, int r) : a(a), r(r), lane(threadIdx.x & 31), first(-1) {
        if (PLACE && lane < a.copies) first = __ldg(a.place + static_cast<size_t>(r) * a.copies + lane);
    }
    __device__ __forceinline__ int named(int c0) const {  // copy c0 + lane
        return c0 == 0 ? first : c0 + lane < a.copies ? __ldg(a.place + static_cast<size_t>(r) * a.copies + c0 + lane) : -1;
    }
    __device__ __forceinline__ void put_scale(float scale) const {  // by one warp
        if constexpr (!PLACE) {
            if (lane == 0) a.row_scale[r] = scale;
        } else {
            for (int c0 = 0; c0 < a.copies; c0 += 32) {
                const int to = named(c0);
                if (to >= 0 && to < a.rows) a.row_scale[to] = scale;
                else if (to != -1) atomicOr(a.err, COLI_DEVERR_GROUPING);
            }
        }
    }
    __device__ __forceinline__ void put(const uint4 &v, int i, int n) const {  // chunk i of n, by whole warps
        int8_t *at = a.codes + 16 * static_cast<size_t>(i);
        if constexpr (!PLACE) {
            if (i < n) *reinterpret_cast<uint4 *>(at + static_cast<size_t>(r) * a.ldc) = v;
        } else {
            for (int c0 = 0; c0 < a.copies; c0 += 32) {
                const int mine = named(c0);
                for (int c = 0; c < min(32, a.copies - c0); ++c) {
                    const int to = __shfl_sync(FULL, mine, c);
                    if (to >= 0 && to < a.rows && i < n) *reinterpret_cast<uint4 *>(at + static_cast<size_t>(to) * a.ldc) = v;
                }
            }
        }
    }
};

// A row by a warp (WARP: WARP_ROWS rows to a CTA) or by a CTA.
template <typename In, bool GLU, bool WARP, bool PLACE>
__global__ void __launch_bounds__(WARP ? 32 * WARP_ROWS : MOST_T, WARP ? 6 : 2) i8_quantize_kernel(const I8QuantArgs a, int align, bool staged) {
    using Held = typename Source<In, GLU>::Held;
    extern __shared__ __align__(16) unsigned char stage[];
    __shared__ uint32_t s_max[MOST_T / 32];
    wait_for_previous();
    dependents_may_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = WARP ? lane : threadIdx.x, tpr = WARP ? 32 : blockDim.x;
    const int r = WARP ? blockIdx.x * WARP_ROWS + warp : blockIdx.x;
    if (r >= a.src_rows) return;
    const int n = (a.k + 15) / 16;
    const In *row = static_cast<const In *>(a.x) + static_cast<size_t>(r) * a.ldx;
    Held held[HOLD];
    const In *src = row;
    int up = a.k;
    if (staged) {
        // rows at any address: by neighbouring lanes into shared memory, chunks from there
        const int padded = n * 16;
        In *mine = reinterpret_cast<In *>(stage) + static_cast<size_t>(WARP ? warp : 0) * padded * (GLU ? 2 : 1);
#pragma unroll
        for (int part = 0; part < (GLU ? 2 : 1); ++part)
            for (int base = i0; base < padded; base += 16 * tpr) {
                In v[16];  // all on their way together
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = base + j * tpr < a.k ? __ldg(row + part * a.k + base + j * tpr) : In(0);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (base + j * tpr < padded) mine[part * padded + base + j * tpr] = v[j];
            }
        if (WARP) __syncwarp();
        else __syncthreads();
        src = mine;
        up = padded;
    }
    float low = 0.f;
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        const int i = i0 + h * tpr;
        if (i >= n) held[h].zero();
        else if (staged) fetch<In, GLU, true>(held[h], low, src, n * 16, up, i, 16);
        else fetch<In, GLU>(held[h], low, src, a.k, up, i, align);
    }
    if (GLU && low < FAR) {
#pragma unroll
        for (int h = 0; h < HOLD; ++h) far_gates(held[h], src, a.k, up, i0 + h * tpr);
    }
    const Target<PLACE> target(a, r);
    uint32_t top = 0u;
#pragma unroll
    for (int h = 0; h < HOLD; ++h) largest(top, held[h]);
    for (int i = i0 + HOLD * tpr; i < n; i += tpr) {
        Held c;
        fetch<In, GLU>(c, low, row, a.k, a.k, i, align);
        if (GLU && low < FAR) far_gates(c, row, a.k, a.k, i);
        largest(top, c);
    }
    top = __reduce_max_sync(FULL, magnitude<Held>(top));
    if (!WARP) {
        if (lane == 0) s_max[warp] = top;
        __syncthreads();
        top = __reduce_max_sync(FULL, lane < tpr / 32 ? s_max[lane] : 0u);
    }
    const Scale s(top);
    if (WARP || warp == 0) target.put_scale(s.value());
#pragma unroll
    for (int h = 0; h < HOLD; ++h)
        if (h * tpr < n) target.put(s.codes(held[h]), i0 + h * tpr, n);
    for (int base = HOLD * tpr; base < n; base += tpr) {
        Held c;
        if (base + i0 < n) fetch<In, GLU>(c, low, row, a.k, a.k, base + i0, align);
        else c.zero();
        if (GLU && low < FAR) far_gates(c, row, a.k, a.k, base + i0);
        target.put(s.codes(c), base + i0, n);
    }
}

// Many rows: a CTA takes them one after another out of a ring in shared memory that bulk copies fill, so that what is on its way
// does not depend on registers.  Rows are whole 16-byte pieces that start at multiples of 16 bytes.  With i8_quantize_kernel's time
// behind the stroke: 1024 / 4096 / 8192 rows of 6144 bf16 values 6.1 / 13.8 / 28 us against 5.0 / 13.5 / 32 (HBM would take 23 for 8192); 1024 /
// 4096 / 16,384 SwiGLU rows of 2048 5.3 / 10.9 / 36 against 5.2 / 10.2 / 40 (26); 1024 / 8192 float32 rows of 2304 4.3 / 16.1 against 3.4 /
// 15.3, of 6144 8192 44 against 38.  So it is ahead from about 64 MB of bf16 rows on, behind below that by up to 1 us, and behind for
// float32.  Instructions bound it, issued in half of the cycles with the warps that 80 registers leave room for.
// (Ties take the exact comparison.  bf16 has few values: x = m / 2 is one, 63.5, and a maximum of 127 / 32 makes hundreds; of normal values 20
// elements in a row of 6144 need it, in 44% of the warps: 8192 such rows 48 us.  The times above are of rows with a few louder channels: 1
// element, 2%.)
constexpr int RING_ROWS = 1024, MOST_SLOTS = 8;
template <typename In, bool GLU> constexpr int RING_HOLD = sizeof(In) == 2 && !GLU ? 4 : 2;
constexpr size_t RING_SMEM = 208 * 1024;  // of all CTAs of an SM

template <typename In, bool GLU, bool PLACE>
__global__ void __launch_bounds__(MOST_T, 2) i8_quantize_ring_kernel(const I8QuantArgs a, int row_bytes, int slots) {
    using Held = typename Source<In, GLU>::Held;
    constexpr int HOLD = RING_HOLD<In, GLU>;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[MOST_SLOTS];
    __shared__ uint32_t s_max[2][MOST_T / 32];
    __shared__ int s_abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (a.k + 15) / 16;
    volatile int *abort = &s_abort;
    const int mine = (a.src_rows - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1;  // (no more CTAs than rows)
    auto load = [&](int j, int slot) {  // by thread 0
        const uint32_t bar = smem_u32(&bars[slot]);
        mbar_expect_tx(bar, row_bytes);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                     ::"r"(smem_u32(ring + slot * row_bytes)),
                       "l"(static_cast<const In *>(a.x) + (blockIdx.x + static_cast<size_t>(j) * gridDim.x) * a.ldx), "r"(row_bytes), "r"(bar) : "memory");
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(smem_u32(&bars[i]), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    wait_for_previous();
    dependents_may_launch();
    if (threadIdx.x == 0)
        for (int j = 0; j < slots && j < mine; ++j) load(j, j);
    int j = 0, slot = 0;
    uint32_t phase = 0;
    for (; j < mine; ++j) {
        const Target<PLACE> target(a, blockIdx.x + j * gridDim.x);
        const bool ok = mbar_wait(smem_u32(&bars[slot]), phase, abort, a.err);
        const In *row = reinterpret_cast<const In *>(ring + slot * row_bytes);
        Held held[HOLD];
        uint32_t top = 0u;
        float low = 0.f;
#pragma unroll
        for (int h = 0; h < HOLD; ++h) {
            const int i = threadIdx.x + h * blockDim.x;
            if (i < n) fetch<In, GLU, true>(held[h], low, row, a.k, a.k, i, 16);
            else held[h].zero();
        }
        if (GLU && low < FAR) {
#pragma unroll
            for (int h = 0; h < HOLD; ++h) far_gates(held[h], row, a.k, a.k, threadIdx.x + h * blockDim.x);
        }
#pragma unroll
        for (int h = 0; h < HOLD; ++h) largest(top, held[h]);
        top = __reduce_max_sync(FULL, magnitude<Held>(top));
        if (lane == 0) s_max[j & 1][warp] = top;
        if (__syncthreads_or(!ok)) break;
        // the row is in registers: its slot takes the next one
        if (threadIdx.x == 0 && j + slots < mine) load(j + slots, slot);
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
        top = __reduce_max_sync(FULL, lane < blockDim.x / 32 ? s_max[j & 1][lane] : 0u);
        const Scale s(top);
        if (warp == 0) target.put_scale(s.value());
#pragma unroll
        for (int h = 0; h < HOLD; ++h)
            if (h * blockDim.x < n) target.put(s.codes(held[h]), threadIdx.x + h * blockDim.x, n);
    }
    if (j < mine && threadIdx.x == 0)  // given up: what was asked for lands before the ring is released
        for (int i = j; i < mine && i < j + slots; ++i) mbar_drain(smem_u32(&bars[i % slots]), (i / slots) & 1);
}

template <typename In, bool GLU, bool PLACE>
cudaError_t launch(const I8QuantArgs &a, cudaStream_t st) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | a.ldx * sizeof(In) | (GLU ? static_cast<size_t>(a.k) * sizeof(In) : 0);
    const int align = at & 15 ? 1 : at & 31 ? 16 : 32;
    const int n = (a.k + 15) / 16;
    const size_t staged = align < 16 ? static_cast<size_t>(n) * 16 * (GLU ? 2 : 1) * sizeof(In) : 0;  // bytes of a row in shared memory
    if (n <= HOLD * 32)
        return launch_early(i8_quantize_kernel<In, GLU, true, PLACE>, dim3((static_cast<unsigned>(a.src_rows) + WARP_ROWS - 1) / WARP_ROWS), 32 * WARP_ROWS,
                            WARP_ROWS * staged, st, 1, a, align, staged > 0);
    auto threads_for = [n](int hold) { return std::min(((n + hold - 1) / hold + 31) / 32 * 32, MOST_T); };
    const size_t row = static_cast<size_t>(a.k) * (GLU ? 2 : 1) * sizeof(In);
    if (a.src_rows >= RING_ROWS && align >= 16 && row % 16 == 0 && n > RING_HOLD<In, GLU> * 32 && n <= RING_HOLD<In, GLU> * MOST_T && 2 * row <= RING_SMEM) {
        const int threads = threads_for(RING_HOLD<In, GLU>);
        auto kernel = i8_quantize_ring_kernel<In, GLU, PLACE>;
        static std::atomic<uint64_t> ready{0};
        const cudaError_t e = allow_smem(kernel, RING_SMEM, ready);
        if (e != cudaSuccess) return e;
        const int ctas = static_cast<int>(std::min<size_t>(std::min(2 * MOST_T / threads, 16), RING_SMEM / (2 * row)));  // of an SM
        const int slots = static_cast<int>(std::min<size_t>(RING_SMEM / ctas / row, MOST_SLOTS));
        return launch_early(kernel, dim3(std::min(a.src_rows, device_sm_count() * ctas)), threads, slots * row, st, 1, a, static_cast<int>(row), slots);
    }
    const bool fits = staged > 0 && staged <= 44 * 1024 && n <= HOLD * MOST_T;  // (of the 48 KB that need no attribute)
    return launch_early(i8_quantize_kernel<In, GLU, false, PLACE>, dim3(a.src_rows), threads_for(HOLD), fits ? staged : 0, st, 1, a, align,
                        fits);
}

}  // namespace

template <typename In>
static cudaError_t launch_of(bool glu, const I8QuantArgs &a, cudaStream_t st) {
    if (a.place) return glu ? launch<In, true, true>(a, st) : launch<In, false, true>(a, st);
    return glu ? launch<In, true, false>(a, st) : launch<In, false, false>(a, st);
}

cudaError_t launch_i8_quantize(int act, bool glu, const I8QuantArgs &a, cudaStream_t st) {
    return act == COLI_ACT_F32 ? launch_of<float>(glu, a, st) : launch_of<uint16_t>(glu, a, st);
}

}  // namespace coli
