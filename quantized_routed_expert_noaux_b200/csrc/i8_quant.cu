// i8_quant.cu -- rows to 8-bit integers with one scale each (coli_moe_i8_quantize), SwiGLU of gate and up rows first
// where asked for, every row written to the places of its copies.
//
// scale = m / 127, m = the row's largest |x| (at least 127 * 2^-126); code = the whole number nearest to x / (m / 127) of
// the real numbers, ties to even.  y = x * fl(127 / m) is at most 2^-16 off the real quotient (|y| <= 127, two
// roundings of 2^-24), so its nearest whole number is the right one unless y lies within 2^-15 of a half.  A chunk that
// holds such a y is decided exactly: 127 |x| against (i + 1/2) m.  With p = fl((i + 1/2) m) and e = (i + 1/2) m - p (an FMA gives
// it exactly), 127 |x| - p is a float32 too: the two are within 2^-13 of each other and 127 |x| has 31 bits; it is compared with
// e.  (Both sides over 128, and times 2^64 where m is below 1, so that nothing overflows or underflows.)
//
// A thread takes chunks of 16 elements; the row's chunks stay in registers between the pass that finds m
// and the one that writes, HOLD to a thread; what rows beyond HOLD * MOST_T chunks have more is read again, from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chunk.h"
#include "i8.h"
#include "internal.h"
#include "pdl.h"

namespace coli {

namespace {

constexpr unsigned FULL = 0xffffffffu;
#ifndef NB
#define NB 3
#define NF 2
#endif
constexpr int HOLD = 2;       // chunks a thread keeps in registers
constexpr int MOST_T = 384;   // threads of a row at most
constexpr int WARP_ROWS = 4;  // rows of a CTA where a warp takes a row

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
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
template <typename In>
__device__ __forceinline__ void load_chunk(Chunk<In> &c, const In *p, int n, int align) {
    if (n >= 16 && align >= 16) c.load(p, align >= 32);
    else load_some(c, p, n);
}

// What is quantised: the row's own elements, or SiLU(gate) * up in float32.
template <typename In, bool GLU> struct Source { using Held = Chunk<In>; };
template <typename In> struct Source<In, true> { using Held = Chunk<float>; };

template <typename In, bool GLU>
__device__ __forceinline__ void fetch(typename Source<In, GLU>::Held &h, const In *row, int k, int i, int align) {
    const int n = k - 16 * i;
    if constexpr (GLU) {
        Chunk<In> g, u;
        load_chunk(g, row + 16 * static_cast<size_t>(i), n, align);
        load_chunk(u, row + k + 16 * static_cast<size_t>(i), n, align);
#pragma unroll
        for (int j = 0; j < 16; ++j) h.v[j] = __fdividef(g.at(j), 1.0f + expf(-g.at(j))) * u.at(j);
    } else {
        load_chunk(h, row + 16 * static_cast<size_t>(i), n, align);
    }
}

constexpr float ROUND = 12582912.0f;                     // 1.5 * 2^23: added, the whole number is in the low bits
constexpr float BORDER = 0.5f - 1.0f / 32768.0f;

__device__ __forceinline__ uint32_t pack4(const uint32_t *b) {  // the low bytes of four words
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

template <typename Held>
__device__ __forceinline__ uint4 encode(const Held &h, float m, float inv) {
    uint32_t b[16];
    float off = 0.f;
    const uint64_t inv2 = pack2(inv, inv), up = pack2(ROUND, ROUND), down = pack2(-ROUND, -ROUND), minus = pack2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t y = mul2(pack2(h.at(2 * i), h.at(2 * i + 1)), inv2), r = add2(y, up);
        float lo, hi, d0, d1;
        unpack2(r, lo, hi);
        unpack2(fma2(add2(r, down), minus, y), d0, d1);  // what rounding took away, exactly
        off = fmaxf(off, fmaxf(fabsf(d0), fabsf(d1)));
        b[2 * i] = __float_as_uint(lo);
        b[2 * i + 1] = __float_as_uint(hi);
    }
    if (off > BORDER) {
        const float up64 = m < 1.f ? 0x1p64f : 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = h.at(i), y = fabsf(x * inv), f = floorf(y);
            if (fabsf(y - f - 0.5f) < 1.0f / 16384.0f) {
                const float g = (f + 0.5f) * 0x1p-7f, ms = m * up64, p = g * ms;
                const float e = fmaf(g, ms, -p), d = fmaf(127.0f * 0x1p-7f, fabsf(x) * up64, -p);
                int c = static_cast<int>(f);
                c += d > e || (d == e && (c & 1));
                b[i] = static_cast<uint32_t>(x < 0.f ? -c : c);
            }
        }
    }
    return make_uint4(pack4(b), pack4(b + 4), pack4(b + 8), pack4(b + 12));
}

// A row by a warp (WARP: WARP_ROWS rows to a CTA) or by a CTA.
template <typename In, bool GLU, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * WARP_ROWS : MOST_T, (WARP ? 3 : 1) * (sizeof(In) == 2 && !GLU ? NB : NF)) i8_quantize_kernel(const I8QuantArgs a, int align) {
    using Held = typename Source<In, GLU>::Held;
    __shared__ uint32_t s_max[MOST_T / 32];
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = WARP ? lane : threadIdx.x, tpr = WARP ? 32 : blockDim.x;
    const int r = WARP ? blockIdx.x * WARP_ROWS + warp : blockIdx.x;
    if (r >= a.src_rows) return;
    const int n = (a.k + 15) / 16;
    const In *row = static_cast<const In *>(a.x) + static_cast<size_t>(r) * a.ldx;
    Held held[HOLD];
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        if (i0 + h * tpr < n) fetch<In, GLU>(held[h], row, a.k, i0 + h * tpr, align);
        else held[h].zero();
    }
    const int32_t *places = a.place ? a.place + static_cast<size_t>(r) * a.copies : nullptr;
    const int first = places ? (lane < a.copies ? __ldg(places + lane) : -1) : (lane ? -1 : r);  // of the first 32 copies, one per lane
    uint32_t top = 0u;
#pragma unroll
    for (int h = 0; h < HOLD; ++h) top = max(top, held[h].amax());
    for (int i = i0 + HOLD * tpr; i < n; i += tpr) {
        Held c;
        fetch<In, GLU>(c, row, a.k, i, align);
        top = max(top, c.amax());
    }
    top = __reduce_max_sync(FULL, top);
    if (!WARP) {
        if (lane == 0) s_max[warp] = top;
        __syncthreads();
        top = __reduce_max_sync(FULL, lane < tpr / 32 ? s_max[lane] : 0u);
    }
    const bool finite = top < INF_BITS;
    const float m = fmaxf(__uint_as_float(top), 127.0f * 0x1p-126f);
    const float scale = finite ? __fdiv_rn(m, 127.0f) : __uint_as_float(0x7fffffffu), inv = finite ? __fdiv_rn(127.0f, m) : 0.f;
    auto where = [&](int c0) {  // of copies c0 .. c0 + 31, one per lane
        const int to = c0 == 0 ? first : c0 + lane < a.copies ? __ldg(places + c0 + lane) : -1;
        return to < -1 || to >= a.rows ? -1 : to;
    };
    if (WARP || warp == 0)
        for (int c0 = 0; c0 < a.copies; c0 += 32) {
            const int to = where(c0);
            if (to >= 0) a.row_scale[to] = scale;
            else if ((c0 == 0 ? first : c0 + lane < a.copies ? __ldg(places + c0 + lane) : -1) != -1) atomicOr(a.err, COLI_DEVERR_GROUPING);
        }
    uint4 code[HOLD];
#pragma unroll
    for (int h = 0; h < HOLD; ++h) code[h] = finite ? encode(held[h], m, inv) : make_uint4(0u, 0u, 0u, 0u);
    auto put = [&](const uint4 &v, int i) {
        const int at = where(0);
        for (int c0 = 0; c0 < a.copies; c0 += 32) {
            const int to = c0 == 0 ? at : where(c0);
            for (unsigned left = __ballot_sync(FULL, to >= 0); left; left &= left - 1) {
                const int row_to = __shfl_sync(FULL, to, __ffs(left) - 1);
                if (i < n) *reinterpret_cast<uint4 *>(a.codes + static_cast<size_t>(row_to) * a.ldc + 16 * static_cast<size_t>(i)) = v;
            }
        }
    };
#pragma unroll
    for (int h = 0; h < HOLD; ++h)
        if (h * tpr < n) put(code[h], i0 + h * tpr);
    for (int base = HOLD * tpr; base < n; base += tpr) {
        Held c;
        if (base + i0 < n) fetch<In, GLU>(c, row, a.k, base + i0, align);
        else c.zero();
        put(finite ? encode(c, m, inv) : make_uint4(0u, 0u, 0u, 0u), base + i0);
    }
}

template <typename In, bool GLU>
cudaError_t launch(const I8QuantArgs &a, cudaStream_t st) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | a.ldx * sizeof(In) | (GLU ? static_cast<size_t>(a.k) * sizeof(In) : 0);
    const int align = at & 15 ? 1 : at & 31 ? 16 : 32;
    const int n = (a.k + 15) / 16;
    if (n <= HOLD * 32)
        return launch_early(i8_quantize_kernel<In, GLU, true>, dim3((static_cast<unsigned>(a.src_rows) + WARP_ROWS - 1) / WARP_ROWS), 32 * WARP_ROWS, 0, st, 1, a, align);
    const int threads = (n + HOLD - 1) / HOLD;
    return launch_early(i8_quantize_kernel<In, GLU, false>, dim3(a.src_rows), threads < MOST_T ? (threads + 31) / 32 * 32 : MOST_T, 0, st, 1, a, align);
}

}  // namespace

cudaError_t launch_i8_quantize(int act, bool glu, const I8QuantArgs &a, cudaStream_t st) {
    if (act == COLI_ACT_F32) return glu ? launch<float, true>(a, st) : launch<float, false>(a, st);
    return glu ? launch<uint16_t, true>(a, st) : launch<uint16_t, false>(a, st);
}

}  // namespace coli
