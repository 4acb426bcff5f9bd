// i8_quant.cu -- rows to 8-bit integers with one scale each (coli_moe_i8_quantize), SwiGLU of gate and up rows first
// where asked for, every row written to the places of its copies.
//
// scale = m / 127, m = the row's largest |x| (at least 127 * 2^-126); code = the whole number nearest to x / (m / 127) of
// the real numbers, ties to even.  y = x * fl(127 / m) is at most 2^-16 off the real quotient (|y| <= 127, two
// roundings of 2^-24), so its nearest whole number is the right one unless y lies within 2^-15 of a half.  A chunk that
// holds such a y is decided exactly: 127 |x| against (i + 1/2) m, both of at most 32 bits, exact in float64.
//
// A thread takes chunks of 16 elements; the row's chunks stay in registers between the pass that finds m
// and the one that writes, up to HOLD of them; longer rows read the rest again, from L2.
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
constexpr int QT = 128;   // threads per CTA
constexpr int HOLD = 4;   // chunks a thread keeps in registers

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
        for (int j = 0; j < 16; ++j) h.v[j] = g.at(j) / (1.0f + expf(-g.at(j))) * u.at(j);
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
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = h.at(i) * inv, r = y + ROUND;
        off = fmaxf(off, fabsf(y - (r - ROUND)));
        b[i] = __float_as_uint(r);
    }
    if (off > BORDER) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = h.at(i), y = fabsf(x * inv), f = floorf(y);
            if (fabsf(y - f - 0.5f) < 1.0f / 16384.0f) {
                const double a = 127.0 * static_cast<double>(fabsf(x)), half = (static_cast<double>(f) + 0.5) * static_cast<double>(m);
                int c = static_cast<int>(f);
                c += a > half || (a == half && (c & 1));
                b[i] = static_cast<uint32_t>(x < 0.f ? -c : c);
            }
        }
    }
    return make_uint4(pack4(b), pack4(b + 4), pack4(b + 8), pack4(b + 12));
}

template <typename In, bool GLU, int TPR>
__global__ void __launch_bounds__(QT) i8_quantize_kernel(const I8QuantArgs a, int align) {
    using Held = typename Source<In, GLU>::Held;
    __shared__ uint32_t s_max[QT / 32];
    wait_for_previous();
    const int lane = threadIdx.x & 31, i0 = threadIdx.x % TPR;
    const int r = blockIdx.x * (QT / TPR) + threadIdx.x / TPR;
    const bool live = r < a.src_rows;
    const int n = (a.k + 15) / 16, rounds = (n + TPR - 1) / TPR;
    const In *row = static_cast<const In *>(a.x) + static_cast<size_t>(live ? r : 0) * a.ldx;
    Held held[HOLD];
    uint32_t top = 0u;
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        held[h].zero();
        if (h < rounds && live && i0 + h * TPR < n) fetch<In, GLU>(held[h], row, a.k, i0 + h * TPR, align);
    }
#pragma unroll
    for (int h = 0; h < HOLD; ++h) top = max(top, held[h].amax());
    for (int i = i0 + HOLD * TPR; live && i < n; i += TPR) {
        Held c;
        fetch<In, GLU>(c, row, a.k, i, align);
        top = max(top, c.amax());
    }
    top = __reduce_max_sync(FULL, top);
    if (TPR > 32) {
        if (lane == 0) s_max[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < QT / 32; ++w) top = max(top, s_max[w]);
    }
    if (!live) return;
    const bool finite = top < INF_BITS;
    const float m = fmaxf(__uint_as_float(top), 127.0f * 0x1p-126f);
    const float scale = finite ? __fdiv_rn(m, 127.0f) : __uint_as_float(0x7fffffffu), inv = finite ? __fdiv_rn(127.0f, m) : 0.f;
    const int32_t *places = a.place ? a.place + static_cast<size_t>(r) * a.copies : nullptr;
    auto put = [&](const Held &h, int i) {
        const uint4 v = finite ? encode(h, m, inv) : make_uint4(0u, 0u, 0u, 0u);
        for (int c = 0; c < a.copies; ++c) {
            const int to = places ? __ldg(places + c) : r;
            if (to >= 0 && to < a.rows) *reinterpret_cast<uint4 *>(a.codes + static_cast<size_t>(to) * a.ldc + 16 * static_cast<size_t>(i)) = v;
        }
    };
#pragma unroll
    for (int h = 0; h < HOLD; ++h)
        if (i0 + h * TPR < n) put(held[h], i0 + h * TPR);
    for (int i = i0 + HOLD * TPR; i < n; i += TPR) {
        Held c;
        fetch<In, GLU>(c, row, a.k, i, align);
        put(c, i);
    }
    for (int c = i0; c < a.copies; c += TPR) {
        const int to = places ? __ldg(places + c) : r;
        if (to >= 0 && to < a.rows) a.row_scale[to] = scale;
        else if (to != -1) atomicOr(a.err, COLI_DEVERR_GROUPING);
    }
}

template <typename In, bool GLU>
cudaError_t launch(const I8QuantArgs &a, cudaStream_t st) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | a.ldx * sizeof(In) | (GLU ? static_cast<size_t>(a.k) * sizeof(In) : 0);
    const int align = at & 15 ? 1 : at & 31 ? 16 : 32;
    // a warp to a row that fits its registers, else four
    if (a.k <= 16 * HOLD * 32)
        return launch_early(i8_quantize_kernel<In, GLU, 32>, dim3((static_cast<unsigned>(a.src_rows) + 3) / 4), QT, 0, st, 1, a, align);
    return launch_early(i8_quantize_kernel<In, GLU, QT>, dim3(a.src_rows), QT, 0, st, 1, a, align);
}

}  // namespace

cudaError_t launch_i8_quantize(int act, bool glu, const I8QuantArgs &a, cudaStream_t st) {
    if (act == COLI_ACT_F32) return glu ? launch<float, true>(a, st) : launch<float, false>(a, st);
    return glu ? launch<uint16_t, true>(a, st) : launch<uint16_t, false>(a, st);
}

}  // namespace coli
