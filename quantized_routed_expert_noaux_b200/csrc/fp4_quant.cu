// fp4_quant.cu -- rows to microscaled 4-bit floating point and back (coli_moe_fp4_quantize,
// coli_moe_fp4_dequantize).
//
// A thread takes chunks of 16 elements: one NV block, or half an MX block whose other half is its
// neighbour lane's.  The row's chunks stay in registers between the pass that finds the row's
// largest value (NV) and the one that writes, up to HOLD chunks per thread; longer rows read
// the rest again, from L2.
//
// Exactness.  The row scale r and the MX block scale are powers of two, so x / r and x / 2^e are
// exact.  NV: y = x / r is divided by the e4m3 block scale s.  A quotient rounded to 24 bits never
// lands on a midpoint m of two codes unless y / s is that midpoint: m * s has at most 7 bits and is
// a float32, so another y differs from it by a unit in its last place, and the quotient from m by
// more than half a unit of its own.  So rounding the correctly rounded quotient to a code equals
// rounding the real one; the same holds for (largest |x| / r) / 6 and e4m3.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"
#include "internal.h"

namespace coli {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int QT = 128;   // threads per CTA
constexpr int HOLD = 4;   // chunks a thread keeps in registers

// 16 elements in their own type
template <typename In> struct Chunk;
template <> struct Chunk<float> {
    float v[16];
    __device__ __forceinline__ void load(const float *p) {
        const float4 *q = reinterpret_cast<const float4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = __ldg(q + i);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    // bits of the largest magnitude as a float32 (>= 0x7f800000 when one is not finite)
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ float at(int i) const { return v[i]; }
};
template <> struct Chunk<uint16_t> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const uint16_t *p) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        return max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

constexpr uint32_t INF_BITS = 0x7f800000u;

// two values -> two e2m1 codes, `lo` in the low nibble (round to nearest even, saturating at 6)
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{ .reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %1, %2; cvt.u32.u8 %0, c; }" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3(float v) {  // v >= 0
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {  // sign bit clear
    const uint32_t e = b >> 3, m = b & 7u;
    return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0.001953125f;
}

__device__ __forceinline__ size_t scale_at(int layout, size_t pitch, int r, int j) {
    return layout == COLI_FP4_ROWS ? static_cast<size_t>(r) * pitch + j
                                   : static_cast<size_t>(r >> 7) * 128 * pitch + static_cast<size_t>(j >> 2) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j & 3);
}

// One chunk: its block scale and codes.  `m`: bits of the block's largest magnitude; `rinv`: 1 / row
// scale (NV).
template <int FMT, typename In>
__device__ __forceinline__ void encode(const Chunk<In> &c, uint32_t m, float rinv, uint2 &codes, uint32_t &scale) {
    codes = make_uint2(0u, 0u);
    if (m >= INF_BITS) {  // a NaN or an infinity
        scale = FMT == COLI_FP4_MX ? 0xffu : 0x7fu;
        return;
    }
    uint32_t w[2] = {0u, 0u};
    if (FMT == COLI_FP4_MX) {
        const int e = max(static_cast<int>(m >> 23) - 2, 0);
        scale = e;
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2] |= e2m1x2(c.at(2 * i) * inv, c.at(2 * i + 1) * inv) << (8 * (i & 3));
    } else {
        scale = e4m3(__fdiv_rn(__uint_as_float(m) * rinv, 6.0f));
        if (scale == 0u) return;
        const float s = e4m3_value(scale);
        const float z = __frcp_rn(s);
        // the correctly rounded y / s from the correctly rounded 1 / s (Markstein, "Computation of
        // elementary functions on the IBM RISC System/6000 processor", 1990)
        auto quotient = [&](float x) {
            const float y = x * rinv, q = y * z;
            return fmaf(-fmaf(q, s, -y), z, q);  // (signs placed so that -0 stays -0)
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2] |= e2m1x2(quotient(c.at(2 * i)), quotient(c.at(2 * i + 1))) << (8 * (i & 3));
    }
    codes = make_uint2(w[0], w[1]);
}

// TPR threads per row, QT / TPR rows per CTA.
template <int FMT, int TPR, typename In>
__global__ void __launch_bounds__(QT) fp4_quant_kernel(const Fp4QuantArgs a, int layout, int out_rows) {
    __shared__ uint32_t s_max[QT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.x * (QT / TPR) + threadIdx.x / TPR, i0 = threadIdx.x % TPR;
    const int n = a.k / 16;  // chunks of a row
    const size_t pitch = fp4_pitch(FMT, a.k);
    bool live = r < a.rows;
    int src = r;
    if (live && a.row_index) {
        if (r < a.n_index) {
            const int s = __ldg(a.row_index + r);
            src = s / a.row_div;
            if (s < 0 || src >= a.src_rows) {
                if (i0 == 0) atomicOr(a.err, COLI_DEVERR_GROUPING);
                src = -1;
            } else if (a.inverse && i0 == 0) {
                a.inverse[s] = r;
            }
        } else {
            src = r - a.n_index;
        }
    }
    const bool read = live && src >= 0;
    const void *base = a.x;
    if (a.x_up) {
        if (r & 16) base = a.x_up;
        src = (r >> 5) * 16 + (r & 15);
    }
    const In *row = static_cast<const In *>(base) + static_cast<size_t>(read ? src : 0) * a.ldx;
    // every lane takes the same number of rounds: neighbours exchange their halves of an MX block
    const int rounds = (n + TPR - 1) / TPR;
    Chunk<In> held[HOLD];
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        const int i = i0 + h * TPR;
        if (read && i < n) held[h].load(row + 16 * static_cast<size_t>(i));
        else held[h].zero();
    }
    float rinv = 1.f, rs = 1.f;
    if (FMT == COLI_FP4_NV) {
        uint32_t top = 0u;
#pragma unroll
        for (int h = 0; h < HOLD; ++h) {
            const uint32_t m = held[h].amax();
            if (m < INF_BITS) top = max(top, m);
        }
        for (int h = HOLD; h < rounds; ++h) {
            const int i = i0 + h * TPR;
            if (read && i < n) {
                Chunk<In> c;
                c.load(row + 16 * static_cast<size_t>(i));
                const uint32_t m = c.amax();
                if (m < INF_BITS) top = max(top, m);
            }
        }
        top = __reduce_max_sync(FULL, top);
        if (TPR > 32) {
            if (lane == 0) s_max[warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < QT / 32; ++w) top = max(top, s_max[w]);
        }
        if (top) {
            const uint32_t e = max(static_cast<int>(top >> 23) - 10, 1);
            rs = __uint_as_float(e << 23);
            rinv = __uint_as_float((254u - e) << 23);
        }
    }
    if (live && i0 == 0 && a.row_scale) a.row_scale[r] = rs;
    auto put = [&](const Chunk<In> &c, int i) {
        uint32_t m = c.amax();
        if (FMT == COLI_FP4_MX) m = max(m, __shfl_xor_sync(FULL, m, 1));
        if (!live || i >= n) return;
        uint2 codes;
        uint32_t scale;
        encode<FMT, In>(c, m, rinv, codes, scale);
        *reinterpret_cast<uint2 *>(a.codes + static_cast<size_t>(r) * (a.k / 2) + 8 * static_cast<size_t>(i)) = codes;
        if (FMT == COLI_FP4_NV) a.scales[scale_at(layout, pitch, r, i)] = static_cast<uint8_t>(scale);
        else if (!(i & 1)) a.scales[scale_at(layout, pitch, r, i >> 1)] = static_cast<uint8_t>(scale);
    };
#pragma unroll
    for (int h = 0; h < HOLD; ++h)
        if (h < rounds) put(held[h], i0 + h * TPR);
    for (int h = HOLD; h < rounds; ++h) {
        const int i = i0 + h * TPR;
        Chunk<In> c;
        if (read && i < n) c.load(row + 16 * static_cast<size_t>(i));
        else c.zero();
        put(c, i);
    }
    // bytes behind the row's last block, and the rows that fill up the last tile
    if (r < out_rows)
        for (int j = (live ? a.k / fp4_block(FMT) : 0) + i0; j < static_cast<int>(pitch); j += TPR)
            a.scales[scale_at(layout, pitch, r, j)] = 0;
}

template <typename Out>
__device__ __forceinline__ void store16(Out *p, const float *v);
template <>
__device__ __forceinline__ void store16<float>(float *p, const float *v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <>
__device__ __forceinline__ void store16<uint16_t>(uint16_t *p, const float *v) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// code 0..15 -> value: e2m1 magnitude from its bits (exponent 0: 0 or 0.5)
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const uint32_t b = e ? ((e + 126u) << 23) | (m << 22) : (m ? 0x3f000000u : 0u);
    return __uint_as_float(b | (c >> 3 << 31));
}

template <int FMT, typename Out>
__global__ void __launch_bounds__(QT) fp4_dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                         const float *__restrict__ row_scale, int layout, int rows, int k,
                                                         Out *__restrict__ out, size_t ldo) {
    const int n = k / 16;
    const size_t pitch = fp4_pitch(FMT, k);
    const size_t total = static_cast<size_t>(rows) * n;
    for (size_t at = static_cast<size_t>(blockIdx.x) * QT + threadIdx.x; at < total; at += static_cast<size_t>(gridDim.x) * QT) {
        const int r = static_cast<int>(at / n), i = static_cast<int>(at % n);
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes) + at);
        const uint32_t b = scales[scale_at(layout, pitch, r, FMT == COLI_FP4_NV ? i : i >> 1)];
        float s;
        if (FMT == COLI_FP4_MX) s = __uint_as_float(b == 0xffu ? 0x7fc00000u : (b ? b << 23 : 0x00400000u));
        else s = (b & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : e4m3_value(b & 0x7fu);
        const float rs = row_scale ? __ldg(row_scale + r) : 1.f;
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = e2m1_value(((j < 8 ? c.x : c.y) >> (4 * (j & 7))) & 15u) * s * rs;
        store16<Out>(out + static_cast<size_t>(r) * ldo + 16 * static_cast<size_t>(i), v);
    }
}

template <int FMT, typename In>
cudaError_t launch_quant(int layout, const Fp4QuantArgs &a, cudaStream_t st) {
    const int out_rows = layout == COLI_FP4_TILES ? (a.rows + 127) / 128 * 128 : a.rows;
    if (a.k <= 1024) {
        fp4_quant_kernel<FMT, 32, In><<<(out_rows + QT / 32 - 1) / (QT / 32), QT, 0, st>>>(a, layout, out_rows);
    } else {
        fp4_quant_kernel<FMT, QT, In><<<out_rows, QT, 0, st>>>(a, layout, out_rows);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, int layout, int act, const Fp4QuantArgs &a, cudaStream_t st) {
    if (fmt == COLI_FP4_MX)
        return act == COLI_ACT_F32 ? launch_quant<COLI_FP4_MX, float>(layout, a, st) : launch_quant<COLI_FP4_MX, uint16_t>(layout, a, st);
    return act == COLI_ACT_F32 ? launch_quant<COLI_FP4_NV, float>(layout, a, st) : launch_quant<COLI_FP4_NV, uint16_t>(layout, a, st);
}

cudaError_t launch_fp4_dequantize(int fmt, int layout, const uint8_t *codes, const uint8_t *scales, const float *row_scale,
                                  int rows, int k, int act, void *out, size_t ldo, cudaStream_t st) {
    const size_t total = static_cast<size_t>(rows) * (k / 16);
    const size_t want = (total + QT - 1) / QT, most = static_cast<size_t>(device_sm_count()) * 16 * 4;
    const int grid = static_cast<int>(want < most ? want : most);
    if (fmt == COLI_FP4_MX) {
        if (act == COLI_ACT_F32) fp4_dequant_kernel<COLI_FP4_MX, float><<<grid, QT, 0, st>>>(codes, scales, row_scale, layout, rows, k, static_cast<float *>(out), ldo);
        else fp4_dequant_kernel<COLI_FP4_MX, uint16_t><<<grid, QT, 0, st>>>(codes, scales, row_scale, layout, rows, k, static_cast<uint16_t *>(out), ldo);
    } else {
        if (act == COLI_ACT_F32) fp4_dequant_kernel<COLI_FP4_NV, float><<<grid, QT, 0, st>>>(codes, scales, row_scale, layout, rows, k, static_cast<float *>(out), ldo);
        else fp4_dequant_kernel<COLI_FP4_NV, uint16_t><<<grid, QT, 0, st>>>(codes, scales, row_scale, layout, rows, k, static_cast<uint16_t *>(out), ldo);
    }
    return cudaGetLastError();
}

}  // namespace coli
