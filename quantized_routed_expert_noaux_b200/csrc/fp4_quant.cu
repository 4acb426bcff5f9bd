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
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "chunk.h"
#include "fp4.h"
#include "internal.h"
#include "pdl.h"

namespace coli {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int QT = 128;   // threads per CTA
constexpr int HOLD = 4;   // chunks a thread keeps in registers

// Two float32 operations in one instruction.
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

// eight values -> eight e2m1 codes, the first in the lowest nibble (round to nearest even, saturating at 6)
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// the two codes of byte `i` of w as two halves
template <int I>
__device__ __forceinline__ float2 e2m1x2_values(uint32_t w) {
    uint32_t h;
    if (I == 0) asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a; }" : "=r"(h) : "r"(w));
    if (I == 1) asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(h) : "r"(w));
    if (I == 2) asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, c; }" : "=r"(h) : "r"(w));
    if (I == 3) asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, d; }" : "=r"(h) : "r"(w));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ uint32_t e4m3(float v) {  // v >= 0
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {  // sign bit clear; 0x7f is NaN
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}
// The correctly rounded x / s from z, the correctly rounded 1 / s (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990); signs placed so that -0 stays -0.
__device__ __forceinline__ float quotient(float x, float s, float z) {
    const float q = x * z;
    return fmaf(-fmaf(q, s, -x), z, q);
}

__device__ __forceinline__ size_t scale_at(int layout, size_t pitch, int r, int j) {
    return layout == COLI_FP4_ROWS ? static_cast<size_t>(r) * pitch + j
                                   : static_cast<size_t>(r >> 7) * 128 * pitch + static_cast<size_t>(j >> 2) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j & 3);
}

// One chunk: its block scale and codes.  `m`: bits of the block's largest magnitude; `rs`, `rinv`: the
// row scale and its inverse (NV).
template <int FMT, typename In>
__device__ __forceinline__ void encode(const Chunk<In> &c, uint32_t m, float rs, float rinv, uint2 &codes, uint32_t &scale) {
    codes = make_uint2(0u, 0u);
    if (m >= INF_BITS) {  // a NaN or an infinity
        scale = FMT == COLI_FP4_MX ? 0xffu : 0x7fu;
        return;
    }
    float v[16];
    if (FMT == COLI_FP4_MX) {
        const int e = max(static_cast<int>(m >> 23) - 2, 0);
        scale = e;
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = c.at(i) * inv;
    } else {
        scale = e4m3(quotient(__uint_as_float(m) * rinv, 6.0f, 1.0f / 6.0f));
        if (scale == 0u) return;
        const float s = e4m3_value(scale), z = __frcp_rn(s);
        if (rinv > 1e-30f && rinv < 1e30f) {
            // x / (r s): r is a power of two, so r s and 1 / (r s) are as exact as s and 1 / s
            const float sr = s * rs, zr = z * rinv;
            // two quotients at a time, from -x (the packed operations have no negated operand)
            const uint64_t s2 = pack2(sr, sr), z2 = pack2(-zr, -zr);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t y = c.negated(i), q = mul2(y, z2);
                unpack2(fma2(fma2(q, s2, y), z2, q), v[2 * i], v[2 * i + 1]);
            }
        } else {  // rows so large or small that r s or 1 / (r s) could leave float32's range
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = quotient(c.at(i) * rinv, s, z);
        }
    }
    codes = make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

// One row by TPR threads (thread i0 of them; a warp, or QT threads, s_max theirs, all of the CTA's threads in
// step): codes to `codes`, scale j
// to put_scale(j), the row scale returned.  `live`: there is a row; `read`: it has a source (zeros if not).
template <int FMT, int TPR, typename In, typename PutScale>
__device__ __forceinline__ float quantize_row(const In *row, bool live, bool read, bool wide, int n, int i0, uint32_t *s_max,
                                              uint8_t *codes, PutScale put_scale) {
    const int lane = threadIdx.x & 31;
    // every lane takes the same number of rounds: neighbours exchange their halves of an MX block
    const int rounds = (n + TPR - 1) / TPR;
    Chunk<In> held[HOLD];
    uint32_t most[HOLD];  // bits of their largest magnitudes
#pragma unroll
    for (int h = 0; h < HOLD; ++h) {
        const int i = i0 + h * TPR;
        if (h >= rounds) break;
        if (read && i < n) held[h].load(row + 16 * static_cast<size_t>(i), wide);
        else held[h].zero();
    }
    float rinv = 1.f, rs = 1.f;
    if (FMT == COLI_FP4_NV) {
        uint32_t top = 0u;
#pragma unroll
        for (int h = 0; h < HOLD; ++h)
            if (h < rounds) {
                most[h] = held[h].amax();
                if (most[h] < INF_BITS) top = max(top, most[h]);
            }
#pragma unroll 4
        for (int h = HOLD; h < rounds; ++h) {
            const int i = i0 + h * TPR;
            if (read && i < n) {
                Chunk<In> c;
                c.load(row + 16 * static_cast<size_t>(i), wide);
                const uint32_t m = c.amax();
                if (m < INF_BITS) top = max(top, m);
            }
        }
        top = __reduce_max_sync(FULL, top);
        if (TPR > 32) {
            if (lane == 0) s_max[(threadIdx.x >> 5) % (QT / 32)] = top;
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
    auto put = [&](const Chunk<In> &c, uint32_t m, int i) {
        if (FMT == COLI_FP4_MX) {
            m = c.amax();
            m = max(m, __shfl_xor_sync(FULL, m, 1));
        }
        if (!live || i >= n) return;
        uint2 q;
        uint32_t scale;
        encode<FMT, In>(c, m, rs, rinv, q, scale);
        *reinterpret_cast<uint2 *>(codes + 8 * static_cast<size_t>(i)) = q;
        if (FMT == COLI_FP4_NV) put_scale(i, static_cast<uint8_t>(scale));
        else if (!(i & 1)) put_scale(i >> 1, static_cast<uint8_t>(scale));
    };
#pragma unroll
    for (int h = 0; h < HOLD; ++h)
        if (h < rounds) put(held[h], most[h], i0 + h * TPR);
    for (int h = HOLD; h < rounds; ++h) {
        const int i = i0 + h * TPR;
        Chunk<In> c;
        if (read && i < n) c.load(row + 16 * static_cast<size_t>(i), wide);
        else c.zero();
        put(c, FMT == COLI_FP4_NV ? c.amax() : 0u, i);
    }
    return rs;
}

// TPR threads per row, QT / TPR rows per CTA.
template <int FMT, int TPR, typename In>
__global__ void __launch_bounds__(QT) fp4_quant_kernel(const Fp4QuantArgs a, int layout, int out_rows) {
    __shared__ uint32_t s_max[QT / 32];
    wait_for_previous();
    const int r = blockIdx.x * (QT / TPR) + threadIdx.x / TPR, i0 = threadIdx.x % TPR;
    const size_t pitch = fp4_pitch(FMT, a.k);
    const bool live = r < a.rows;
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
    const bool wide = ((reinterpret_cast<uintptr_t>(base) | a.ldx * sizeof(In)) & 31) == 0;
    const float rs = quantize_row<FMT, TPR, In>(row, live, read, wide, a.k / 16, i0, s_max, a.codes + static_cast<size_t>(r) * (a.k / 2),
                                                [&](int j, uint8_t v) { a.scales[scale_at(layout, pitch, r, j)] = v; });
    if (live && i0 == 0 && a.row_scale) a.row_scale[r] = rs;
    // bytes behind the row's last block, and the rows that fill up the last tile
    if (r < out_rows)
        for (int j = (live ? a.k / fp4_block(FMT) : 0) + i0; j < static_cast<int>(pitch); j += TPR)
            a.scales[scale_at(layout, pitch, r, j)] = 0;
}

// Rows of an index that takes every source row several times (the slots of a token's experts): a CTA
// quantises `per` source rows once, ST / TPR at a time, into shared memory, then goes through the whole index;
// a thread that meets one of them starts its bulk copies to the row that asks for it.  The index is read
// gridDim.x times, from L2.  Rows whose index is bad are the first CTA's, copies of a row of zeros.  16,384 rows of
// 6144 bf16 elements from 2048 (NV): 21 us against 47 with every row quantised by itself; 4096 rows from 512, 7
// against 13.
constexpr int ST = 256, SEG = 4096;
constexpr int SPREAD_SMEM = 88 * 1024;  // two CTAs per SM at least
constexpr int SPREAD_MIN = 1024;        // rows
constexpr int SPREAD_CTAS = 512;        // about, where shared memory allows it

template <int FMT, int TPR, typename In>
__global__ void __launch_bounds__(ST, sizeof(In) == 2 ? 4 : 2) fp4_spread_kernel(const Fp4QuantArgs a, int per) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ uint32_t s_max[ST / 32];
    wait_for_previous();
    const int tid = threadIdx.x;
    const int pitch = static_cast<int>(fp4_pitch(FMT, a.k)), half = a.k / 2;
    const int each = half + pitch;                      // bytes of a row in shared memory, a multiple of 16
    float *s_rs = reinterpret_cast<float *>(sm + static_cast<size_t>(per + 1) * each);  // (row `per`: zeros)
    const int t0 = blockIdx.x * per, nt = min(per, a.src_rows - t0);
    const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | a.ldx * sizeof(In)) & 31) == 0;
    for (int i0 = 0; i0 < nt; i0 += ST / TPR) {
        const int i = i0 + tid / TPR;
        const bool live = i < nt;
        unsigned char *codes = sm + (live ? i : 0) * each, *scales = codes + half;
        const In *row = static_cast<const In *>(a.x) + static_cast<size_t>(live ? t0 + i : 0) * a.ldx;
        const float rs = quantize_row<FMT, TPR, In>(row, live, live, wide, a.k / 16, tid % TPR, s_max + tid / TPR * (TPR / 32), codes,
                                                    [&](int j, uint8_t v) { scales[j] = v; });
        if (live) {
            for (int j = a.k / fp4_block(FMT) + tid % TPR; j < pitch; j += TPR) scales[j] = 0;
            if (tid % TPR == 0) s_rs[i] = rs;
        }
        __syncthreads();
    }
    for (int j = tid; j < each / 16; j += ST) reinterpret_cast<uint4 *>(sm + static_cast<size_t>(per) * each)[j] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_rs[per] = 1.f;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the bulk copies read what was just written
    __syncthreads();
    // row i of shared memory to output row r
    auto copy = [&](int i, int r) {
        const unsigned char *from = sm + i * each;
        uint8_t *c = a.codes + static_cast<size_t>(r) * half, *d = a.scales + static_cast<size_t>(r) * pitch;
        const uint32_t src = static_cast<uint32_t>(__cvta_generic_to_shared(from));
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(c), "r"(src), "r"(half) : "memory");
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(d), "r"(src + half), "r"(pitch) : "memory");
        if (a.row_scale) a.row_scale[r] = s_rs[i];
    };
    for (int i = tid; i < nt && a.n_index + t0 + i < a.rows; i += ST) copy(i, a.n_index + t0 + i);
    const long lo = static_cast<long>(t0) * a.row_div, hi = lo + static_cast<long>(nt) * a.row_div, end = static_cast<long>(a.src_rows) * a.row_div;
    for (int base = 0; base < a.n_index; base += SEG) {
        int v[SEG / ST];  // all of the segment's loads before the first test
#pragma unroll
        for (int i = 0; i < SEG / ST; ++i) v[i] = __ldg(a.row_index + min(base + i * ST + tid, a.n_index - 1));
#pragma unroll
        for (int i = 0; i < SEG / ST; ++i) {
            const int r = base + i * ST + tid, s = v[i];
            if (r < a.n_index) {
                if (s >= lo && s < hi) {
                    copy(static_cast<int>(static_cast<uint32_t>(s - lo) / static_cast<uint32_t>(a.row_div)), r);
                    if (a.inverse) a.inverse[s] = r;
                } else if (blockIdx.x == 0 && (s < 0 || s >= end)) {
                    copy(per, r);
                    atomicOr(a.err, COLI_DEVERR_GROUPING);
                }
            }
        }
    }
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

template <typename Out>
__device__ __forceinline__ void store16(Out *p, const float *v, bool wide);
template <>
__device__ __forceinline__ void store16<float>(float *p, const float *v, bool wide) {
    if (wide) {
        store32(p, reinterpret_cast<const uint32_t *>(v));
        store32(p + 8, reinterpret_cast<const uint32_t *>(v + 8));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <>
__device__ __forceinline__ void store16<uint16_t>(uint16_t *p, const float *v, bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    if (wide) {
        store32(p, w);
        return;
    }
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// TPR threads per row, QT / TPR rows per CTA at a time.
template <int FMT, int TPR, typename Out>
__global__ void __launch_bounds__(QT) fp4_dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                         const float *__restrict__ row_scale, int layout, int rows, int k,
                                                         Out *__restrict__ out, size_t ldo) {
    wait_for_previous();
    const int n = k / 16;
    const size_t pitch = fp4_pitch(FMT, k);
    const bool wide = ((reinterpret_cast<uintptr_t>(out) | ldo * sizeof(Out)) & 31) == 0;
    for (int r = blockIdx.x * (QT / TPR) + threadIdx.x / TPR; r < rows; r += gridDim.x * (QT / TPR)) {
        float rs = row_scale ? __ldg(row_scale + r) : 1.f, unit = 1.f;
        if (FMT == COLI_FP4_MX && fabsf(rs) < 1.f) {  // code * block scale may overflow (6 * 2^127) where the value does not
            unit = 0.25f;
            rs *= 4.f;
        }
        const uint2 *row = reinterpret_cast<const uint2 *>(codes) + static_cast<size_t>(r) * n;
        Out *o = out + static_cast<size_t>(r) * ldo;
        for (int i = threadIdx.x % TPR; i < n; i += TPR) {
            const uint2 c = __ldg(row + i);
            const uint32_t b = __ldg(scales + scale_at(layout, pitch, r, FMT == COLI_FP4_NV ? i : i >> 1));
            float s;
            if (FMT == COLI_FP4_MX) s = __uint_as_float(b == 0xffu ? 0x7fc00000u : (b ? b << 23 : 0x00400000u)) * unit;
            else s = e4m3_value(b & 0x7fu);
            float v[16];
            auto four = [&](uint32_t w, float *d) {
                const float2 e[4] = {e2m1x2_values<0>(w), e2m1x2_values<1>(w), e2m1x2_values<2>(w), e2m1x2_values<3>(w)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // code * block scale is exact: one rounding to float32, by the row scale
                    d[2 * j] = e[j].x * s * rs;
                    d[2 * j + 1] = e[j].y * s * rs;
                }
            };
            four(c.x, v);
            four(c.y, v + 8);
            store16<Out>(o + 16 * static_cast<size_t>(i), v, wide);
        }
    }
}

// Source rows per CTA of the spreading kernel; 0: every row by itself.  What each costs, in picoseconds: a row
// quantised once more, AGAIN per element; a row copied, 440 with every SM at work, 0.3 per element, and 1.17 for
// each CTA that reads its entry of the index.  The last is what limits the batch: shared memory holds a few rows,
// so the CTAs grow with the source rows, and their passes over the index with the square (262,144 rows of 6144
// bf16 elements, 8 times each: 30.4 ms, row by row 6.3; 2048 rows: 21 us against 47).  Both kernels were timed on
// 1522 sizes (both formats and types, 1024 to 2 million rows of 512 to 16,384 elements, 2 to 32 copies): the rule
// takes the slower one by more than 10% in 24 of them, by 23% at most; spreading always would in 460, by up to 2.5
// times.  Scales are copied in pieces of 16 bytes: MX rows with an odd number of k-blocks go row by row (by 8-byte
// stores the spreading kernel was never the faster one for them).
template <int FMT, typename In>
int spread_rows(int layout, const Fp4QuantArgs &a) {
    constexpr double AGAIN = FMT == COLI_FP4_MX ? (sizeof(In) == 4 ? 1.12 : 0.74) : (sizeof(In) == 4 ? 1.42 : 0.89);
    if (layout != COLI_FP4_ROWS || !a.row_index || a.src_rows == 0 || a.rows < SPREAD_MIN || a.rows / 2 < a.src_rows) return 0;
    const size_t pitch = fp4_pitch(FMT, a.k), each = a.k / 2 + pitch;
    if (pitch % 16 || (reinterpret_cast<uintptr_t>(a.codes) | reinterpret_cast<uintptr_t>(a.scales)) & 15) return 0;
    const int at_once = ST / (a.k <= 2048 ? 32 : QT), turns = (a.src_rows + at_once * SPREAD_CTAS - 1) / (at_once * SPREAD_CTAS);
    const int fit = static_cast<int>(SPREAD_SMEM / (each + sizeof(float))) - 1, per = fit < at_once * turns ? fit : at_once * turns;
    if (per < 1) return 0;
    const double rows = a.rows, k = a.k, ctas = (a.src_rows + per - 1) / per, sms = device_sm_count();
    return (rows - a.src_rows) * k * AGAIN > rows * (440.0 * (ctas < sms ? sms / ctas : 1.0) + 0.3 * k + 1.17 * ctas) ? per : 0;
}

template <int FMT, int TPR, typename In>
cudaError_t launch_spread(const Fp4QuantArgs &a, int per, cudaStream_t st) {
    const size_t smem = (per + 1) * (a.k / 2 + fp4_pitch(FMT, a.k) + sizeof(float));
    const cudaError_t e = cudaFuncSetAttribute(fp4_spread_kernel<FMT, TPR, In>, cudaFuncAttributeMaxDynamicSharedMemorySize, SPREAD_SMEM);
    if (e != cudaSuccess) return e;
    return launch_early(fp4_spread_kernel<FMT, TPR, In>, dim3((a.src_rows + per - 1) / per), ST, smem, st, 1, a, per);
}

template <int FMT, typename In>
cudaError_t launch_quant(int layout, const Fp4QuantArgs &a, cudaStream_t st) {
    if (const int per = spread_rows<FMT, In>(layout, a)) return a.k <= 2048 ? launch_spread<FMT, 32, In>(a, per, st) : launch_spread<FMT, QT, In>(a, per, st);
    const int out_rows = layout == COLI_FP4_TILES ? (a.rows + 127) / 128 * 128 : a.rows;
    if (a.k <= 2048) return launch_early(fp4_quant_kernel<FMT, 32, In>, dim3((out_rows + QT / 32 - 1) / (QT / 32)), QT, 0, st, 1, a, layout, out_rows);
    return launch_early(fp4_quant_kernel<FMT, QT, In>, dim3(out_rows), QT, 0, st, 1, a, layout, out_rows);
}

template <int FMT, int TPR>
cudaError_t launch_dequant_tpr(int layout, const uint8_t *codes, const uint8_t *scales, const float *row_scale, int rows, int k, int act,
                        void *out, size_t ldo, cudaStream_t st) {
    const int want = (rows + QT / TPR - 1) / (QT / TPR), most = device_sm_count() * 64;
    const int grid = want < most ? want : most;
    if (act == COLI_ACT_F32)
        return launch_early(fp4_dequant_kernel<FMT, TPR, float>, dim3(grid), QT, 0, st, 1, codes, scales, row_scale, layout, rows, k, static_cast<float *>(out), ldo);
    return launch_early(fp4_dequant_kernel<FMT, TPR, uint16_t>, dim3(grid), QT, 0, st, 1, codes, scales, row_scale, layout, rows, k, static_cast<uint16_t *>(out), ldo);
}

template <int FMT>
cudaError_t launch_dequant(int layout, const uint8_t *codes, const uint8_t *scales, const float *row_scale, int rows, int k, int act,
                           void *out, size_t ldo, cudaStream_t st) {
    if (k <= 1024) return launch_dequant_tpr<FMT, 32>(layout, codes, scales, row_scale, rows, k, act, out, ldo, st);
    return launch_dequant_tpr<FMT, QT>(layout, codes, scales, row_scale, rows, k, act, out, ldo, st);
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, int layout, int act, const Fp4QuantArgs &a, cudaStream_t st) {
    if (fmt == COLI_FP4_MX)
        return act == COLI_ACT_F32 ? launch_quant<COLI_FP4_MX, float>(layout, a, st) : launch_quant<COLI_FP4_MX, uint16_t>(layout, a, st);
    return act == COLI_ACT_F32 ? launch_quant<COLI_FP4_NV, float>(layout, a, st) : launch_quant<COLI_FP4_NV, uint16_t>(layout, a, st);
}

cudaError_t launch_fp4_dequantize(int fmt, int layout, const uint8_t *codes, const uint8_t *scales, const float *row_scale,
                                  int rows, int k, int act, void *out, size_t ldo, cudaStream_t st) {
    return fmt == COLI_FP4_MX ? launch_dequant<COLI_FP4_MX>(layout, codes, scales, row_scale, rows, k, act, out, ldo, st)
                              : launch_dequant<COLI_FP4_NV>(layout, codes, scales, row_scale, rows, k, act, out, ldo, st);
}

}  // namespace coli
