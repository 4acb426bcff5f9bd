// chunk.h -- 16 elements of a row in a thread's registers, loaded in whole sectors (the quantisers).  All names
// stay local to the including .cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace coli {
namespace {

// Two float32 values in one register pair.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }

// 32 bytes by one thread: whole sectors in one request (both at 32-byte boundaries).
__device__ __forceinline__ void load32(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
}
__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// 16 elements in their own type
template <typename In> struct Chunk;
template <> struct Chunk<float> {
    float v[16];
    __device__ __forceinline__ void load(const float *p, bool wide) {
        if (wide) {
            uint32_t a[8], b[8];
            load32(p, a);
            load32(p + 8, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = __uint_as_float(a[i]);
                v[8 + i] = __uint_as_float(b[i]);
            }
            return;
        }
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
    __device__ __forceinline__ uint64_t negated(int i) const { return pack2(-v[2 * i], -v[2 * i + 1]); }  // elements 2 i, 2 i + 1
};
template <> struct Chunk<uint16_t> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const uint16_t *p, bool wide) {
        if (wide) {
            load32(p, w);
            return;
        }
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
    __device__ __forceinline__ uint64_t negated(int i) const {
        const uint32_t n = w[i] ^ 0x80008000u;
        return pack2(__uint_as_float(n << 16), __uint_as_float(n & 0xffff0000u));
    }
};

constexpr uint32_t INF_BITS = 0x7f800000u;

}  // namespace
}  // namespace coli
