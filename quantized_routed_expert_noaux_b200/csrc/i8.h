// i8.h -- 8-bit operands: launch parameters of the quantiser and the product (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

// Sums of |a w| <= 2^14 stay in 32 bits up to this k.
constexpr int I8_MAX_K = (1 << 17) - 1;

struct I8QuantArgs {
    const void *x;
    int src_rows, k;
    size_t ldx;            // elements
    const int32_t *place;  // [src_rows][copies] or nullptr: row i -> row i
    int copies, rows;
    int8_t *codes;
    size_t ldc;            // bytes
    float *row_scale;
    int *err;
};
cudaError_t launch_i8_quantize(int act, bool glu, const I8QuantArgs &a, cudaStream_t st);

struct I8ProductArgs {
    coli_i8_rows a;
    coli_i8_mats w;
    int k;
    const int32_t *offsets;
    int out_type;
    void *out;
    size_t ldo;            // elements
    int *err;
};
cudaError_t launch_i8_product(const I8ProductArgs &p, cudaStream_t st);

}  // namespace coli
