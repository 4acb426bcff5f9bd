// fp4.h -- microscaled 4-bit operands: sizes, and the launch parameters shared by the quantiser,
// the product and the expert path that calls them (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

constexpr int FP4_KB = 256;  // elements of a k-block: 128 bytes of codes per row

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == COLI_FP4_MX ? 32 : 16; }
// bytes of a row of block scales: whole k-blocks
__host__ __device__ constexpr size_t fp4_pitch(int fmt, int k) {
    return static_cast<size_t>((k + FP4_KB - 1) / FP4_KB) * (FP4_KB / fp4_block(fmt));
}
__host__ __device__ constexpr size_t fp4_scale_bytes(int fmt, int layout, int rows, int k) {
    return (layout == COLI_FP4_TILES ? (static_cast<size_t>(rows) + 127) / 128 * 128 : static_cast<size_t>(rows)) * fp4_pitch(fmt, k);
}

struct Fp4QuantArgs {
    const void *x;
    int src_rows;
    size_t ldx;                 // elements
    const int32_t *row_index;   // source row of output row r: row_index[r] / row_div (nullptr: r)
    int n_index, row_div;       // rows from n_index on: source row r - n_index
    int32_t *inverse;           // inverse[row_index[r]] = r, or nullptr
    int rows, k;
    uint8_t *codes, *scales;
    float *row_scale;
    int *err;
};
cudaError_t launch_fp4_quantize(int fmt, int layout, int act, const Fp4QuantArgs &a, cudaStream_t st);
cudaError_t launch_fp4_dequantize(int fmt, int layout, const uint8_t *codes, const uint8_t *scales, const float *row_scale,
                                  int rows, int k, int act, void *out, size_t ldo, cudaStream_t st);

// What the product's epilogue writes: the sums in float32 or bf16, or SwiGLU of gate and up sums in
// bf16 (weight rows in runs of 16 gate rows and the same 16 up rows; out has n / 2 columns).
enum { FP4_OUT_F32 = 0, FP4_OUT_BF16 = 1, FP4_OUT_SWIGLU = 2 };

struct Fp4ProductArgs {
    coli_fp4_rows a;
    coli_fp4_mats w;
    const coli_fp4_mats *shared;  // one more matrix for the rows offsets[count] .. a.rows - 1, or nullptr
    int k;
    const int32_t *offsets;
    int out_kind;
    void *out;
    size_t ldo;                   // elements
    int *err;
};
cudaError_t launch_fp4_product(int fmt, const Fp4ProductArgs &p, cudaStream_t st);

}  // namespace coli
