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
    const void *x_up = nullptr; // packing a record: rows 32 j + 16 + i come from row 16 j + i of x_up, 32 j + i of x
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
    int shared_rows;              // how many those are when every row has its group
    int k;
    const int32_t *offsets;
    int out_kind;
    void *out;
    size_t ldo;                   // elements
    int *err;
};
cudaError_t launch_fp4_product(int fmt, const Fp4ProductArgs &p, cudaStream_t st);

// Records in 4-bit containers: byte offsets of the parts, and the record's bytes.
struct Fp4Record {
    size_t w1, wd, s1, sd, r1, rd, bytes;
};
inline bool fp4_wfmt(int wfmt) { return wfmt == COLI_W_MXFP4 || wfmt == COLI_W_NVFP4; }
inline int fp4_of(int wfmt) { return wfmt == COLI_W_MXFP4 ? COLI_FP4_MX : COLI_FP4_NV; }
inline Fp4Record fp4_record(int hidden, int inter, int wfmt) {
    const size_t H = hidden, I = inter;
    const int f = fp4_of(wfmt);
    const bool rows = f == COLI_FP4_NV;
    Fp4Record r;
    r.w1 = 0;
    r.wd = r.w1 + I * H;
    r.s1 = r.wd + H * I / 2;
    r.sd = r.s1 + fp4_scale_bytes(f, COLI_FP4_TILES, 2 * inter, hidden);
    r.r1 = r.sd + fp4_scale_bytes(f, COLI_FP4_TILES, hidden, inter);
    r.rd = r.r1 + (rows ? 2 * I * 4 : 0);
    r.bytes = r.rd + (rows ? H * 4 : 0);
    return r;
}

// The expert half over such records (fp4_ffn.cu): buffers of the workspace.
struct Fp4Buffers {
    uint8_t *xc, *xs;  // [slots]: x of each slot's token
    float *xr;
    void *h;           // [slots][I] bf16
    uint8_t *hc, *hs;
    float *hr;
    void *y;           // [slots][H] bf16
    int32_t *inverse;  // [T*K]: position of a slot in the grouped order
};
struct FfnParams;
cudaError_t launch_ffn_fp4(const FfnParams &f, int wfmt, const Fp4Buffers &b, cudaStream_t st);

}  // namespace coli
