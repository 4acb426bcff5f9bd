// sorted_rows.h -- slots sorted by expert, their rows, and the weighted sum back with its gradient: launch
// parameters (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

struct SortArgs {
    const int32_t *ids;    // [T * K]
    int T, K, E;
    int32_t *offsets, *perm, *place;
    // the rows (x nullptr: none)
    const void *x;
    int hidden;
    size_t ldx, ldr;       // elements
    void *rows;
    int *err;
};
cudaError_t launch_sort_rows(int act, const SortArgs &a, cudaStream_t st);

struct CombineArgs {
    const void *y;         // [rows][hidden]
    int rows, T, K, hidden;
    size_t ldy;
    const int32_t *place;  // [T][K]
    const float *w;        // [T][K] or nullptr
    const void *add;       // [T][hidden] or nullptr
    void *out;
    size_t ld_add, ldo;
    int *err;
};
cudaError_t launch_combine(int act, int out_type, const CombineArgs &a, cudaStream_t st);

struct CombineGradArgs {
    const void *y;         // [rows][hidden]; nullptr where dw is
    int rows, T, K, hidden;
    size_t ldy;
    const int32_t *place;
    const float *w;        // [T][K] or nullptr
    const void *dout;      // [T][hidden]
    void *dy;              // [rows][hidden] or nullptr
    float *dw;             // [T][K] or nullptr
    size_t ld_dout, ld_dy;
    int *err;
};
cudaError_t launch_combine_grad(int act, int out_type, const CombineGradArgs &a, cudaStream_t st);

}  // namespace coli
