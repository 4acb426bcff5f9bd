// route_scores.h -- launcher of the router from scores (not installed).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

cudaError_t launch_route_scores(const coli_moe_router &r, const void *logits, size_t ld, const float *bias, int T,
                                int32_t *ids, float *w, cudaStream_t st);

}  // namespace coli
