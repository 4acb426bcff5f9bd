// fp4_ffn.cu -- a4..a7 over records in microscaled 4-bit containers: x of every slot's token to 4 bits
// (grouped order), one grouped product with SwiGLU for gate and up, h to 4 bits, one grouped product for
// down, and the weighted combine.  The shared expert is one more group of both products.
//
// The combine adds a token's experts in the order of its slots, then the shared expert: no atomics, the
// same bits every time.  It reads y in bf16: each term is rounded once more (2^-9 of it), which the 4-bit
// operands' own rounding (2^-3 of a value) hides, and half the bytes of float32 travel (2048 tokens, 9
// experts each, hidden 6144: 226 MB written and read instead of 453).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.h"
#include "internal.h"
#include "pdl.h"

namespace coli {

namespace {

constexpr int CT = 128;  // threads: 8 columns each

__global__ void __launch_bounds__(CT) fp4_combine_kernel(const __nv_bfloat16 *__restrict__ y, const float *__restrict__ w,
                                                         const int32_t *__restrict__ inverse, const int32_t *__restrict__ perm,
                                                         int T, int K, int S, int H, float *__restrict__ out) {
    wait_for_previous();
    const int t = blockIdx.x, c = (blockIdx.y * CT + threadIdx.x) * 8;
    if (c >= H) return;
    const int TK = T * K;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](int row, float f) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(y + static_cast<size_t>(row) * H + c));
        const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] = fmaf(f, __uint_as_float(v[i] << 16), acc[2 * i]);
            acc[2 * i + 1] = fmaf(f, __uint_as_float(v[i] & 0xffff0000u), acc[2 * i + 1]);
        }
    };
    for (int k = 0; k < K; ++k) {
        const int s = t * K + k;
        // a slot that the grouping did not place (an expert id out of range) has no position: what
        // `inverse` holds there is not perm's
        const int pos = __ldg(inverse + s);
        if (pos < 0 || pos >= TK || __ldg(perm + pos) != s) continue;
        add(pos, __ldg(w + s));
    }
    if (S) add(TK + t, 1.f);
    float4 *o = reinterpret_cast<float4 *>(out + static_cast<size_t>(t) * H + c);
    o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

}  // namespace

cudaError_t launch_ffn_fp4(const FfnParams &f, int wfmt, const Fp4Buffers &b, cudaStream_t st) {
    const int fmt = fp4_of(wfmt), TK = f.T * f.K, slots = TK + f.T * f.S;
    const Fp4Record r = fp4_record(f.H, f.I, wfmt);
    const bool rows = fmt == COLI_FP4_NV;
    cudaError_t e;

    Fp4QuantArgs a;
    a.x = f.x;
    a.src_rows = f.T;
    a.ldx = static_cast<size_t>(f.H);
    a.row_index = f.perm;
    a.n_index = TK;
    a.row_div = f.K;
    a.inverse = b.inverse;
    a.rows = slots;
    a.k = f.H;
    a.codes = b.xc;
    a.scales = b.xs;
    a.row_scale = b.xr;
    a.err = f.err;
    if ((e = launch_fp4_quantize(fmt, COLI_FP4_ROWS, f.act, a, st)) != cudaSuccess) return e;

    auto mats = [&](const uint8_t *rec, int count, bool down) {
        coli_fp4_mats m;
        m.codes = rec + (down ? r.wd : r.w1);
        m.scales = rec + (down ? r.sd : r.s1);
        m.row_scale = rows ? reinterpret_cast<const float *>(rec + (down ? r.rd : r.r1)) : nullptr;
        m.count = count;
        m.n = down ? f.H : 2 * f.I;
        m.codes_stride = m.scales_stride = f.stride;
        m.row_scale_stride = f.stride / 4;
        return m;
    };
    Fp4ProductArgs p;
    p.offsets = f.offsets;
    p.err = f.err;
    p.a = {b.xc, b.xs, rows ? b.xr : nullptr, slots};
    p.w = mats(f.experts, f.E, false);
    coli_fp4_mats shared = f.S ? mats(f.shared, 1, false) : p.w;
    p.shared = f.S ? &shared : nullptr;
    p.shared_rows = f.T * f.S;
    p.k = f.H;
    p.out_kind = FP4_OUT_SWIGLU;
    p.out = b.h;
    p.ldo = static_cast<size_t>(f.I);
    if ((e = launch_fp4_product(fmt, p, st)) != cudaSuccess) return e;

    a.x = b.h;
    a.src_rows = slots;
    a.ldx = static_cast<size_t>(f.I);
    a.row_index = nullptr;
    a.inverse = nullptr;
    a.k = f.I;
    a.codes = b.hc;
    a.scales = b.hs;
    a.row_scale = b.hr;
    if ((e = launch_fp4_quantize(fmt, COLI_FP4_ROWS, COLI_ACT_BF16, a, st)) != cudaSuccess) return e;

    p.a = {b.hc, b.hs, rows ? b.hr : nullptr, slots};
    p.w = mats(f.experts, f.E, true);
    if (f.S) shared = mats(f.shared, 1, true);
    p.k = f.I;
    p.out_kind = FP4_OUT_BF16;
    p.out = b.y;
    p.ldo = static_cast<size_t>(f.H);
    if ((e = launch_fp4_product(fmt, p, st)) != cudaSuccess) return e;

    return launch_early(fp4_combine_kernel, dim3(f.T, (f.H / 8 + CT - 1) / CT), CT, 0, st, 1, static_cast<const __nv_bfloat16 *>(b.y), f.topk_w, b.inverse,
                        f.perm, f.T, f.K, f.S, f.H, f.out);
}

}  // namespace coli
