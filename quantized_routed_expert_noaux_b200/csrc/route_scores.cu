// route_scores.cu -- a2 in its general form (coli_moe_route_scores): softmax or sigmoid scores,
// optional selection bias, groups by their best or their two best experts, masked experts.
//
// One warp per token; lane l holds the experts l * VPL .. l * VPL + VPL - 1, so that a group of
// experts is a run of lanes and all groups reduce at once in a few shuffles.  What is compared is
// an unsigned integer key that orders as the value does, 0 for an expert that cannot be chosen:
// 32 bits of the logit itself without a bias (the score grows with it, no rounding takes part in
// the choice), 64 bits of the double c = s + bias with one.  A warp's largest key is then one
// redux.sync (three with 64 bits: high word, low word, lowest id) instead of five rounds of
// shuffles and comparisons.
// Bound: arithmetic, not the E * 4 bytes per token (see the launcher's figures).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "internal.h"

namespace coli {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int ROUTE_WARPS = 4;

// Order-preserving keys; every value but NaN and -inf maps above 0 (and those two are given 0).
__device__ __forceinline__ uint32_t key32(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are one value
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key64(double v) {
    if (!(v > -static_cast<double>(INFINITY))) return 0ull;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double unkey64(uint64_t k) {
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k & ~(1ull << 63) : ~k));
}
__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ double sigmoid(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(FULL, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = static_cast<uint32_t>(v >> 32);
    const uint32_t mh = __reduce_max_sync(FULL, hi);
    const uint32_t ml = __reduce_max_sync(FULL, hi == mh ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(mh) << 32) | ml;
}

struct RouteArgs {
    const void *logits;
    size_t ld;
    const float *bias;
    int T, E, K, G, TG;
    int softmax, group_max, renorm;
    float scaling;
    int32_t *ids;
    float *w;
};

// What a group is ranked by: its largest key, or the sum of its two largest scores.
// (best, second) of one lane merged with another's.
template <typename Key>
__device__ __forceinline__ void merge2(Key &a1, Key &a2, Key b1, Key b2) {
    const Key lo = a1 < b1 ? a1 : b1;
    a1 = a1 < b1 ? b1 : a1;
    a2 = a2 < b2 ? b2 : a2;
    a2 = a2 < lo ? lo : a2;
}
template <typename Key>
__device__ __forceinline__ Key shfl_xor(Key v, int o) { return __shfl_xor_sync(FULL, v, o); }
template <>
__device__ __forceinline__ uint64_t shfl_xor<uint64_t>(uint64_t v, int o) {
    return __shfl_xor_sync(FULL, static_cast<unsigned long long>(v), o);
}

template <int VPL, bool BIAS, typename In>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_scores_kernel(const RouteArgs a) {
    using Key = typename std::conditional<BIAS, uint64_t, uint32_t>::type;
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const In *row = static_cast<const In *>(a.logits) + static_cast<size_t>(t) * a.ld;
    const int e0 = lane * VPL;
    float l[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        float x = -INFINITY;
        if (e0 + v < a.E) {
            if (sizeof(In) == 4) x = __ldg(reinterpret_cast<const float *>(row) + e0 + v);
            else x = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(row) + e0 + v)) << 16);
        }
        l[v] = x > -INFINITY ? x : -INFINITY;  // NaN masks as -inf does
    }
    // softmax: the row's maximum and float32 or double sum (double where biased scores are compared)
    float top = -INFINITY;
    double sum = 1.0;
    if (a.softmax) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) top = fmaxf(top, l[v]);
        top = unkey32(warp_max(key32(top)));  // NaN when every expert is masked: nothing is read from it then
    }
    // exp(l - top); the largest logit (+inf too) gives 1
    auto expd = [&](float x) { return x == top ? 1.0 : exp(static_cast<double>(x) - static_cast<double>(top)); };
    auto expf_ = [&](float x) { return x == top ? 1.0f : expf(x - top); };
    Key key[VPL];
    if (BIAS) {
        double s[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) s[v] = l[v] == -INFINITY ? 0.0 : (a.softmax ? expd(l[v]) : sigmoid(l[v]));
        if (a.softmax) {
            sum = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v) sum += s[v];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
            const double inv = 1.0 / sum;
#pragma unroll
            for (int v = 0; v < VPL; ++v) s[v] *= inv;
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            key[v] = e0 + v < a.E && l[v] > -INFINITY ? static_cast<Key>(key64(s[v] + static_cast<double>(__ldg(a.bias + e0 + v)))) : Key(0);
    } else {
        if (a.softmax && !a.renorm) {
            float fs = 0.f;
#pragma unroll
            for (int v = 0; v < VPL; ++v) fs += l[v] == -INFINITY ? 0.f : expf_(l[v]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) fs += __shfl_xor_sync(FULL, fs, o);
            sum = static_cast<double>(fs);
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = static_cast<Key>(key32(l[v]));
    }
    // ---- groups: drop the keys of those that are not kept
    if (a.TG < a.G) {
        const int gs = a.E / a.G;
        // what a group with the keys b1 >= b2 is ranked by, as a 64-bit key (0: nothing to choose)
        auto rank_of = [&](Key b1, Key b2) -> uint64_t {
            if (b1 == 0) return 0ull;
            if (a.group_max) return static_cast<uint64_t>(b1);
            double r;
            if (BIAS) {
                r = unkey64(b1) + (b2 ? unkey64(b2) : 0.0);
            } else {
                const float f1 = unkey32(static_cast<uint32_t>(b1));
                r = a.softmax ? expd(f1) : sigmoid(f1);
                if (b2) {
                    const float f2 = unkey32(static_cast<uint32_t>(b2));
                    r += a.softmax ? expd(f2) : sigmoid(f2);
                }
            }
            return key64(r);
        };
        uint32_t kept = 0u;
        uint64_t mine = 0ull;  // rank of group `lane`
        const int seg = gs / VPL;  // lanes of a group
        if (gs % VPL == 0 && (seg & (seg - 1)) == 0) {
            Key b1 = 0, b2 = 0;
#pragma unroll
            for (int v = 0; v < VPL; ++v) merge2<Key>(b1, b2, key[v], Key(0));
            for (int o = 1; o < seg; o <<= 1) {
                const Key c1 = shfl_xor<Key>(b1, o), c2 = shfl_xor<Key>(b2, o);
                merge2<Key>(b1, b2, c1, c2);
            }
            const uint64_t r = rank_of(b1, b2);
            const uint64_t got = __shfl_sync(FULL, static_cast<unsigned long long>(r), lane < a.G ? lane * seg : 0);
            if (lane < a.G) mine = got;
        } else {
            for (int g = 0; g < a.G; ++g) {
                Key b1 = 0, b2 = 0;
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    if ((e0 + v) / gs == g) merge2<Key>(b1, b2, key[v], Key(0));
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const Key c1 = shfl_xor<Key>(b1, o), c2 = shfl_xor<Key>(b2, o);
                    merge2<Key>(b1, b2, c1, c2);
                }
                const uint64_t r = rank_of(b1, b2);
                if (lane == g) mine = r;
            }
        }
        // a group's place: how many groups come before it
        int before = 0;
        for (int g = 0; g < a.G; ++g) {
            const uint64_t o = __shfl_sync(FULL, static_cast<unsigned long long>(mine), g);
            before += o > mine || (o == mine && g < lane);
        }
        kept = __ballot_sync(FULL, lane < a.G && before < a.TG);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (e0 + v < a.E && !((kept >> ((e0 + v) / gs)) & 1u)) key[v] = 0;
    }
    // ---- K picks; lane k keeps the expert of slot k
    int my_id = -1;
    uint32_t taken = 0u;  // of this lane's experts (VPL <= 32)
    int n = 0;
    for (; n < a.K; ++n) {
        Key best = 0;
        int at = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (key[v] > best) { best = key[v]; at = v; }
        const Key m = warp_max(best);
        if (m == 0) break;
        const int id = __reduce_min_sync(FULL, best == m ? static_cast<unsigned>(e0 + at) : 0xffffffffu);
        if (id / VPL == lane) {
            taken |= 1u << (id % VPL);
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (v == id % VPL) key[v] = 0;
        }
        if (lane == n) my_id = id;
    }
    const int chosen = n;
    for (; n < a.K; ++n) {  // too few: the lowest ids that are left
        unsigned low = 0xffffffffu;
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v)
            if (e0 + v < a.E && !((taken >> v) & 1u)) low = e0 + v;
        const int id = __reduce_min_sync(FULL, low);
        if (id / VPL == lane) taken |= 1u << (id % VPL);
        if (lane == n) my_id = id;
    }
    // ---- weights of the chosen, one per lane.  Renormalised softmax: relative to the largest
    // chosen logit, so that a row whose maximum was masked by its group keeps its digits;
    // sigmoid: in double, so that a row of very negative logits does.
    float x = -INFINITY;
    if (lane < chosen) {
        if (sizeof(In) == 4) x = __ldg(reinterpret_cast<const float *>(row) + my_id);
        else x = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(row) + my_id)) << 16);
    }
    float wt = 0.f;
    if (a.softmax) {
        if (a.renorm) top = unkey32(__reduce_max_sync(FULL, key32(x)));
        float s = lane < chosen ? expf_(x) : 0.f;
        if (a.renorm) {
            float d = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
            wt = d > 0.f ? s / d : 0.f;
        } else {
            wt = lane < chosen ? static_cast<float>(static_cast<double>(s) / sum) : 0.f;
        }
    } else {
        double s = lane < chosen ? sigmoid(x) : 0.0;
        if (a.renorm) {
            double d = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
            s = d > 0.0 ? s / d : 0.0;
        }
        wt = static_cast<float>(s);
    }
    if (lane < a.K) {
        a.ids[static_cast<size_t>(t) * a.K + lane] = my_id;
        a.w[static_cast<size_t>(t) * a.K + lane] = wt * a.scaling;
    }
}

template <int VPL>
void launch_vpl(const RouteArgs &a, int act, cudaStream_t st) {
    const int grid = (a.T + ROUTE_WARPS - 1) / ROUTE_WARPS;
    if (a.bias) {
        if (act == COLI_ACT_F32) route_scores_kernel<VPL, true, float><<<grid, ROUTE_WARPS * 32, 0, st>>>(a);
        else route_scores_kernel<VPL, true, uint16_t><<<grid, ROUTE_WARPS * 32, 0, st>>>(a);
    } else {
        if (act == COLI_ACT_F32) route_scores_kernel<VPL, false, float><<<grid, ROUTE_WARPS * 32, 0, st>>>(a);
        else route_scores_kernel<VPL, false, uint16_t><<<grid, ROUTE_WARPS * 32, 0, st>>>(a);
    }
}

}  // namespace

cudaError_t launch_route_scores(const coli_moe_router &r, const void *logits, size_t ld, const float *bias, int T,
                                int32_t *ids, float *w, cudaStream_t st) {
    RouteArgs a;
    a.logits = logits;
    a.ld = ld;
    a.bias = bias;
    a.T = T;
    a.E = r.n_experts;
    a.K = r.top_k;
    a.G = r.n_group;
    a.TG = r.topk_group;
    a.softmax = r.score == COLI_SCORE_SOFTMAX;
    a.group_max = r.group_score == COLI_GROUP_MAX;
    a.renorm = r.renorm;
    a.scaling = static_cast<float>(r.scaling);
    a.ids = ids;
    a.w = w;
    const int vpl = (a.E + 31) / 32;
    if (vpl <= 1) launch_vpl<1>(a, r.logits, st);
    else if (vpl <= 2) launch_vpl<2>(a, r.logits, st);
    else if (vpl <= 4) launch_vpl<4>(a, r.logits, st);
    else if (vpl <= 8) launch_vpl<8>(a, r.logits, st);
    else if (vpl <= 16) launch_vpl<16>(a, r.logits, st);
    else launch_vpl<32>(a, r.logits, st);
    return cudaGetLastError();
}

}  // namespace coli
