// route_scores.cu -- a2 in its general form (coli_moe_route_scores): softmax or sigmoid scores,
// optional selection bias, groups by their best or their two best experts, masked experts.
//
// One warp per token; lane l holds the experts l * VPL .. l * VPL + VPL - 1, so that a group of
// experts is a run of lanes and all groups reduce at once in a few shuffles.  What is compared is
// an unsigned integer key that orders as the value does, 0 for an expert that cannot be chosen:
// 32 bits of the logit itself without a bias (the score grows with it, no rounding takes part in
// the choice), 64 bits of the double c = s + bias with one.  A warp's largest key is then one
// redux.sync (two with 64 bits, high word and low word) and a ballot for the lane it is in, instead
// of five rounds of shuffles and comparisons.  Most tokens are chosen in float32 with the expert's
// place in the key's last bits (choose_fast); where its errors could matter, exactly.
// Bound: instructions, not the E * 4 bytes per token.  16,384 tokens of 256 float32 logits with a
// bias, 4 of 8 groups kept: 18.8 us, 780 instructions per token and warp, issued in 76% of the cycles
// (11 us if they were in all); the logits alone would take 2.6 us.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "internal.h"
#include "pdl.h"
#include "route_scores.h"

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

__device__ __forceinline__ float load_one(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_one(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16); }
template <int N>
__device__ __forceinline__ void load_run(const float *p, float (&d)[N]) {
#pragma unroll
    for (int i = 0; i + 4 <= N; i += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(p + i));
        d[i] = f.x; d[i + 1] = f.y; d[i + 2] = f.z; d[i + 3] = f.w;
    }
}
template <int N>
__device__ __forceinline__ void load_run(const uint16_t *p, float (&d)[N]) {
#pragma unroll
    for (int i = 0; i + 8 <= N; i += 8) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p + i));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            d[i + 2 * j] = __uint_as_float(w[j] << 16);
            d[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

struct RouteArgs {
    const void *logits;
    size_t ld;
    const float *bias;
    int T, E, K, G, TG;
    int softmax, group_max, renorm;
    int fast;  // the groups are whole runs of lanes, 1 << seg_shift each
    int gs, seg_shift;
    float inv_gs;
    int vec;   // rows (and the bias) allow 16-byte loads of a lane's experts
    float scaling;
    int32_t *ids;
    float *w;
};

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

// exp(l - top); the largest logit (+inf too) gives 1
__device__ __forceinline__ double exp_above(float l, float top) { return l == top ? 1.0 : exp(static_cast<double>(l) - static_cast<double>(top)); }
__device__ __forceinline__ float expf_above(float l, float top) { return l == top ? 1.0f : expf(l - top); }

// A token's choice, compared exactly (64-bit keys of double scores with a bias, 32-bit keys of the logits
// without).  Lane k gets the expert of slot k in my_id; `chosen` of the K were there to choose.
template <int VPL, bool BIAS>
__device__ __forceinline__ void choose_exact(const RouteArgs &a, const float (&l)[VPL], int e0, int lane, int &my_id, int &chosen, float &top, double &sum) {
    using Key = typename std::conditional<BIAS, uint64_t, uint32_t>::type;
    top = -INFINITY;
    sum = 1.0;
    // softmax: the row's maximum and float32 or double sum (double where biased scores are compared)
    if (a.softmax) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) top = fmaxf(top, l[v]);
        top = unkey32(warp_max(key32(top)));  // NaN when every expert is masked: nothing is read from it then
    }
    Key key[VPL];
    if (BIAS) {
        double s[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) s[v] = l[v] == -INFINITY ? 0.0 : (a.softmax ? exp_above(l[v], top) : sigmoid(l[v]));
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
            for (int v = 0; v < VPL; ++v) fs += l[v] == -INFINITY ? 0.f : expf_above(l[v], top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) fs += __shfl_xor_sync(FULL, fs, o);
            sum = static_cast<double>(fs);
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = static_cast<Key>(key32(l[v]));
    }
    // ---- groups: drop the keys of those that are not kept
    if (a.TG < a.G) {
        // the group of expert e < 1024: e + 1/2 is further than a rounding from a multiple of gs
        auto group_of = [&](int e) { return static_cast<int>((static_cast<float>(e) + 0.5f) * a.inv_gs); };
        // what a group with the keys b1 >= b2 is ranked by, as a 64-bit key (0: nothing to choose)
        auto rank_of = [&](Key b1, Key b2) -> uint64_t {
            if (b1 == 0) return 0ull;
            if (a.group_max) return static_cast<uint64_t>(b1);
            double r;
            if (BIAS) {
                r = unkey64(b1) + (b2 ? unkey64(b2) : 0.0);
            } else {
                const float f1 = unkey32(static_cast<uint32_t>(b1));
                r = a.softmax ? exp_above(f1, top) : sigmoid(f1);
                if (b2) {
                    const float f2 = unkey32(static_cast<uint32_t>(b2));
                    r += a.softmax ? exp_above(f2, top) : sigmoid(f2);
                }
            }
            return key64(r);
        };
        uint32_t kept = 0u;
        uint64_t mine = 0ull;  // rank of group `lane`
        if (a.fast) {
            const int seg = 1 << a.seg_shift;  // lanes of a group
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
                    if (group_of(e0 + v) == g) merge2<Key>(b1, b2, key[v], Key(0));
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
            if (e0 + v < a.E && !((kept >> group_of(e0 + v)) & 1u)) key[v] = 0;
    }
    // ---- K picks; lane k keeps the expert of slot k
    my_id = -1;
    uint32_t taken = 0u;  // of this lane's experts (VPL <= 32)
    int n = 0;
    for (; n < a.K; ++n) {
        Key best = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) best = key[v] > best ? key[v] : best;
        const Key m = warp_max(best);
        if (m == 0) break;
        // lanes hold runs of experts: the lowest lane, and its lowest place, has the lowest id
        const int owner = __ffs(__ballot_sync(FULL, best == m)) - 1;
        int at = 0;
        if (lane == owner) {
#pragma unroll
            for (int v = VPL - 1; v >= 0; --v)
                if (key[v] == m) at = v;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (v == at) key[v] = 0;
            taken |= 1u << at;
        }
        const int id = __shfl_sync(FULL, e0 + at, owner);
        if (lane == n) my_id = id;
    }
    chosen = n;
    for (; n < a.K; ++n) {  // too few: the lowest ids that are left
        unsigned low = 0xffffffffu;
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v)
            if (e0 + v < a.E && !((taken >> v) & 1u)) low = e0 + v;
        const int id = __reduce_min_sync(FULL, low);
        if (id / VPL == lane) taken |= 1u << (id % VPL);  // (VPL is a power of two)
        if (lane == n) my_id = id;
    }
}

// 1 / (1 + 2^(-l log2 e)) by the approximate instructions: ex2 within 2^-22, rcp within 2^-23 of their results.
__device__ __forceinline__ float sigmoid_fast(float l) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// Descending order of a lane's keys (Batcher's odd-even merge sort; VPL a power of two).
template <int VPL>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[VPL]) {
#pragma unroll
    for (int p = 1; p < VPL; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < VPL; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < VPL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(k[i + j], k[i + j + q]), lo = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                        k[i + j + q] = lo;
                    }
}

// The same choice in float32 where its errors cannot change it: false where two values that are compared
// lie too close (with random float32 logits about one token in a hundred), or fewer than K can be chosen.
// The place of an expert among its lane's is kept in the last bits of its key, VPL - 1 - place, so a
// lane's keys can be sorted; a pick is then one redux.sync of the first keys and a shift in one lane.
// Errors in units of 2^-24.  With a bias: sigmoid, (4 + 1.5 |l|) of exp(-l), of which s takes s (1 - s), the
// sum's 1 and the reciprocal's 2 make 5; softmax, expf's 4, its argument's rounding 1, a sum of VPL
// terms per lane and 5 rounds VPL + 5 of s; the sum with the bias 1 of c.  The place costs 2 VPL units of |c|, or
// of |l| without a bias, and VPL 2^-149 where float32's last place is no smaller (equal logits of 0 differ by
// their places alone); of bf16 logits it takes bits that are zero, and equal logits come in the order of
// their ids.  Groups by two scores without a bias: the scores' errors alone.
template <int VPL, bool BIAS, typename In>
__device__ __forceinline__ bool choose_fast(const RouteArgs &a, const float (&l)[VPL], int e0, int lane, int &my_id, float &top, double &sum) {
    constexpr bool EXACT = !BIAS && sizeof(In) == 2;
    constexpr float UNIT = 5.9604644775390625e-8f;  // 2^-24
    const bool groups = a.TG < a.G, top2 = groups && !a.group_max;
    float c[VPL], smax = 1.f;
    if (a.softmax) {
        top = l[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) top = fmaxf(top, l[v]);
        top = unkey32(warp_max(key32(top)));
        if (!(fabsf(top) < INFINITY)) return false;  // +inf, or every expert masked
    }
    if (a.softmax && (BIAS || !a.renorm || top2)) {
        float fs = 0.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            c[v] = expf(l[v] - top);
            fs += c[v];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) fs += __shfl_xor_sync(FULL, fs, o);
        sum = static_cast<double>(fs);
        smax = 1.0f / fs;
    } else if (!a.softmax && (BIAS || top2)) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) c[v] = sigmoid_fast(fmaxf(l[v], -60.0f));
    }
    if (BIAS) {
        float bias[VPL];
        if (VPL >= 4 && a.vec) {
            load_run<VPL>(a.bias + e0, bias);
        } else {
#pragma unroll
            for (int v = 0; v < VPL; ++v) bias[v] = __ldg(a.bias + min(e0 + v, a.E - 1));
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float f = fmaxf((a.softmax ? c[v] * smax : c[v]) + bias[v], -INFINITY);  // NaN: not to be chosen
            c[v] = l[v] > -INFINITY ? f : -INFINITY;  // (l is -inf behind the last expert)
        }
    }
    auto value = [&](int v) { return BIAS ? c[v] : l[v]; };
    // how far a float32 value of magnitude m may be off; the place alone, VPL units of the last place, which are
    // 2^-149 each for logits below 2^-125 (scores with a bias are off by more than that already)
    auto off = [&](float m) { return BIAS ? UNIT * ((VPL + 16) * (smax + m) + 2 * VPL * m) : fmaxf(UNIT * (2 * VPL * m), VPL * 1.40129846e-45f); };
    bool mine = true;  // this lane's experts are of a group that is kept
    if (groups) {
        // a group's lanes: 1 << seg_shift of them (the launcher's rule)
        float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float f = BIAS || !top2 ? value(v) : (l[v] > -INFINITY ? c[v] : -INFINITY);
            b2 = fmaxf(b2, fminf(b1, f));
            b1 = fmaxf(b1, f);
        }
        for (int o = 1; o < (1 << a.seg_shift); o <<= 1) {
            const float c1 = __shfl_xor_sync(FULL, b1, o), c2 = __shfl_xor_sync(FULL, b2, o);
            b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
            b1 = fmaxf(b1, c1);
        }
        const int g = lane >> a.seg_shift;
        const float r = g >= a.G ? -INFINITY : (top2 && b2 > -INFINITY ? b1 + b2 : b1);
        // how close two ranks may be: with a bias by the largest magnitudes that were added; sums of scores
        // without one by the scores' errors (softmax numerators: relative to the largest, 1)
        float gtol = 0.f;
        if (BIAS) {
            const float mag = fabsf(b1) + (top2 ? fabsf(b2) : 0.f);
            gtol = 4.0f * off(__uint_as_float(__reduce_max_sync(FULL, mag < INFINITY ? __float_as_uint(mag) : 0u)));
        } else if (top2) {
            gtol = 4.0f * UNIT * (VPL + 16);
        }
        int above = 0, near = 0;  // groups certainly before this one; groups too close to tell (and itself)
        if (BIAS || top2) {
#pragma unroll 4
            for (int o = 0; o < a.G; ++o) {
                const float d = __shfl_sync(FULL, r, o << a.seg_shift) - r;
                above += d > gtol;
                near += fabsf(d) <= gtol;
            }
            near -= r > -INFINITY;
        } else {  // the logits themselves: ties go to the lower group
#pragma unroll 4
            for (int o = 0; o < a.G; ++o) {
                const float q = __shfl_sync(FULL, r, o << a.seg_shift);
                above += q > r || (q == r && o < g);
            }
        }
        mine = above + near < a.TG;
        // a close group that could push this one across the border, or a kept group without an expert
        // to choose: leave the token to the exact choice
        if (__any_sync(FULL, g < a.G && ((near > 0 && above < a.TG && !mine) || (mine && r == -INFINITY)))) return false;
    }
    // (-inf has a key too, below every other's: NONE and up are values that can be chosen)
    constexpr uint32_t NONE = 0x00800000u;
    uint32_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const uint32_t b = __float_as_uint(value(v) + 0.0f);  // -0 and +0 are one value
        const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
        key[v] = (k & ~static_cast<uint32_t>(VPL - 1)) | static_cast<uint32_t>(VPL - 1 - v);
    }
    sort_keys<VPL>(key);
    if (!mine) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = 0u;
    }
    uint32_t got = 0u;  // lane n: key of pick n
    int from = 0;       // and the lane it came from
    for (int n = 0; n < a.K; ++n) {
        const uint32_t m = __reduce_max_sync(FULL, key[0]);
        // (equal logits: the lowest lane has the lowest id, whatever the place in the key says)
        constexpr uint32_t SAME = EXACT ? ~static_cast<uint32_t>(VPL - 1) : FULL;
        const int owner = __ffs(__ballot_sync(FULL, (key[0] & SAME) == (m & SAME))) - 1;
        const uint32_t k = EXACT ? __shfl_sync(FULL, key[0], owner) : m;
        if (lane == n) {
            got = k;
            from = owner;
        }
        if (lane == owner) {
#pragma unroll
            for (int v = 0; v + 1 < VPL; ++v) key[v] = key[v + 1];
            key[VPL - 1] = 0u;
        }
    }
    my_id = from * VPL + (VPL - 1 - static_cast<int>(got & (VPL - 1)));
    if (EXACT) return !__any_sync(FULL, lane < a.K && got < NONE);
    // every pick has to be clear of the next one, and the last of the best that was left
    const uint32_t left = __reduce_max_sync(FULL, key[0]);
    uint32_t next = __shfl_down_sync(FULL, got, 1);
    if (lane == a.K - 1) next = left;
    const float x = unkey32(got), y = unkey32(next);
    const bool clear = lane >= a.K || (got >= NONE && (next < NONE || x - y > 2.0f * off(fmaxf(fabsf(x), fabsf(y)))));
    return __all_sync(FULL, clear);
}

template <int VPL, bool BIAS, typename In>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_scores_kernel(const RouteArgs a) {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const In *row = static_cast<const In *>(a.logits) + static_cast<size_t>(t) * a.ld;
    const int e0 = lane * VPL;
    float l[VPL];
    if (VPL * sizeof(In) >= 16 && a.vec) {  // 16-byte loads: E = 32 VPL and rows are aligned
        load_run<VPL>(row + e0, l);
#pragma unroll
        for (int v = 0; v < VPL; ++v) l[v] = fmaxf(l[v], -INFINITY);  // NaN masks as -inf does
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float x = load_one(row + min(e0 + v, a.E - 1));
            l[v] = e0 + v < a.E ? fmaxf(x, -INFINITY) : -INFINITY;
        }
    }
    int my_id, chosen = a.K;
    float top;
    double sum;
    if (!a.fast || !choose_fast<VPL, BIAS, In>(a, l, e0, lane, my_id, top, sum))
        choose_exact<VPL, BIAS>(a, l, e0, lane, my_id, chosen, top, sum);
    // ---- weights of the chosen, one per lane.  Renormalised softmax: relative to the largest
    // chosen logit, so that a row whose maximum was masked by its group keeps its digits; sigmoid of
    // very negative logits alone: in double, for the same reason.
    float x = -INFINITY;
    if (lane < chosen) {
        if (sizeof(In) == 4) x = __ldg(reinterpret_cast<const float *>(row) + my_id);
        else x = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(row) + my_id)) << 16);
    }
    float wt = 0.f;
    if (a.softmax) {
        if (a.renorm) top = unkey32(__reduce_max_sync(FULL, key32(x)));
        float s = lane < chosen ? expf_above(x, top) : 0.f;
        if (a.renorm) {
            float d = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
            wt = d > 0.f ? s / d : 0.f;
        } else {
            wt = lane < chosen ? static_cast<float>(static_cast<double>(s) / sum) : 0.f;
        }
    } else if (a.renorm && !__any_sync(FULL, x > -40.0f)) {
        double s = lane < chosen ? sigmoid(x) : 0.0, d = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
        wt = d > 0.0 ? static_cast<float>(s / d) : 0.f;
    } else {
        wt = lane < chosen ? 1.0f / (1.0f + expf(-x)) : 0.f;
        if (a.renorm) {
            float d = wt;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
            wt = wt / d;
        }
    }
    if (lane < a.K) {
        a.ids[static_cast<size_t>(t) * a.K + lane] = my_id;
        a.w[static_cast<size_t>(t) * a.K + lane] = wt * a.scaling;
    }
}

template <int VPL>
cudaError_t launch_vpl(RouteArgs a, int act, cudaStream_t st) {
    const int gs = a.E / a.G, seg = gs / VPL;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | (a.bias ? reinterpret_cast<uintptr_t>(a.bias) : 0) | (a.ld * (act == COLI_ACT_F32 ? 4 : 2));
    a.vec = a.E == 32 * VPL && at % 16 == 0;
    a.fast = a.TG == a.G || (gs % VPL == 0 && (seg & (seg - 1)) == 0);
    a.gs = gs;
    a.inv_gs = 1.0f / static_cast<float>(gs);
    a.seg_shift = 0;
    while ((2 << a.seg_shift) <= seg) ++a.seg_shift;
    const int grid = (a.T + ROUTE_WARPS - 1) / ROUTE_WARPS;
    auto go = [&](auto kernel) { return launch_early(kernel, dim3(grid), ROUTE_WARPS * 32, 0, st, 1, a); };
    if (a.bias) return act == COLI_ACT_F32 ? go(route_scores_kernel<VPL, true, float>) : go(route_scores_kernel<VPL, true, uint16_t>);
    return act == COLI_ACT_F32 ? go(route_scores_kernel<VPL, false, float>) : go(route_scores_kernel<VPL, false, uint16_t>);
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
    if (vpl <= 1) return launch_vpl<1>(a, r.logits, st);
    if (vpl <= 2) return launch_vpl<2>(a, r.logits, st);
    if (vpl <= 4) return launch_vpl<4>(a, r.logits, st);
    if (vpl <= 8) return launch_vpl<8>(a, r.logits, st);
    if (vpl <= 16) return launch_vpl<16>(a, r.logits, st);
    return launch_vpl<32>(a, r.logits, st);
}

}  // namespace coli
