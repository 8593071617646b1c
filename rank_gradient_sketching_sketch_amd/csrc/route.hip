// Routing: the experts that every token takes, their weights, and the
// weights' gradient carried back to the logits. What stands before the sort of
// experts.hip, and behind combine's gradient.
//
// For a token's logits x and the experts' biases b (balance; not part of the
// weights):
//   s_e = softmax(x)_e or 1 / (1 + exp(-x_e)),   key_e = s_e + b_e,
//   groups of E / G neighbouring experts: only the topk_groups whose best one
//   or two keys sum highest are left,
//   id_j = the j-th highest key left (ties: the lower index),
//   w_j  = c s_(id_j), divided by the sum of the chosen s where renormalised.
// An expert whose key is -inf or NaN is never chosen; a choice that finds
// none is -1 with weight 0, which the sort drops. A softmax with a logit of
// +inf has no values: there the logits are the keys and the weights NaN.
//
// Choices are whole numbers that must not hang on rounding: they are those of
// keys formed and compared in fp64. Where no bias and no sum of two keys
// enters, the logits themselves are compared, which sort like their scores.
// Otherwise fp32 keys are tried first, with what they may be off by: only
// where two keys that had to be told apart are nearer than that are fp64 ones
// formed, of the few experts in question (sigmoid) or of all (softmax, and
// groups in doubt). Weights are fp32, as ratios of exponentials of differences
// that cannot overflow or all vanish.
//
// A wave per token. Up to some thousand tokens the time is one wave's chain of
// choices, not memory (4 MB of logits are 1 us). 4096 tokens to 8 of 256
// experts, four of eight groups: 9.2 us (a token or two in doubt, at the end of
// it all, are 1.7 of them), 10.6 with fp64 keys for all. Above that it is the
// instructions that a whole wave spends on every choice of one token: 16384
// tokens 23.2 us and 29.1, 65536 tokens 76 and 96, where the logits are 3.5 and
// 14 us.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace logra {

constexpr int kRouteThreads = 256, kRouteTokens = kRouteThreads / 64;

template <int BF16>
__device__ __forceinline__ float route_logit(const void *x, int64_t at) {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(x)[at]) << 16);
    return static_cast<const float *>(x)[at];
}

// A step of a reduction towards lane 63: lane L gets lane L - n's value (rows
// of 16 lanes), then the rows' last lanes are carried on. Lanes without a
// source keep `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t old, uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(old), static_cast<int>(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double old, double v) {
    const uint64_t o = __builtin_bit_cast(uint64_t, old), w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_u32<CTRL, ROWS>(static_cast<uint32_t>(o), static_cast<uint32_t>(w));
    const uint32_t hi = dpp_u32<CTRL, ROWS>(static_cast<uint32_t>(o >> 32), static_cast<uint32_t>(w >> 32));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f32(float old, float v) {
    return __uint_as_float(dpp_u32<CTRL, ROWS>(__float_as_uint(old), __float_as_uint(v)));
}

__device__ __forceinline__ uint32_t lane_u32(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ float lane_f32(float v, int lane) { return __uint_as_float(lane_u32(__float_as_uint(v), lane)); }
__device__ __forceinline__ double lane_f64(double v, int lane) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = lane_u32(static_cast<uint32_t>(w), lane), hi = lane_u32(static_cast<uint32_t>(w >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Reductions over the wave, the same in every lane.
__device__ __forceinline__ float wave_max_f32(float v) {
    v = fmaxf(v, dpp_f32<0x111, 0xF>(v, v));
    v = fmaxf(v, dpp_f32<0x112, 0xF>(v, v));
    v = fmaxf(v, dpp_f32<0x114, 0xF>(v, v));
    v = fmaxf(v, dpp_f32<0x118, 0xF>(v, v));
    v = fmaxf(v, dpp_f32<0x142, 0xA>(v, v));
    v = fmaxf(v, dpp_f32<0x143, 0xC>(v, v));
    return lane_f32(v, 63);
}
__device__ __forceinline__ float wave_sum_f32(float v) {
    v += dpp_f32<0x111, 0xF>(0.f, v);
    v += dpp_f32<0x112, 0xF>(0.f, v);
    v += dpp_f32<0x114, 0xF>(0.f, v);
    v += dpp_f32<0x118, 0xF>(0.f, v);
    v += dpp_f32<0x142, 0xA>(0.f, v);
    v += dpp_f32<0x143, 0xC>(0.f, v);
    return lane_f32(v, 63);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_f64<0x111, 0xF>(0.0, v);
    v += dpp_f64<0x112, 0xF>(0.0, v);
    v += dpp_f64<0x114, 0xF>(0.0, v);
    v += dpp_f64<0x118, 0xF>(0.0, v);
    v += dpp_f64<0x142, 0xA>(0.0, v);
    v += dpp_f64<0x143, 0xC>(0.0, v);
    return lane_f64(v, 63);
}

// The two kinds of keys. fp32 values as whole numbers that sort like them (0:
// not to be chosen; both zeros are one key), and fp64 keys (-inf: not to be
// chosen).
struct FloatKey {
    using Key = uint32_t;
    static __device__ __forceinline__ Key none() { return 0u; }
    static __device__ __forceinline__ Key of(float x) {
        const uint32_t b = __float_as_uint(x + 0.f);
        return x > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
    }
    static __device__ __forceinline__ float value(Key k) {
        return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
    }
    static __device__ __forceinline__ Key add(Key a, Key b) { return of(value(a) + value(b)); }
    static __device__ __forceinline__ Key larger(Key a, Key b) { return a > b ? a : b; }
    static __device__ __forceinline__ Key smaller(Key a, Key b) { return a > b ? b : a; }
    static __device__ __forceinline__ Key lane(Key v, int l) { return lane_u32(v, l); }
    static __device__ __forceinline__ Key other(Key v, int o) {
        return static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o));
    }
    // rows of 16 lanes by DPP (0 where a lane has no source), the four rows by scalars
    static __device__ __forceinline__ Key over_wave(Key v) {
        v = larger(v, dpp_u32<0x111, 0xF>(0u, v));
        v = larger(v, dpp_u32<0x112, 0xF>(0u, v));
        v = larger(v, dpp_u32<0x114, 0xF>(0u, v));
        v = larger(v, dpp_u32<0x118, 0xF>(0u, v));
        return larger(larger(lane_u32(v, 15), lane_u32(v, 31)), larger(lane_u32(v, 47), lane_u32(v, 63)));
    }
};
struct ScoreKey {
    using Key = double;
    static __device__ __forceinline__ Key none() { return -INFINITY; }
    static __device__ __forceinline__ Key add(Key a, Key b) { return a + b; }
    static __device__ __forceinline__ Key larger(Key a, Key b) { return fmax(a, b); }
    static __device__ __forceinline__ Key smaller(Key a, Key b) { return fmin(a, b); }
    static __device__ __forceinline__ Key lane(Key v, int l) { return lane_f64(v, l); }
    static __device__ __forceinline__ Key other(Key v, int o) { return __shfl_xor(v, o); }
    static __device__ __forceinline__ Key over_wave(Key v) {
        v = larger(v, dpp_f64<0x111, 0xF>(v, v));
        v = larger(v, dpp_f64<0x112, 0xF>(v, v));
        v = larger(v, dpp_f64<0x114, 0xF>(v, v));
        v = larger(v, dpp_f64<0x118, 0xF>(v, v));
        v = larger(v, dpp_f64<0x142, 0xA>(v, v));
        v = larger(v, dpp_f64<0x143, 0xC>(v, v));
        return lane_f64(v, 63);
    }
};

// exp(min(x, 0) - shift) / (1 + exp(-|x|)): the sigmoid of x times exp(-shift).
__device__ __forceinline__ float sigmoid_shifted(float x, float shift) {
    return expf(fminf(x, 0.f) - shift) / (1.f + expf(-fabsf(x)));
}

struct RouteArgs {
    const void *logits;
    int64_t ld, T;
    const float *bias;
    int E, K, sigmoid, groups, kept, best, renorm;
    int size, span;       // experts of a group, lanes of a group
    float scale;
    int32_t *ids;
    float *weights;
};

// What fp32 keys may be off by: `part` for two scores, and 2^-24 of each key
// where the bias is added to its score: 2^-22 of the larger of two keys is twice
// that. A group's sum of two keys has the roundings of both, which are those of
// the keys' sizes, however small a sum they leave where their signs differ, and
// one of its own: two groups 2^-22 of the most that a group's two magnitudes add
// up to, taken twice again. That is the most of all groups, not of the two that
// are compared: one above the border with large keys may belong below it.
struct RouteDoubt {
    float part;
    __device__ __forceinline__ bool near(float a, float b) const {
        return !(a - b > part + 0x1p-22f * fmaxf(fabsf(a), fabsf(b)));
    }
    __device__ __forceinline__ bool near_sums(float a, float b, float size) const {
        return !(a - b > 2.f * part + 0x1p-21f * size);
    }
};

__device__ __forceinline__ double route_sigmoid(double x) { return 1.0 / (1.0 + exp(-x)); }

// Which experts the lanes' keys lead to: lane j gets choice j, or -1.
// CHECK: what could not be told. In doubt about choices, lane j has the j-th
// highest key's expert of `found`, which are all that can be among the choices.
enum RouteTold { kRouteAll, kRouteNotOrder, kRouteNothing };
template <class P, bool CHECK, int N>
__device__ __forceinline__ RouteTold route_choose(const RouteArgs &a, typename P::Key (&key)[N], int e0, RouteDoubt doubt,
                                                  int *my_id, int *found) {
    using Key = typename P::Key;
    const int lane = threadIdx.x & 63;
    *my_id = -1;
    if (a.groups > 1) {
        const int group = lane / a.span;
        Key one = P::none(), two = P::none();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            two = P::larger(two, P::smaller(one, key[i]));
            one = P::larger(one, key[i]);
        }
        for (int o = 1; o < a.span; o <<= 1) {
            const Key one2 = P::other(one, o), two2 = P::other(two, o);
            two = P::larger(P::smaller(one, one2), P::larger(two, two2));
            one = P::larger(one, one2);
        }
        const Key sum = a.best == 2 && two > P::none() ? P::add(one, two) : one;
        int better = 0;
        for (int g = 0; g < a.groups; ++g) {
            const Key s = P::lane(sum, g * a.span);
            better += s > sum || (s == sum && g < group);
        }
        const bool out = better >= a.kept;
        if constexpr (CHECK) {
            // the lowest sum that stays against the highest that does not
            const Key low = P::lane(sum, __builtin_ctzll(__ballot(better == a.kept - 1)));
            const Key high = P::lane(sum, __builtin_ctzll(__ballot(better == a.kept)));
            if (high > P::none()) {
                if (a.best == 2) {
                    // by every group's size, so by the largest
                    const float size = (one > P::none() ? fabsf(P::value(one)) : 0.f) + (two > P::none() ? fabsf(P::value(two)) : 0.f);
                    if (__ballot(doubt.near_sums(P::value(low), P::value(high), size)) != 0) return kRouteNothing;
                } else if (doubt.near(P::value(low), P::value(high))) {
                    return kRouteNothing;
                }
            }
        }
        if (out) {
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = P::none();
        }
    }
    // choice by choice: the largest of the lanes' largest, in the lowest lane
    // that holds it
    float value = -INFINITY;        // lane j: of choice j
    int id = -1;
    auto next = [&](int j, Key *most) {
        Key best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < N; ++i) {
            const bool more = key[i] > best;
            best = more ? key[i] : best;
            at = more ? i : at;
        }
        *most = P::over_wave(best);
        if (!(*most > P::none())) return false;
        const int from = __builtin_ctzll(__ballot(best == *most));
        const int e = static_cast<int>(lane_u32(static_cast<uint32_t>(e0 + at), from));
        if (lane == j) {
            id = e;
            if constexpr (CHECK) value = P::value(*most);
        }
        const int taken = lane == from ? at : -1;
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = i == taken ? P::none() : key[i];
        return true;
    };
    Key most;
    int j = 0;
    while (j < a.K && next(j, &most)) ++j;
    *my_id = id;
    if constexpr (CHECK) {
        const float before = dpp_f32<0x138, 0xF>(value, value);      // the lane before's
        bool close = __ballot(lane > 0 && lane < j && doubt.near(before, value)) != 0;
        if (j == a.K) {
            // the experts that may come before the last choice
            const float last = lane_f32(value, a.K - 1);
            while (next(j, &most) && doubt.near(last, P::value(most))) {
                close = true;
                if (++j > min(a.K + 8, 64)) return kRouteNothing;      // many alike, as where a router starts from zeros
            }
        }
        *my_id = lane < j ? id : -1;
        *found = j;
        return close ? kRouteNotOrder : kRouteAll;
    }
    return kRouteAll;
}

// The order of `found` experts, one in each of the first lanes, by keys of
// sigmoids in fp64; lane j gets choice j.
template <int BF16>
__device__ __forceinline__ int route_order(const RouteArgs &a, int64_t t, int id, int found) {
    const int lane = threadIdx.x & 63;
    double key = ScoreKey::none();
    if (lane < found) key = route_sigmoid(route_logit<BF16>(a.logits, t * a.ld + id)) + (a.bias ? static_cast<double>(a.bias[id]) : 0.0);
    int rank = 0;
    for (int i = 0; i < found; ++i) {
        const double k = lane_f64(key, i);
        rank += k > key || (k == key && static_cast<int>(lane_u32(static_cast<uint32_t>(id), i)) < id);
    }
    int out = -1;
    for (int i = 0; i < found; ++i)
        if (lane == static_cast<int>(lane_u32(static_cast<uint32_t>(rank), i)) && lane < a.K)
            out = static_cast<int>(lane_u32(static_cast<uint32_t>(id), i));
    return out;
}

// A wave per token. The lanes are dealt to the groups (span of them each, a
// power of two) and each lane holds up to N neighbouring experts of its
// group, so that lane and place in it sort like the expert's index, and what
// concerns one group stays among its lanes.
template <int N, int BF16, int SCORES>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteTokens + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const int group = lane / a.span, q0 = (lane & (a.span - 1)) * N;
    const int e0 = group * a.size + q0, have = group < a.groups ? max(0, min(N, a.size - q0)) : 0;
    float x[N];
    bool nan = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = i < have ? route_logit<BF16>(a.logits, t * a.ld + e0 + i) : -INFINITY;
        nan |= x[i] != x[i];
        top = fmaxf(top, x[i]);
    }
    const bool any_nan = __ballot(nan) != 0;
    // softmax: all logits against the largest
    float denom = 1.f;
    bool no_scores = false;      // a logit of +inf
    float score[N];
    if (!a.sigmoid && (SCORES || !a.renorm)) {
        top = wave_max_f32(top);
        denom = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            score[i] = x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
            denom += score[i];
        }
        denom = wave_sum_f32(denom);
        no_scores = top == INFINITY;
    }

    int my_id, found;
    if constexpr (SCORES) {
        float bias[N];
        uint32_t key[N];
#pragma unroll
        for (int i = 0; i < N; ++i) bias[i] = a.bias && i < have ? a.bias[e0 + i] : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = a.sigmoid ? 1.f / (1.f + expf(-x[i])) : score[i] / denom;
            key[i] = FloatKey::of(x[i] > -INFINITY ? s + bias[i] : -INFINITY);
        }
        // A sigmoid is three roundings and an exponential within 2^-23 (together
        // 2^-22; two of them 2^-21). A softmax has its exponential's argument
        // rounded (score times |d| 2^-24, at most 0.37 2^-24 of the largest
        // score), the exponential, up to N + 6 roundings of the sum (2^-18.7
        // with N = 32) and the quotient: 2^-18 of the largest score for two.
        const RouteDoubt doubt{a.sigmoid ? 0x1p-21f : 0x1p-18f / denom};
        const RouteTold told = route_choose<FloatKey, true>(a, key, e0, doubt, &my_id, &found);
        // keys are NaN where there are no scores: none was found
        if (told == kRouteNotOrder && a.sigmoid) {
            my_id = route_order<BF16>(a, t, my_id, found);
        } else if (told != kRouteAll || no_scores) {
            double wide[N], sum = 0.0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const double d = x[i];
                wide[i] = x[i] > -INFINITY ? (a.sigmoid ? route_sigmoid(d) : exp(d - static_cast<double>(top))) : 0.0;
                sum += wide[i];
            }
            if (!a.sigmoid) sum = wave_sum_f64(sum);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!a.sigmoid) wide[i] /= sum;
                const double d = x[i];
                const double k = no_scores ? (bias[i] > -INFINITY ? d : NAN) : wide[i] + static_cast<double>(bias[i]);
                wide[i] = x[i] > -INFINITY && k == k ? k : ScoreKey::none();
            }
            route_choose<ScoreKey, false>(a, wide, e0, doubt, &my_id, &found);
        }
    } else {
        uint32_t key[N];
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = FloatKey::of(x[i]);
        route_choose<FloatKey, false>(a, key, e0, RouteDoubt{0.f}, &my_id, &found);
    }

    const bool chosen = my_id >= 0;
    const float my_x = chosen ? route_logit<BF16>(a.logits, t * a.ld + my_id) : 0.f;
    float w;
    if (a.renorm) {
        const float most = wave_max_f32(chosen ? my_x : -INFINITY);
        const float p = !chosen ? 0.f : a.sigmoid ? sigmoid_shifted(my_x, fminf(most, 0.f)) : expf(my_x - most);
        w = p / wave_sum_f32(p);
    } else {
        w = a.sigmoid ? sigmoid_shifted(my_x, 0.f) : expf(my_x - top) / denom;
    }
    if (any_nan || no_scores) w = NAN;
    if (lane < a.K) {
        a.ids[t * a.K + lane] = my_id;
        a.weights[t * a.K + lane] = chosen ? a.scale * w : 0.f;
    }
}

// LDS accesses of the wave before this are done before those after it.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

struct RouteBackwardArgs {
    const void *logits;
    int64_t ld, T;
    int E, K, sigmoid, renorm;
    float scale;
    const int32_t *ids;
    const float *dw;
    void *dx;
    int64_t lddx;
};

// A wave per token: lane j holds choice j and what the gradient puts at its
// expert, q_j = dL/ds_j ds_j/dx_j; then the row is written by lanes that hold
// experts lane + 64 i. With p the chosen scores, P their sum (1 where not
// renormalised) and g_j = c dw_j:
//   sigmoid  q_j = p_j / P (1 - s_j) (g_j - sum_i p_i / P g_i)   (without the sum: not renormalised)
//   softmax  q_j = p_j / P (g_j - sum_i p_i / P g_i), or not renormalised
//            q_j = p_j g_j and every expert's gradient gets - s_e sum_i q_i.
// Two choices of one expert add up.
//
// Which choice an expert has is looked up in a row of bytes per wave: every
// choice writes its lane there and reads it back, and only where one finds
// another's lane (an expert chosen twice) are the choices gone through one by
// one. 16384 tokens, 8 of 128 experts: 6.9 us, 9.3 before the look-up and with
// loads one after the other; the rows read and written are 16.8 MB, 3.4 us at a
// copy's rate. The chosen logits are read after the ids, also where the wave has
// the whole row in registers already: a second wait for memory.
template <int N, int BF16>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteBackwardArgs a) {
    __shared__ uint8_t owner[kRouteTokens][64 * N];
    const int lane = threadIdx.x & 63;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteTokens + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const bool whole = !a.sigmoid && !a.renorm;
    // what does not hang on the ids is asked for with them (65536 tokens of 128
    // experts 21.3 -> 19.2 us)
    int id = lane < a.K ? a.ids[t * a.K + lane] : -1;
    const float dw = lane < a.K ? a.dw[t * a.K + lane] : 0.f;
    float row[N];
#pragma unroll
    for (int i = 0; i < N; ++i) row[i] = -INFINITY;
    if (whole) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 64 * i < a.E) row[i] = route_logit<BF16>(a.logits, t * a.ld + lane + 64 * i);
    }
    id = id >= 0 && id < a.E ? id : -1;
    const bool chosen = id >= 0;
    const float x = chosen ? route_logit<BF16>(a.logits, t * a.ld + id) : -INFINITY;
    const float g = chosen ? a.scale * dw : 0.f;
    float q;
    if (whole) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, row[i]);
        top = wave_max_f32(top);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            row[i] = row[i] == -INFINITY ? 0.f : expf(row[i] - top);
            sum += row[i];
        }
        sum = wave_sum_f32(sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;       // a row of -inf alone
        q = x == -INFINITY ? 0.f : expf(x - top) * inv * g;
        const float all = wave_sum_f32(q);
#pragma unroll
        for (int i = 0; i < N; ++i) row[i] = -(row[i] * inv * all);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) row[i] = 0.f;
        if (a.renorm) {
            const float most = wave_max_f32(x);
            float p = x == -INFINITY ? 0.f : a.sigmoid ? sigmoid_shifted(x, fminf(most, 0.f)) : expf(x - most);
            const float sum = wave_sum_f32(p);
            p = sum == 0.f ? 0.f : p / sum;
            q = p * (g - wave_sum_f32(p * g));
            if (a.sigmoid && chosen) q *= sigmoid_shifted(-x, 0.f);
        } else {
            q = x == -INFINITY ? 0.f : sigmoid_shifted(x, 0.f) * sigmoid_shifted(-x, 0.f) * g;
        }
    }
    uint8_t *who = owner[threadIdx.x >> 6];
#pragma unroll
    for (int i = 0; i < N; ++i) who[lane + 64 * i] = 255;
    wave_lds_order();
    if (chosen) who[id] = static_cast<uint8_t>(lane);
    wave_lds_order();
    if (__ballot(chosen && who[id] != lane) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = who[lane + 64 * i];
            const float add = __shfl(q, j & 63);
            if (j < 64) row[i] += add;
        }
    } else {
        for (int j = 0; j < a.K; ++j) {
            const int at = static_cast<int>(lane_u32(static_cast<uint32_t>(id), j));
            const float add = lane_f32(q, j);
            if (at < 0) continue;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at == lane + 64 * i) row[i] += add;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 64 * i;
        if (e >= a.E) continue;
        if (BF16)
            static_cast<uint16_t *>(a.dx)[t * a.lddx + e] = static_cast<uint16_t>(pack_bf16x2(row[i], 0.f));
        else
            static_cast<float *>(a.dx)[t * a.lddx + e] = row[i];
    }
}

// The lanes of a group: as many as divide the wave among the groups.
static int route_span(int groups) {
    int span = 64;
    while (64 / span < groups) span >>= 1;
    return span;
}

template <int N, int BF16>
static void route_n(const RouteArgs &a, bool scores, dim3 grid, hipStream_t st) {
    if (scores)
        hipLaunchKernelGGL((route_kernel<N, BF16, 1>), grid, dim3(kRouteThreads), 0, st, a);
    else
        hipLaunchKernelGGL((route_kernel<N, BF16, 0>), grid, dim3(kRouteThreads), 0, st, a);
}

hipError_t launch_route(const RouteCall &c, hipStream_t st) {
    RouteArgs a;
    a.logits = c.logits;
    a.ld = c.ld;
    a.T = c.T;
    a.bias = c.bias;
    a.E = c.E;
    a.K = c.K;
    a.sigmoid = c.sigmoid;
    a.groups = c.kept < c.groups ? c.groups : 1;      // all groups kept: none matters
    a.kept = c.kept;
    a.best = c.best;
    a.renorm = c.renorm;
    a.size = c.E / a.groups;
    a.span = route_span(a.groups);
    a.scale = c.scale;
    a.ids = c.ids;
    a.weights = c.weights;
    const bool scores = c.bias || (a.groups > 1 && c.best == 2);
    const int n = (a.size + a.span - 1) / a.span;
    const dim3 grid(static_cast<uint32_t>((c.T + kRouteTokens - 1) / kRouteTokens));
    auto go = [&](auto width) {
        constexpr int N = decltype(width)::value;
        if (c.bf16) route_n<N, 1>(a, scores, grid, st);
        else route_n<N, 0>(a, scores, grid, st);
    };
    if (n <= 1) go(std::integral_constant<int, 1>{});
    else if (n <= 2) go(std::integral_constant<int, 2>{});
    else if (n <= 4) go(std::integral_constant<int, 4>{});
    else if (n <= 8) go(std::integral_constant<int, 8>{});
    else if (n <= 16) go(std::integral_constant<int, 16>{});
    else go(std::integral_constant<int, 32>{});
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteCall &c, const float *dw, void *dx, int64_t lddx, hipStream_t st) {
    RouteBackwardArgs a;
    a.logits = c.logits;
    a.ld = c.ld;
    a.T = c.T;
    a.E = c.E;
    a.K = c.K;
    a.sigmoid = c.sigmoid;
    a.renorm = c.renorm;
    a.scale = c.scale;
    a.ids = c.ids;
    a.dw = dw;
    a.dx = dx;
    a.lddx = lddx;
    const int n = (c.E + 63) / 64;
    const dim3 grid(static_cast<uint32_t>((c.T + kRouteTokens - 1) / kRouteTokens));
    auto go = [&](auto width) {
        constexpr int N = decltype(width)::value;
        if (c.bf16) hipLaunchKernelGGL((route_backward_kernel<N, 1>), grid, dim3(kRouteThreads), 0, st, a);
        else hipLaunchKernelGGL((route_backward_kernel<N, 0>), grid, dim3(kRouteThreads), 0, st, a);
    };
    if (n <= 1) go(std::integral_constant<int, 1>{});
    else if (n <= 2) go(std::integral_constant<int, 2>{});
    else if (n <= 4) go(std::integral_constant<int, 4>{});
    else if (n <= 8) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 16>{});
    return hipGetLastError();
}

}  // namespace logra
