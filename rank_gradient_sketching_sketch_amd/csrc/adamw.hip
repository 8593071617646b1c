// AdamW over many tensors at once, for what the sketch leaves out: embeddings,
// norm gains, router weights.
//
//   g' = c g             (c from the gradients' norm, see below)
//   m' = b1 m + (1 - b1) g',   v' = b2 v + (1 - b2) g'^2
//   p' = p - (lr wd p + lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps))
//
// The moments of all tensors lie one after the other in blocks of 256
// elements, every tensor beginning a block. In 32 bits they are fp32. In 8
// bits m and sqrt(v) are e4m3 codes with one fp32 scale per block and moment
// (the largest of a block is 448 scales): the root needs half the binades that
// v would. The update itself uses the fp32 m' and v', so a step's rounding
// reaches later steps alone.
//
// The codes are rounded up or down by chance (16 bits of a counter hash per
// value, the library's own, keyed by seed and step), not to nearest: a step
// moves v by about 1 - b2 = 0.1 % of itself, a code's step is 6 to 12 % of the
// root, so the nearest code would be the old one for ever. Each rounding, of m
// and of the root, is unbiased; the root's square is not: it is too high by the
// rounding's variance, code step times what a step moves the root by, which adds
// up to 3 to 6 % of v (gradients drawn from one Gaussian each, any b2 near 1; 4.9 %
// measured after 1000 steps, b2 0.99; 12 % where the block's scale moves as much),
// so steps are some 2 % shorter. A root that is not zero keeps at least the
// smallest code, as a moment m over a root of zero would be a step of m / eps.
//
// Sums are fp32 in the order of the formulas (no contraction), which fixes the
// codes bit by bit.
//
// Bound by memory: parameters and moments read and written once, gradients
// read, copies written. 49 M elements, fp32: 256 us, 5.4 TB/s; 115 M with bf16
// gradients and copies and moments in 8 bits (16.06 bytes an element): 363 us,
// 5.1 TB/s.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "signs.hpp"

#pragma clang fp contract(off)

namespace logra {

constexpr int kAdamThreads = 256;
constexpr int kAdamPerWG = kAdamThreads / 32;      // blocks that a workgroup has at a time, half a wave each

#define LOGRA_GLOBAL __attribute__((address_space(1)))
typedef u32x4_t u32x4_a2_t __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4_t __attribute__((aligned(4)));
typedef LOGRA_GLOBAL char abytes;

template <int BF16>
__device__ __forceinline__ float adam_get(const abytes *p, int64_t i) {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(((const LOGRA_GLOBAL uint16_t *)p)[i]) << 16);
    return ((const LOGRA_GLOBAL float *)p)[i];
}
template <int BF16>
__device__ __forceinline__ void adam_put(abytes *p, int64_t i, float v) {
    if (BF16) ((LOGRA_GLOBAL uint16_t *)p)[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
    else ((LOGRA_GLOBAL float *)p)[i] = v;
}
template <int BF16>
__device__ __forceinline__ void adam_load8(const abytes *p, int64_t i, float (&v)[8]) {
    if (BF16) {
        const u32x4_t w = *(const LOGRA_GLOBAL u32x4_a2_t *)(p + 2 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = bf16_lo(w[e]);
            v[2 * e + 1] = bf16_hi(w[e]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4_t w = *(const LOGRA_GLOBAL u32x4_a4_t *)(p + 4 * i + 16 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = __uint_as_float(w[e]);
        }
    }
}
template <int BF16>
__device__ __forceinline__ void adam_store8(abytes *p, int64_t i, const float (&v)[8]) {
    if (BF16) {
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        *(LOGRA_GLOBAL u32x4_a2_t *)(p + 2 * i) = w;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[4 * h + e]);
            *(LOGRA_GLOBAL u32x4_a4_t *)(p + 4 * i + 16 * h) = w;
        }
    }
}

// Eight elements of a tensor from element i of its rows laid end to end, n of
// them to be had; ld: the row stride. Elements that are not there are zeros.
template <int BF16>
__device__ __forceinline__ void adam_load(uint64_t addr, int64_t i, int n, int64_t cols, int64_t ld, float (&v)[8]) {
    const abytes *p = (const abytes *)addr;
    if (ld == cols && n == 8) {
        adam_load8<BF16>(p, i, v);
        return;
    }
    int64_t row = ld == cols ? 0 : i / cols, col = i - row * cols;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0.f;
        if (e < n) v[e] = adam_get<BF16>(p, row * ld + col);
        if (++col == cols && ld != cols) {
            col = 0;
            ++row;
        }
    }
}
template <int BF16>
__device__ __forceinline__ void adam_store(uint64_t addr, int64_t i, int n, int64_t cols, int64_t ld,
                                           const float (&v)[8]) {
    abytes *p = (abytes *)addr;
    if (ld == cols && n == 8) {
        adam_store8<BF16>(p, i, v);
        return;
    }
    int64_t row = ld == cols ? 0 : i / cols, col = i - row * cols;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e < n) adam_put<BF16>(p, row * ld + col, v[e]);
        if (++col == cols && ld != cols) {
            col = 0;
            ++row;
        }
    }
}

// Largest of the half-wave (32 lanes).
__device__ __forceinline__ uint32_t half_max(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t w = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o));
        v = v > w ? v : w;
    }
    return v;
}

// A block's scale from the bits of its largest magnitude, and what its values
// are multiplied by. A block that is all but zero is zeros; one that is not
// finite becomes NaN.
__device__ __forceinline__ float adam_scale(uint32_t most, float *inv) {
    const float amax = __uint_as_float(most);
    if (most >= 0x7F800000u) {
        *inv = 0.f;
        return __uint_as_float(0x7FC00000u);
    }
    const bool live = amax >= 0x1p-100f;
    *inv = live ? 448.f / amax : 0.f;
    return live ? amax / 448.f : 0.f;
}

// The e4m3 values below or above |x| inv, by chance: u is uniform in
// 0 .. 65535, taken in the middle of its step. 20 mantissa bits are dropped
// from normal values; subnormal ones (below 2^-6) are whole multiples of 2^-9,
// which few blocks have: they are looked at only if a lane does.
__device__ __forceinline__ void adam_round(float (&x)[8], float inv, const uint32_t (&u)[8]) {
    float a[8], q[8];
    uint32_t least = ~0u;          // of the bits above zero
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // the largest may come out a unit or two above 448: cut off again
        a[e] = fabsf(x[e]) * inv;
        q[e] = __uint_as_float((__float_as_uint(a[e]) + (u[e] << 4 | 8u)) & 0xFFF00000u);      // zero stays
        least = min(least, __float_as_uint(a[e]) - 1u);
    }
    if (__ballot(least < __float_as_uint(0x1p-6f) - 1u) != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = floorf(a[e] * 512.f + (static_cast<float>(u[e]) + 0.5f) * 0x1p-16f) * 0x1p-9f;
            q[e] = a[e] < 0x1p-6f ? s : q[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = copysignf(q[e], x[e]);
}

// Square roots: the reciprocal root's estimate (one unit off at most) and a
// correction by the remainder, which is the correctly rounded root but where
// that lies within 2^-20 of a unit of the middle between two values. Outside
// of what the remainder is exact for, the library's.
__device__ __forceinline__ void adam_roots(const float (&v)[8], float (&r)[8]) {
    uint32_t least = ~0u, most = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = __builtin_amdgcn_rsqf(fmaxf(v[e], 0x1p-100f));
        const float s = v[e] * y;
        r[e] = fmaf(fmaf(-s, s, v[e]), 0.5f * y, s);
        least = min(least, __float_as_uint(v[e]) - 1u);
        most = max(most, __float_as_uint(v[e]));
    }
    if (__ballot(least < __float_as_uint(0x1p-100f) - 1u || most > __float_as_uint(0x1p100f)) != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = sqrtf(v[e]);
    }
}

// Eight exact e4m3 values as codes.
__device__ __forceinline__ u32x2_t adam_pack(const float (&q)[8]) {
    u32x2_t w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        w[h] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], v, true));
    }
    return w;
}
__device__ __forceinline__ void adam_unpack(u32x2_t w, float scale, float (&v)[8]) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), false);
        const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), true);
        v[4 * h] = lo[0] * scale;
        v[4 * h + 1] = lo[1] * scale;
        v[4 * h + 2] = hi[0] * scale;
        v[4 * h + 3] = hi[1] * scale;
    }
}

// The entry that holds block b, found by a whole wave (as in the gradient
// lists: each lane looks at the last of one of 64 parts of the range).
__device__ __forceinline__ int adam_find(const AdamEntry *t, int n, int64_t b) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (n > 1) {
        const int part = (n + 63) / 64, i = min((lane + 1) * part, n) - 1;
        const uint64_t past = __ballot(t[lo + i].first + t[lo + i].blocks > b);
        const int at = __builtin_ctzll(past) * part;
        lo += at;
        n = min(part, n - at);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

template <int BITS, int P16, int G16>
__device__ __forceinline__ void adam_block(const AdamCall &c, const AdamEntry &e, int64_t b, float coef) {
    const int l = threadIdx.x & 31;
    const int64_t i = (b - e.first) * kAdamBlock + 8 * l, s = b * kAdamBlock + 8 * l;
    const int n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), e.rows * e.cols - i)));
    float p[8], g[8], m[8], v[8], r[8];
    adam_load<P16>(e.param, i, n, e.cols, e.ld_param, p);
    adam_load<G16>(e.grad, i, n, e.cols, e.ld_grad, g);
    if (BITS == 8) {
        const u32x2_t mc = *reinterpret_cast<const u32x2_t *>(static_cast<const uint8_t *>(c.m) + s);
        const u32x2_t vc = *reinterpret_cast<const u32x2_t *>(static_cast<const uint8_t *>(c.v) + s);
        adam_unpack(mc, c.scales[b], m);
        adam_unpack(vc, c.scales[c.blocks + b], r);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = r[q] * r[q];
    } else {
        const float *ms = static_cast<const float *>(c.m) + s, *vs = static_cast<const float *>(c.v) + s;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4_t a = *reinterpret_cast<const u32x4_t *>(ms + 4 * h);
            const u32x4_t w = *reinterpret_cast<const u32x4_t *>(vs + 4 * h);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                m[4 * h + q] = __uint_as_float(a[q]);
                v[4 * h + q] = __uint_as_float(w[q]);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float gc = g[q] * coef;
        m[q] = c.beta1 * m[q] + c.rest1 * gc;
        v[q] = c.beta2 * v[q] + c.rest2 * (gc * gc);
    }
    adam_roots(v, r);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        // a quotient by a reciprocal's estimate: within 2^-22 of the update
        const float upd = c.rate * (m[q] * __builtin_amdgcn_rcpf(fmaf(r[q], c.root_scale, c.eps)));
        p[q] = p[q] - fmaf(c.decay, p[q], upd);
    }
    adam_store<P16>(e.param, i, n, e.cols, e.ld_param, p);
    if (e.copy) {
        if (e.copy_bf16) adam_store<1>(e.copy, i, n, e.cols, e.ld_copy, p);
        else adam_store<0>(e.copy, i, n, e.cols, e.ld_copy, p);
    }
    if (BITS == 8) {
        uint32_t mm = 0, mv = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t a = __float_as_uint(m[q]) & 0x7FFFFFFFu, w = __float_as_uint(v[q]) & 0x7FFFFFFFu;
            mm = mm > a ? mm : a;
            mv = mv > w ? mv : w;
        }
        // the largest root is the root of the largest v
        mv = half_max(mv);
        float inv_m, inv_r;
        const float scale_m = adam_scale(half_max(mm), &inv_m);
        const float scale_r = adam_scale(mv >= 0x7F800000u ? mv : __float_as_uint(sqrtf(__uint_as_float(mv))), &inv_r);
        uint32_t um[8], ur[8];
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
            const uint64_t w = splitmix_finalize(c.key + (static_cast<uint64_t>(s + q) / 2 + 1) * kGolden);
            const uint32_t lo = static_cast<uint32_t>(w), hi = static_cast<uint32_t>(w >> 32);
            um[q] = lo & 0xFFFFu;
            um[q + 1] = hi & 0xFFFFu;
            ur[q] = lo >> 16;
            ur[q + 1] = hi >> 16;
        }
        const float least = scale_r > 0.f ? 0x1p-9f : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = r[q];
        adam_round(m, inv_m, um);
        adam_round(v, inv_r, ur);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = r[q] > 0.f ? fmaxf(v[q], least) : v[q];
        *reinterpret_cast<u32x2_t *>(static_cast<uint8_t *>(c.m) + s) = adam_pack(m);
        *reinterpret_cast<u32x2_t *>(static_cast<uint8_t *>(c.v) + s) = adam_pack(v);
        if (l == 0) {
            c.scales[b] = scale_m;
            c.scales[c.blocks + b] = scale_r;
        }
    } else {
        float *ms = static_cast<float *>(c.m) + s, *vs = static_cast<float *>(c.v) + s;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4_t a, w;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = __float_as_uint(m[4 * h + q]);
                w[q] = __float_as_uint(v[4 * h + q]);
            }
            *reinterpret_cast<u32x4_t *>(ms + 4 * h) = a;
            *reinterpret_cast<u32x4_t *>(vs + 4 * h) = w;
        }
    }
}

// Every workgroup has a run of blocks, each half of a wave every eighth of
// them; it finds the run's first tensor and walks on from there.
template <int BITS>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamCall c) {
    float coef = 1.f;
    if (c.norm) {
        const float norm = *c.norm;
        if (!(norm < INFINITY)) return;           // infinity or NaN: the step is left out
        if (norm > c.max_norm) coef = static_cast<float>(c.max_norm / static_cast<double>(norm));
    }
    const int64_t g = blockIdx.x, G = gridDim.x;
    const int64_t b0 = c.blocks * g / G, b1 = c.blocks * (g + 1) / G;
    if (b0 >= b1) return;
    int at = adam_find(c.table, c.n, b0);
    AdamEntry e = c.table[at];
    for (int64_t b = b0 + (threadIdx.x >> 5); b < b1; b += kAdamPerWG) {
        while (b >= e.first + e.blocks) e = c.table[++at];
        if (e.param_bf16) {
            if (e.grad_bf16) adam_block<BITS, 1, 1>(c, e, b, coef);
            else adam_block<BITS, 1, 0>(c, e, b, coef);
        } else {
            if (e.grad_bf16) adam_block<BITS, 0, 1>(c, e, b, coef);
            else adam_block<BITS, 0, 0>(c, e, b, coef);
        }
    }
}

hipError_t launch_adamw(const AdamCall &c, int bits, hipStream_t st) {
    const int64_t wgs = (c.blocks + kAdamPerWG - 1) / kAdamPerWG;
    // 115 M elements with 8-bit moments, us with 1024 / 2048 / 4096 / 16384 workgroups
    // at most: 402 / 401 / 392 / 363; 49 M with fp32 moments 283 / 280 / 275 / 260, 256
    // with one for every eight blocks
    const int64_t most = 1 << 16;
    const dim3 grid(static_cast<uint32_t>(wgs < most ? wgs : most));
    hipLaunchKernelGGL(bits == 8 ? adamw_kernel<8> : adamw_kernel<32>, grid, dim3(kAdamThreads), 0, st, c);
    return hipGetLastError();
}

}  // namespace logra
