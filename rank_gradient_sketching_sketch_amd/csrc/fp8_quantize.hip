// e4m3 codes with one fp32 scale per block: what the 8-bit products of
// fp8_matmul.hip read.
//
//   scale = max |x| / 448 over the block (1 for a block of zeros),
//   code  = e4m3(x / scale), to nearest even; 448 is e4m3's largest.
//
// Blocks are 1 x 128 (activations and gradients, along the contraction) or
// 128 x 128 (weights; the same blocks serve W and its transpose, so one weight
// has one set of codes in two orders). Quotients are IEEE divisions: an
// element's code hangs on its block alone. A NaN becomes the code for NaN, a
// block with an infinity the scale infinity.
//
// Bound by memory: x read once, codes and scales written once. 128 experts of
// 768 x 2048 in bf16 turned round: 121 us, 5.0 TB/s (a copy's rate is 5.1; with
// division instructions 154 us).
#include <math.h>

#include "common.hpp"
#include "launch.hpp"

namespace logra {

constexpr int kQuantThreads = 256;
constexpr float kE4M3Max = 448.f;

// global memory takes wide accesses at any address
typedef u32x4_t u32x4_q2_t __attribute__((aligned(2)));
typedef u32x4_t u32x4_q4_t __attribute__((aligned(4)));
typedef u32x2_t u32x2_q1_t __attribute__((aligned(1)));

__device__ __forceinline__ float quant_clamp(float q) {      // a NaN stays
    return q > kE4M3Max ? kE4M3Max : q < -kE4M3Max ? -kE4M3Max : q;
}

// Eight codes. Quotients are those of IEEE divisions: with the correctly
// rounded reciprocal of the scale, two corrections by the remainder give the
// correctly rounded quotient (Markstein), in five operations instead of ten,
// where nothing under- or overflows on the way: quotients that matter are
// above 2^-11 and the scale is kept above 2^-90. There no quotient is above 448
// but by its own rounding, either. Elsewhere (in a lane of the wave) the
// division itself. The remainder is taken as s q - x, whose zero times -y leaves a
// quotient of -0 its sign (x - s q would make it +0): which way is taken hangs on
// the wave's other blocks, a code must not.
__device__ __forceinline__ u32x2_t quant_codes(const float (&x)[8], float scale) {
    float q[8];
    if (__ballot(!(scale > 0x1p-90f && scale < 0x1p90f)) == 0) {
        const float y = 1.f / scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q0 = x[e] * y;
            const float q1 = fmaf(fmaf(scale, q0, -x[e]), -y, q0);
            q[e] = fmaf(fmaf(scale, q1, -x[e]), -y, q1);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = quant_clamp(x[e] / scale);
    }
    u32x2_t w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        w[h] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], v, true));
    }
    return w;
}

__device__ __forceinline__ float quant_scale(float amax) {
    const float s = amax / kE4M3Max;
    return s > 0.f ? s : 1.f;
}

// Up to eight elements of a row from column c of `cols`, zeros behind it.
template <int BF16>
__device__ __forceinline__ void quant_load(const char *row, int64_t c, int64_t cols, float (&x)[8]) {
    if (c + 8 <= cols) {
        if (BF16) {
            const u32x4_t w = *reinterpret_cast<const u32x4_q2_t *>(row + 2 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = bf16_lo(w[e]);
                x[2 * e + 1] = bf16_hi(w[e]);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4_t w = *reinterpret_cast<const u32x4_q4_t *>(row + 4 * c + 16 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * h + e] = __uint_as_float(w[e]);
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = 0.f;
        if (c + e < cols)
            x[e] = BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[c + e]) << 16)
                        : reinterpret_cast<const float *>(row)[c + e];
    }
}

__device__ __forceinline__ float quant_amax(const float (&x)[8], float m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
    return m;
}

// 1 x 128 blocks: sixteen lanes a block.
template <int BF16>
__global__ __launch_bounds__(kQuantThreads) void quant_rows_kernel(const char *__restrict__ x, int64_t ldx,
                                                                   int64_t rows, int64_t cols, int kb,
                                                                   uint8_t *__restrict__ codes, int64_t ldc,
                                                                   float *__restrict__ scales) {
    const int64_t block = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 16) + (threadIdx.x >> 4);
    const int64_t r = block / kb;
    const int b = static_cast<int>(block - r * kb), i = threadIdx.x & 15;
    const int64_t c = 128 * static_cast<int64_t>(b) + 8 * i;
    const bool live = r < rows;
    float v[8];
    quant_load<BF16>(x + (live ? r * ldx * (BF16 ? 2 : 4) : 0), c, live ? cols : 0, v);
    float m = quant_amax(v, 0.f);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float scale = quant_scale(m);
    if (!live) return;
    const u32x2_t w = quant_codes(v, scale);
    uint8_t *dst = codes + r * ldc + c;
    if (c + 8 <= cols) {
        *reinterpret_cast<u32x2_q1_t *>(dst) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < cols) dst[e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
    }
    if (i == 0) scales[r * kb + b] = scale;
}

// 128 x 128 blocks, a workgroup each: thread (g, h) has rows 4 g .. 4 g + 3,
// columns 8 h .. and 64 + 8 h .. . Turned, the codes of four rows and one
// column are one word of the LDS tile's row for that column (33 words a row:
// the words that a wave writes at once are on 64 banks).
constexpr int kQuantPitch = 33;

template <int BF16, int TURNED>
__global__ __launch_bounds__(kQuantThreads) void quant_tiles_kernel(const char *__restrict__ x, int64_t ldx,
                                                                    int64_t rows, int64_t cols, int rb, int kb,
                                                                    uint8_t *__restrict__ codes, int64_t ldc,
                                                                    float *__restrict__ scales) {
    __shared__ float part[kQuantThreads / 64];
    __shared__ uint32_t tile[TURNED ? 128 * kQuantPitch : 1];
    const int64_t id = blockIdx.x, per = static_cast<int64_t>(rb) * kb;
    const int64_t batch = id / per;
    const int rest = static_cast<int>(id - batch * per), br = rest / kb, bc = rest - br * kb;
    const int64_t r0 = 128 * static_cast<int64_t>(br), c0 = 128 * static_cast<int64_t>(bc);
    const int g = threadIdx.x >> 3, h = threadIdx.x & 7;
    x += batch * rows * ldx * (BF16 ? 2 : 4);
    codes += batch * (TURNED ? cols : rows) * ldc;
    float v[4][2][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 4 * g + i;
        const bool live = r < rows;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            quant_load<BF16>(x + (live ? r * ldx * (BF16 ? 2 : 4) : 0), c0 + 64 * q + 8 * h, live ? cols : 0, v[i][q]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) m = quant_amax(v[i][q], m);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 64; ++i) m = fmaxf(m, part[i]);
    const float scale = quant_scale(m);
    if (threadIdx.x == 0) scales[batch * per + (TURNED ? static_cast<int64_t>(bc) * rb + br : rest)] = scale;
    if (!TURNED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 4 * g + i;
            if (r >= rows) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t c = c0 + 64 * q + 8 * h;
                const u32x2_t w = quant_codes(v[i][q], scale);
                uint8_t *dst = codes + r * ldc + c;
                if (c + 8 <= cols) {
                    *reinterpret_cast<u32x2_q1_t *>(dst) = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < cols) dst[e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
                }
            }
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        u32x2_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = quant_codes(v[i][q], scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // byte e of the four rows in one word
            const uint32_t sel = static_cast<uint32_t>(e % 4) | static_cast<uint32_t>(4 + e % 4) << 8;
            const uint32_t lo = __builtin_amdgcn_perm(w[1][e / 4], w[0][e / 4], 0x0C0C0000u | sel);
            const uint32_t hi = __builtin_amdgcn_perm(w[3][e / 4], w[2][e / 4], 0x0C0C0000u | sel);
            tile[(64 * q + 8 * h + e) * kQuantPitch + g] = lo | hi << 16;
        }
    }
    __syncthreads();
    // eight threads a row of the turned tile, sixteen codes each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = 32 * i + (threadIdx.x >> 3), w0 = 4 * h;
        if (c0 + c >= cols) break;
        const uint32_t *src = tile + c * kQuantPitch + w0;
        uint8_t *dst = codes + (c0 + c) * ldc + r0 + 4 * w0;
        const int64_t left = rows - (r0 + 4 * w0);
        typedef u32x4_t u32x4_q1_t __attribute__((aligned(1)));
        if (left >= 16) {
            *reinterpret_cast<u32x4_q1_t *>(dst) = u32x4_t{src[0], src[1], src[2], src[3]};
        } else {
            for (int e = 0; e < 16; ++e)
                if (e < left) dst[e] = static_cast<uint8_t>(src[e / 4] >> (8 * (e % 4)));
        }
    }
}

hipError_t launch_fp8_quantize(const QuantizeCall &c, hipStream_t st) {
    const int kb = static_cast<int>((c.cols + 127) / 128);
    const char *x = static_cast<const char *>(c.x);
    if (c.block_rows == 1) {
        const int64_t rows = c.batch * c.rows, blocks = rows * kb;
        const dim3 grid(static_cast<uint32_t>((blocks + kQuantThreads / 16 - 1) / (kQuantThreads / 16)));
        hipLaunchKernelGGL(c.bf16 ? quant_rows_kernel<1> : quant_rows_kernel<0>, grid, dim3(kQuantThreads), 0, st, x,
                           c.ldx, rows, c.cols, kb, c.codes, c.ldc, c.scales);
        return hipGetLastError();
    }
    const int rb = static_cast<int>((c.rows + 127) / 128);
    const dim3 grid(static_cast<uint32_t>(c.batch * rb * kb));
    auto kernel = c.turned ? (c.bf16 ? quant_tiles_kernel<1, 1> : quant_tiles_kernel<0, 1>)
                           : (c.bf16 ? quant_tiles_kernel<1, 0> : quant_tiles_kernel<0, 0>);
    hipLaunchKernelGGL(kernel, grid, dim3(kQuantThreads), 0, st, x, c.ldx, c.rows, c.cols, rb, kb, c.codes, c.ldc,
                       c.scales);
    return hipGetLastError();
}

}  // namespace logra
