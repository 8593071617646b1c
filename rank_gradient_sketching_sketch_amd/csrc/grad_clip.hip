// Global L2 norm over many gradients, and clipping by it.
//
//   norm = sqrt(sum_m sum_i g_mi^2),  coef = max_norm / norm where norm is
//   finite and above max_norm, else 1,  out_mi = coef * g_mi.
//
// The gradients of a step are many tensors (one sketch per projection,
// plus the dense gradients of what is not sketched), so the kernels walk a
// device table of them, cut into chunks of at most kGradChunk elements; each
// workgroup takes a contiguous range of chunks, finds its first one by
// bisection and steps through the table from there.
//
// Sums are taken in fp64 (squares of fp32 values neither overflow nor vanish
// there): per thread, over the workgroup by a fixed tree, and over the
// workgroups' partials in a fixed order, so results do not depend on timing.
// The scaling kernel's workgroups each add the partials themselves (at most
// kGradMaxWGs doubles, from the L2), so no workgroup waits for another and
// no counter has to be reset.
#include "common.hpp"
#include "launch.hpp"

namespace logra {

constexpr int kGradThreads = 256;

// Tensors need only their element's alignment (global memory takes 16-byte
// accesses at any address). The table holds their addresses as numbers, so
// the global address space is named here, else flat accesses would be built.
#define LOGRA_GLOBAL __attribute__((address_space(1)))
typedef u32x4_t u32x4_u2_t __attribute__((aligned(2)));
typedef u32x4_t u32x4_u4_t __attribute__((aligned(4)));
typedef LOGRA_GLOBAL char gbytes;

// Elements per 16-byte access of a type.
template <int BF16>
constexpr int grad_vec() { return BF16 ? 8 : 4; }

template <int BF16>
__device__ __forceinline__ float grad_get(const gbytes *p, int64_t i) {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(((const LOGRA_GLOBAL uint16_t *)p)[i]) << 16);
    return ((const LOGRA_GLOBAL float *)p)[i];
}

template <int BF16>
__device__ __forceinline__ void grad_put(gbytes *p, int64_t i, float v) {
    if (BF16)
        ((LOGRA_GLOBAL uint16_t *)p)[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
    else
        ((LOGRA_GLOBAL float *)p)[i] = v;
}

// V consecutive elements from index i (V * element size a multiple of 16).
template <int BF16, int V>
__device__ __forceinline__ void grad_load(const gbytes *p, int64_t i, float (&v)[V]) {
    if (BF16) {
#pragma unroll
        for (int q = 0; q < V / 8; ++q) {
            const u32x4_t w = *(const LOGRA_GLOBAL u32x4_u2_t *)(p + 2 * (i + 8 * q));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[8 * q + 2 * e] = bf16_lo(w[e]);
                v[8 * q + 2 * e + 1] = bf16_hi(w[e]);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const u32x4_t w = *(const LOGRA_GLOBAL u32x4_u4_t *)(p + 4 * (i + 4 * q));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * q + e] = __uint_as_float(w[e]);
        }
    }
}

template <int BF16, int V>
__device__ __forceinline__ void grad_store(gbytes *p, int64_t i, const float (&v)[V]) {
    if (BF16) {
#pragma unroll
        for (int q = 0; q < V / 8; ++q) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[8 * q + 2 * e], v[8 * q + 2 * e + 1]);
            *(LOGRA_GLOBAL u32x4_u2_t *)(p + 2 * (i + 8 * q)) = w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[4 * q + e]);
            *(LOGRA_GLOBAL u32x4_u4_t *)(p + 4 * (i + 4 * q)) = w;
        }
    }
}

// One chunk of a tensor: rows x cols elements from `at` (element index with
// row stride ld). Rows of a tensor without gaps are one long row.
struct GradChunk {
    gbytes *p;
    int64_t at, ld;
    int rows, cols;
};

__device__ __forceinline__ GradChunk grad_chunk(const GradEntry &e, int64_t c) {
    GradChunk k;
    k.p = (gbytes *)e.addr;
    k.ld = e.ld;
    if (e.rows_per_chunk > 0) {
        const int64_t r0 = c * e.rows_per_chunk;
        k.at = r0 * e.ld;
        k.rows = static_cast<int>(min(static_cast<int64_t>(e.rows_per_chunk), e.rows - r0));
        k.cols = static_cast<int>(e.cols);
    } else {
        const int64_t row = c / e.segs_per_row, seg = c - row * e.segs_per_row;
        const int64_t c0 = seg * e.seg_len;
        k.at = row * e.ld + c0;
        k.rows = 1;
        k.cols = static_cast<int>(min(static_cast<int64_t>(e.seg_len), e.cols - c0));
    }
    return k;
}

// f(chunk-local unit) over the chunk's units of V elements: a whole unit
// calls full(index), the rest of a row calls one(index) per element.
template <int V, int U, class Full, class One>
__device__ __forceinline__ void grad_units(int rows, int cols, Full full, One one) {
    const int upr = (cols + V - 1) / V;
    const int n = rows * upr;
    for (int u0 = threadIdx.x; u0 < n; u0 += U * blockDim.x) {
        int row[U], col[U];
        bool whole[U], some[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int u = u0 + q * blockDim.x;
            row[q] = rows == 1 ? 0 : u / upr;
            col[q] = (u - row[q] * upr) * V;
            some[q] = u < n;
            whole[q] = some[q] && col[q] + V <= cols;
        }
        full(row, col, whole);
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (some[q] && !whole[q])
                for (int e = col[q]; e < cols; ++e) one(row[q], e);
    }
}

constexpr int kGradUnroll = 4;

template <int BF16>
__device__ __forceinline__ double grad_chunk_sumsq(GradChunk k, double sum) {
    constexpr int V = grad_vec<BF16>(), U = kGradUnroll;
    if (k.ld == k.cols) k.cols *= k.rows, k.rows = 1;
    grad_units<V, U>(
        k.rows, k.cols,
        [&](const int (&row)[U], const int (&col)[U], const bool (&whole)[U]) {
            float v[U][V];
#pragma unroll
            for (int q = 0; q < U; ++q) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[q][e] = 0.f;
                if (whole[q]) grad_load<BF16, V>(k.p, k.at + row[q] * k.ld + col[q], v[q]);
            }
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const double d = v[q][e];
                    sum = fma(d, d, sum);
                }
        },
        [&](int row, int col) {
            const double d = grad_get<BF16>(k.p, k.at + row * k.ld + col);
            sum = fma(d, d, sum);
        });
    return sum;
}

template <int IN16, int OUT16>
__device__ __forceinline__ void grad_chunk_scale(GradChunk k, GradChunk o, float coef) {
    constexpr int V = (IN16 || OUT16) ? 8 : 4, U = kGradUnroll;
    if (k.ld == k.cols && o.ld == o.cols) k.cols *= k.rows, k.rows = 1;
    grad_units<V, U>(
        k.rows, k.cols,
        [&](const int (&row)[U], const int (&col)[U], const bool (&whole)[U]) {
            float v[U][V];
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (whole[q]) grad_load<IN16, V>(k.p, k.at + row[q] * k.ld + col[q], v[q]);
#pragma unroll
            for (int q = 0; q < U; ++q) {
                if (!whole[q]) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) v[q][e] *= coef;
                grad_store<OUT16, V>(o.p, o.at + row[q] * o.ld + col[q], v[q]);
            }
        },
        [&](int row, int col) {
            grad_put<OUT16>(o.p, o.at + row * o.ld + col, coef * grad_get<IN16>(k.p, k.at + row * k.ld + col));
        });
}

// The entry that holds chunk c (entries without elements hold none).
__device__ __forceinline__ int grad_find(const GradEntry *t, int n, int64_t c) {
    int lo = 0, hi = n;                  // first entry whose chunks end behind c
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t[mid].first + t[mid].chunks <= c) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Sum over the workgroup by a fixed tree; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockDim.x >> 6;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if (lane == 0) lds[wave] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < n; ++i) s += lds[i];
    return s;
}

__device__ __forceinline__ double grad_range_sumsq(const GradEntry *t, int n, int64_t c0, int64_t c1) {
    double sum = 0.0;
    if (c0 < c1) {
        int i = grad_find(t, n, c0);
        for (int64_t c = c0; c < c1; ++c) {
            while (c >= t[i].first + t[i].chunks) ++i;
            const GradEntry e = t[i];
            const GradChunk k = grad_chunk(e, c - e.first);
            sum = e.bf16 ? grad_chunk_sumsq<1>(k, sum) : grad_chunk_sumsq<0>(k, sum);
        }
    }
    return sum;
}

__device__ __forceinline__ void grad_range_scale(const GradEntry *t, const GradEntry *to, int n, int64_t c0,
                                                 int64_t c1, float coef) {
    if (c0 >= c1) return;
    int i = grad_find(t, n, c1 - 1);
    for (int64_t c = c1 - 1; c >= c0; --c) {
        while (c < t[i].first || t[i].chunks == 0) --i;
        const GradEntry e = t[i], o = to[i];
        const GradChunk k = grad_chunk(e, c - e.first), d = grad_chunk(o, c - e.first);
        if (e.bf16) {
            if (o.bf16) grad_chunk_scale<1, 1>(k, d, coef);
            else grad_chunk_scale<1, 0>(k, d, coef);
        } else {
            if (o.bf16) grad_chunk_scale<0, 1>(k, d, coef);
            else grad_chunk_scale<0, 0>(k, d, coef);
        }
    }
}

// A norm that is not finite (a gradient that is not) clips nothing: the
// caller sees it in *norm and skips the step.
__device__ __forceinline__ float clip_coef(double norm, float max_norm) {
    return (norm > max_norm && norm < __builtin_inf()) ? static_cast<float>(max_norm / norm) : 1.f;
}

__global__ __launch_bounds__(kGradThreads) void grad_sumsq_kernel(const GradEntry *__restrict__ t, int n,
                                                                  int64_t chunks, double *__restrict__ partials) {
    __shared__ double lds[kGradThreads / 64];
    const int64_t g = blockIdx.x, G = gridDim.x;
    const double s = block_sum(grad_range_sumsq(t, n, chunks * g / G, chunks * (g + 1) / G), lds);
    if (threadIdx.x == 0) partials[g] = s;
}

__device__ __forceinline__ double grad_partials_sum(const double *partials, int n, double *lds) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) s += partials[i];
    return block_sum(s, lds);
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(const double *__restrict__ partials, int n,
                                                                 float *__restrict__ norm) {
    __shared__ double lds[kGradThreads / 64];
    const double s = sqrt(grad_partials_sum(partials, n, lds));
    if (threadIdx.x == 0) *norm = static_cast<float>(s);
}

__global__ __launch_bounds__(kGradThreads) void grad_scale_kernel(
    const GradEntry *__restrict__ t, const GradEntry *__restrict__ to, int n, int64_t chunks,
    const double *__restrict__ partials, int n_partials, float max_norm, int in_place, float *__restrict__ norm,
    float *__restrict__ coef_out) {
    __shared__ double lds[kGradThreads / 64];
    const double s = sqrt(grad_partials_sum(partials, n_partials, lds));
    const float coef = clip_coef(s, max_norm);
    const int64_t g = blockIdx.x, G = gridDim.x;
    if (g == 0 && threadIdx.x == 0) {
        *norm = static_cast<float>(s);
        *coef_out = coef;
    }
    // a factor of one changes nothing in place
    if (in_place && coef == 1.f) return;
    grad_range_scale(t, to, n, chunks * g / G, chunks * (g + 1) / G, coef);
}

int grad_workgroups(int64_t chunks) {
    return static_cast<int>(chunks < 1 ? 1 : chunks < kGradMaxWGs ? chunks : kGradMaxWGs);
}

hipError_t launch_grad_norm(const GradEntry *t, int n, int64_t chunks, double *partials, float *norm,
                            hipStream_t st) {
    const int g = grad_workgroups(chunks);
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(g), dim3(kGradThreads), 0, st, t, n, chunks, partials);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradThreads), 0, st, partials, g, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradEntry *t, const GradEntry *to, int n, int64_t chunks, float max_norm,
                            double *partials, float *norm, float *coef, hipStream_t st) {
    const int g = grad_workgroups(chunks);
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(g), dim3(kGradThreads), 0, st, t, n, chunks, partials);
    hipLaunchKernelGGL(grad_scale_kernel, dim3(g), dim3(kGradThreads), 0, st, t, to, n, chunks, partials, g,
                       max_norm, t == to ? 1 : 0, norm, coef);
    return hipGetLastError();
}

}  // namespace logra
