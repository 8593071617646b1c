// Global L2 norm over many gradients, and clipping by it.
//
//   norm = sqrt(sum_m sum_i g_mi^2),  coef = max_norm / norm where norm is
//   finite and above max_norm, else 1,  out_mi = coef * g_mi.
//
// The gradients of a step are many tensors (one sketch per projection,
// plus the dense gradients of what is not sketched), so the kernels walk a
// device table of them, cut into chunks of at most kGradChunk elements; each
// workgroup takes a contiguous range of chunks, finds the first one's tensor
// and steps through the table from there, reading what lies in one
// tensor without gaps as one run.
//
// Sums are taken in fp64 (squares of fp32 values neither overflow nor vanish
// there, and the reads hide the arithmetic): per thread, over the workgroup by
// a fixed tree, and over the workgroups' partials in a fixed order, so results
// do not depend on timing. The scaling kernel's workgroups each add the
// partials themselves (at most kGradMaxWGs doubles, from the L2), so no
// workgroup waits for another and no counter has to be reset. Few elements are
// done by one workgroup in one launch.
//
// Bound by memory: the gradients are read twice (the factor is known only
// when all have been read once) and written once. 196 fp32 sketches of 1.42 GB
// in all, scaled into other tensors: 214 us for the sum (6.6 TB/s) and 532 us
// for the scaling (5.4 TB/s); a copy of 1 GiB reaches 5.2 TB/s on this card.
// What it took from a first version's 323 + 603 us: runs over whole tensors
// instead of chunks with a table look-up each (223 + 579), then streaming
// loads and stores and four times the workgroups for the scaling. Reading
// the second time from the back, to meet what the last-level cache kept,
// changed nothing.
#include "common.hpp"
#include "launch.hpp"

namespace logra {

constexpr int kGradThreads = 256;
constexpr int kGradSmallThreads = 1024;
// What one workgroup takes alone, in one launch: nine tensors of 1536 elements
// take it 5.0 us, two launches of the others 9.1 us.
constexpr int64_t kGradSmallChunks = 32, kGradSmallElements = 32768;
// Elements above which loads and stores are marked as not to be kept in the
// caches: 256 MB of fp32, what the last-level cache holds. A count of bytes
// would let bf16 lists of 128 to 256 MB be kept; that was not measured.
constexpr int64_t kGradStream = 1ll << 26;

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
template <int BF16, int V, int NT = 0>
__device__ __forceinline__ void grad_load(const gbytes *p, int64_t i, float (&v)[V]) {
    if (BF16) {
#pragma unroll
        for (int q = 0; q < V / 8; ++q) {
            const LOGRA_GLOBAL u32x4_u2_t *src = (const LOGRA_GLOBAL u32x4_u2_t *)(p + 2 * (i + 8 * q));
            const u32x4_t w = NT ? __builtin_nontemporal_load(src) : *src;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[8 * q + 2 * e] = bf16_lo(w[e]);
                v[8 * q + 2 * e + 1] = bf16_hi(w[e]);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const LOGRA_GLOBAL u32x4_u4_t *src = (const LOGRA_GLOBAL u32x4_u4_t *)(p + 4 * (i + 4 * q));
            const u32x4_t w = NT ? __builtin_nontemporal_load(src) : *src;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * q + e] = __uint_as_float(w[e]);
        }
    }
}

// The first n < V of them, zeros behind: the requests go out together.
template <int BF16, int V>
__device__ __forceinline__ void grad_load_some(const gbytes *p, int64_t i, int n, float (&v)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        v[e] = 0.f;
        if (e < n) v[e] = grad_get<BF16>(p, i + e);
    }
}

template <int BF16, int V, int NT = 0>
__device__ __forceinline__ void grad_store(gbytes *p, int64_t i, const float (&v)[V]) {
    if (BF16) {
#pragma unroll
        for (int q = 0; q < V / 8; ++q) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[8 * q + 2 * e], v[8 * q + 2 * e + 1]);
            LOGRA_GLOBAL u32x4_u2_t *dst = (LOGRA_GLOBAL u32x4_u2_t *)(p + 2 * (i + 8 * q));
            if (NT) __builtin_nontemporal_store(w, dst);
            else *dst = w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[4 * q + e]);
            LOGRA_GLOBAL u32x4_u4_t *dst = (LOGRA_GLOBAL u32x4_u4_t *)(p + 4 * (i + 4 * q));
            if (NT) __builtin_nontemporal_store(w, dst);
            else *dst = w;
        }
    }
}

// The threads that go through a run or a chunk together: a workgroup, or one
// of its waves.
struct GradGroup {
    int id, size;
};

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

// f(chunk-local unit) over the chunk's units of V elements: whole units go to
// full(rows, columns, which), the rest of a row to rest(row, column).
template <int V, int U, class Full, class Some>
__device__ __forceinline__ void grad_units(GradGroup g, int rows, int cols, Full full, Some rest) {
    const int upr = (cols + V - 1) / V;
    const int n = rows * upr;
    for (int u0 = g.id; u0 < n; u0 += U * g.size) {
        int row[U], col[U];
        bool whole[U], some[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int u = u0 + q * g.size;
            row[q] = rows == 1 ? 0 : u / upr;
            col[q] = (u - row[q] * upr) * V;
            some[q] = u < n;
            whole[q] = some[q] && col[q] + V <= cols;
        }
        full(row, col, whole);
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (some[q] && !whole[q]) rest(row[q], col[q]);
    }
}

// Units of gapped chunks, and fp32 bytes of runs, that a thread has in flight.
constexpr int kGradUnroll = 4, kGradRunBytes = 128;

// A run of n elements without gaps: whole(index) for every U units of V
// elements of a thread at once while they last, then unit by unit, then
// one(index) for the last elements (fewer than V).
template <int V, int U, class Many, class Unit, class One>
__device__ __forceinline__ void grad_run(GradGroup g, int64_t n, Many many, Unit unit, One one) {
    const int64_t step = static_cast<int64_t>(g.size) * V;
    int64_t i = static_cast<int64_t>(g.id) * V;
    for (; i + (U - 1) * step + V <= n; i += U * step) many(i, step);
    for (; i + V <= n; i += step) unit(i);
    const int64_t e = n / V * V + g.id;      // the last elements: one for each of the first threads
    if (e < n) one(e);
}

template <int BF16, int NT>
__device__ __forceinline__ double grad_run_sumsq(GradGroup g, const gbytes *p, int64_t n, double sum) {
    constexpr int V = grad_vec<BF16>(), U = kGradRunBytes / 16 / (BF16 ? 2 : 1);
    auto add = [&](float x) {
        const double d = x;
        sum = fma(d, d, sum);
    };
    grad_run<V, U>(
        g, n,
        [&](int64_t i, int64_t step) {
            float v[U][V];
#pragma unroll
            for (int q = 0; q < U; ++q) grad_load<BF16, V, NT>(p, i + q * step, v[q]);
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int e = 0; e < V; ++e) add(v[q][e]);
        },
        [&](int64_t i) {
            float v[V];
            grad_load<BF16, V>(p, i, v);
#pragma unroll
            for (int e = 0; e < V; ++e) add(v[e]);
        },
        [&](int64_t i) { add(grad_get<BF16>(p, i)); });
    return sum;
}

template <int IN16, int OUT16, int NT>
__device__ __forceinline__ void grad_run_scale(GradGroup g, const gbytes *p, gbytes *o, int64_t n, float coef) {
    constexpr int V = (IN16 || OUT16) ? 8 : 4, U = kGradRunBytes / 4 / V;
    grad_run<V, U>(
        g, n,
        [&](int64_t i, int64_t step) {
            float v[U][V];
#pragma unroll
            for (int q = 0; q < U; ++q) grad_load<IN16, V, NT>(p, i + q * step, v[q]);
#pragma unroll
            for (int q = 0; q < U; ++q) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[q][e] *= coef;
                grad_store<OUT16, V, NT>(o, i + q * step, v[q]);
            }
        },
        [&](int64_t i) {
            float v[V];
            grad_load<IN16, V>(p, i, v);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= coef;
            grad_store<OUT16, V>(o, i, v);
        },
        [&](int64_t i) { grad_put<OUT16>(o, i, coef * grad_get<IN16>(p, i)); });
}

// Chunks of tensors with gaps between their rows.
template <int BF16>
__device__ __forceinline__ double grad_chunk_sumsq(GradGroup g, GradChunk k, double sum) {
    constexpr int V = grad_vec<BF16>(), U = kGradUnroll;
    grad_units<V, U>(
        g, k.rows, k.cols,
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
            float v[V];
            grad_load_some<BF16, V>(k.p, k.at + row * k.ld + col, k.cols - col, v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const double d = v[e];
                sum = fma(d, d, sum);
            }
        });
    return sum;
}

template <int IN16, int OUT16>
__device__ __forceinline__ void grad_chunk_scale(GradGroup g, GradChunk k, GradChunk o, float coef) {
    constexpr int V = (IN16 || OUT16) ? 8 : 4, U = kGradUnroll;
    grad_units<V, U>(
        g, k.rows, k.cols,
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
            float v[V];
            grad_load_some<IN16, V>(k.p, k.at + row * k.ld + col, k.cols - col, v);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < k.cols - col) grad_put<OUT16>(o.p, o.at + row * o.ld + col + e, coef * v[e]);
        });
}

// The entry that holds chunk c (entries without elements hold none), found by
// whole waves: each lane looks at the last of one of 64 parts of the range.
__device__ __forceinline__ int grad_find(const GradEntry *t, int n, int64_t c) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (n > 1) {                      // the entry is among n from lo
        const int part = (n + 63) / 64, i = min((lane + 1) * part, n) - 1;
        const uint64_t past = __ballot(t[lo + i].first + t[lo + i].chunks > c);
        const int at = __builtin_ctzll(past) * part;
        lo += at;
        n = min(part, n - at);
    }
    return __builtin_amdgcn_readfirstlane(lo);
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

// First element of an entry's chunk c, of a tensor without gaps.
__device__ __forceinline__ int64_t grad_run_at(const GradEntry &e, int64_t c) {
    if (e.rows_per_chunk > 0) return min(c * e.rows_per_chunk, e.rows) * e.cols;
    const int64_t row = c / e.segs_per_row;
    return row * e.cols + (c - row * e.segs_per_row) * e.seg_len;
}

// f(entry, its number, first chunk, last chunk + 1) for the part of every
// entry that chunks c0 .. c1 - 1 of the list hold.
template <class F>
__device__ __forceinline__ void grad_entries(const GradEntry *t, int n, int64_t c0, int64_t c1, F f) {
    if (c0 >= c1) return;
    for (int i = grad_find(t, n, c0); c0 < c1; ++i) {
        const GradEntry e = t[i];
        const int64_t last = min(c1, e.first + e.chunks);
        if (c0 < last) f(e, i, c0 - e.first, last - e.first);
        c0 = max(c0, last);
    }
}

template <int NT>
__device__ __forceinline__ double grad_entry_sumsq(GradGroup g, const GradEntry &e, int64_t a, int64_t b, double sum) {
    if (e.ld == e.cols) {
        const int64_t from = grad_run_at(e, a), n = grad_run_at(e, b) - from;
        const gbytes *p = (const gbytes *)e.addr + from * (e.bf16 ? 2 : 4);
        return e.bf16 ? grad_run_sumsq<1, NT>(g, p, n, sum) : grad_run_sumsq<0, NT>(g, p, n, sum);
    }
    for (int64_t c = a; c < b; ++c) {
        const GradChunk k = grad_chunk(e, c);
        sum = e.bf16 ? grad_chunk_sumsq<1>(g, k, sum) : grad_chunk_sumsq<0>(g, k, sum);
    }
    return sum;
}

template <int IN16, int OUT16, int NT>
__device__ __forceinline__ void grad_entry_scale(GradGroup g, const GradEntry &e, const GradEntry &o, int64_t a,
                                                 int64_t b, float coef) {
    if (e.ld == e.cols && o.ld == o.cols) {
        const int64_t from = grad_run_at(e, a);
        grad_run_scale<IN16, OUT16, NT>(g, (const gbytes *)e.addr + from * (IN16 ? 2 : 4),
                                        (gbytes *)o.addr + from * (OUT16 ? 2 : 4), grad_run_at(e, b) - from, coef);
        return;
    }
    for (int64_t c = a; c < b; ++c) grad_chunk_scale<IN16, OUT16>(g, grad_chunk(e, c), grad_chunk(o, c), coef);
}

template <int NT>
__device__ __forceinline__ void grad_entry_scale_any(GradGroup g, const GradEntry &e, const GradEntry &o, int64_t a,
                                                     int64_t b, float coef) {
    if (e.bf16) {
        if (o.bf16) grad_entry_scale<1, 1, NT>(g, e, o, a, b, coef);
        else grad_entry_scale<1, 0, NT>(g, e, o, a, b, coef);
    } else {
        if (o.bf16) grad_entry_scale<0, 1, NT>(g, e, o, a, b, coef);
        else grad_entry_scale<0, 0, NT>(g, e, o, a, b, coef);
    }
}

// A norm that is not finite (a gradient that is not) clips nothing: the
// caller sees it in *norm and skips the step.
__device__ __forceinline__ float clip_coef(double norm, float max_norm) {
    return (norm > max_norm && norm < __builtin_inf()) ? static_cast<float>(max_norm / norm) : 1.f;
}

template <int NT>
__global__ __launch_bounds__(kGradThreads) void grad_sumsq_kernel(const GradEntry *__restrict__ t, int n,
                                                                  int64_t chunks, double *__restrict__ partials) {
    __shared__ double lds[kGradThreads / 64];
    const int64_t g = blockIdx.x, G = gridDim.x;
    const GradGroup group{static_cast<int>(threadIdx.x), kGradThreads};
    double sum = 0.0;
    grad_entries(t, n, chunks * g / G, chunks * (g + 1) / G, [&](const GradEntry &e, int, int64_t a, int64_t b) {
        sum = grad_entry_sumsq<NT>(group, e, a, b, sum);
    });
    const double s = block_sum(sum, lds);
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

template <int NT>
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
    const GradGroup group{static_cast<int>(threadIdx.x), kGradThreads};
    grad_entries(t, n, chunks * g / G, chunks * (g + 1) / G, [&](const GradEntry &e, int i, int64_t a, int64_t b) {
        grad_entry_scale_any<NT>(group, e, to[i], a, b, coef);
    });
}

// All of it by one workgroup, a chunk per wave at a time (at most 64 tensors:
// each lane looks at one entry to find the chunk's); to and coef_out null: the
// norm alone.
__global__ __launch_bounds__(kGradSmallThreads) void grad_small_kernel(const GradEntry *__restrict__ t,
                                                                       const GradEntry *__restrict__ to, int n,
                                                                       int chunks, float max_norm, int in_place,
                                                                       float *__restrict__ norm,
                                                                       float *__restrict__ coef_out) {
    __shared__ double lds[kGradSmallThreads / 64];
    const int lane = threadIdx.x & 63;
    const GradGroup group{lane, 64};
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t end = lane < n ? t[lane].first + t[lane].chunks : chunks;
    auto each = [&](auto f) {
        for (int c = wave; c < chunks; c += kGradSmallThreads / 64) {
            const int i = __builtin_ctzll(__ballot(end > c));
            const GradEntry e = t[i];
            f(e, i, c - e.first);
        }
    };
    double sum = 0.0;
    each([&](const GradEntry &e, int, int64_t c) { sum = grad_entry_sumsq<0>(group, e, c, c + 1, sum); });
    const double s = sqrt(block_sum(sum, lds));
    const float coef = clip_coef(s, max_norm);
    if (threadIdx.x == 0) {
        *norm = static_cast<float>(s);
        if (coef_out) *coef_out = coef;
    }
    if (!to || (in_place && coef == 1.f)) return;
    each([&](const GradEntry &e, int i, int64_t c) { grad_entry_scale_any<0>(group, e, to[i], c, c + 1, coef); });
}

// As many chunks for every workgroup, but for the last ones.
static int grad_workgroups(int64_t chunks) {
    if (chunks < 1) return 1;
    const int64_t each = (chunks + kGradMaxWGs - 1) / kGradMaxWGs;
    return static_cast<int>((chunks + each - 1) / each);
}

static bool grad_small(int n, int64_t chunks, int64_t elements) {
    return n <= 64 && chunks <= kGradSmallChunks && elements <= kGradSmallElements;
}

size_t grad_workspace(int n, int64_t chunks, int64_t elements) {
    return grad_small(n, chunks, elements) ? 0 : static_cast<size_t>(grad_workgroups(chunks)) * sizeof(double);
}

hipError_t launch_grad_norm(const GradEntry *t, int n, int64_t chunks, int64_t elements, double *partials,
                            float *norm, hipStream_t st) {
    if (grad_small(n, chunks, elements)) {
        hipLaunchKernelGGL(grad_small_kernel, dim3(1), dim3(kGradSmallThreads), 0, st, t, nullptr, n,
                           static_cast<int>(chunks), 0.f, 0,
                           norm, nullptr);
        return hipGetLastError();
    }
    const int g = grad_workgroups(chunks);
    hipLaunchKernelGGL(elements > kGradStream ? grad_sumsq_kernel<1> : grad_sumsq_kernel<0>, dim3(g),
                       dim3(kGradThreads), 0, st, t, n, chunks, partials);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradThreads), 0, st, partials, g, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradEntry *t, const GradEntry *to, int n, int64_t chunks, int64_t elements,
                            float max_norm, double *partials, float *norm, float *coef, hipStream_t st) {
    const int in_place = t == to ? 1 : 0;
    if (grad_small(n, chunks, elements)) {
        hipLaunchKernelGGL(grad_small_kernel, dim3(1), dim3(kGradSmallThreads), 0, st, t, to, n,
                           static_cast<int>(chunks), max_norm, in_place, norm, coef);
        return hipGetLastError();
    }
    const int g = grad_workgroups(chunks);
    const bool stream = elements > kGradStream;
    hipLaunchKernelGGL(stream ? grad_sumsq_kernel<1> : grad_sumsq_kernel<0>, dim3(g), dim3(kGradThreads), 0, st, t, n,
                       chunks, partials);
    hipLaunchKernelGGL(stream ? grad_scale_kernel<1> : grad_scale_kernel<0>, dim3(stream ? 4 * g : g),
                       dim3(kGradThreads), 0, st, t, to, n, chunks, partials, g, max_norm, in_place, norm, coef);
    return hipGetLastError();
}

}  // namespace logra
