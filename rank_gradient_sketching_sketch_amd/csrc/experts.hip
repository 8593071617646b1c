// Rows sorted by expert and back: what stands between a token's activations
// and the experts' projections (whose sketches are in sketch_experts.hip).
//
// Pair p = t K + j is token t's j-th choice of expert, ids[t][j]; choices
// outside 0 .. E-1 are dropped. The pairs sorted by expert (pairs of one
// expert in their own order) have places 0 .. N_kept - 1:
//   offsets[e] .. offsets[e + 1]  the places of expert e's pairs
//   order[place] = p              (-1 behind the last)
//   slots[p] = place              (-1 for a dropped pair)
// and with optional weights w[t][j] (absent: 1)
//   gather            Xs[slots[t][j]] = w[t][j] X[t]
//   combine           Y[t] = sum_j w[t][j] Ys[slots[t][j]]
//   combine backward  dYs[slots[t][j]] = w[t][j] dY[t],  dw[t][j] = <dY[t], Ys[slots[t][j]]>.
// The gradient of gather is combine, with the same weights.
//
// All of them are bound by memory. The row kernels give each token a
// workgroup, so that a token's own row crosses the memory bus once however
// many experts it goes to. Rows of Xs and dYs that no pair maps to are not
// written. 4096 tokens, 8 of 128 experts, bf16 rows of 2048: gather 27 us
// (147 MB, 5.4 TB/s), combine 25.5 us (151 MB, 5.9 TB/s), combine backward 55 us
// (277 MB, 5.0 TB/s); a copy of 1 GiB reaches 5.2 TB/s on this card.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace logra {

// ------------------------------------------------------------------- sort --
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
// Up to kSortSelf pairs the sort is one launch: every workgroup counts all
// pairs itself and places its own kSortChunk of them. Above that a launch of
// counts goes first, whose sums the workgroups then add up. (128 experts: 4096
// pairs 5.6 us in one launch, 4160 pairs 4.7 us and 2.4 us for the counts in
// two; 32768 pairs 17.5 us in one, 6.0 us and 2.7 to 4 us in two.)
constexpr int kSortSelf = 4096, kSortChunk = 1024;
constexpr int kSortMaxBlocks = 256;

struct SortPlan {
    int blocks = 1;
    int chunk = 0;     // pairs per workgroup, a multiple of 1024
};

static SortPlan plan_sort(int64_t n) {
    SortPlan p;
    const int64_t c = n <= kSortSelf ? 1 : (n + kSortMaxBlocks - 1) / kSortMaxBlocks;
    p.chunk = static_cast<int>((c + kSortChunk - 1) / kSortChunk * kSortChunk);
    if (n > p.chunk) p.blocks = static_cast<int>((n + p.chunk - 1) / p.chunk);
    return p;
}

struct SortIds {
    const void *ids;
    int64_t ld;
    int K, E, wide;
    // expert of pair p, E for a dropped one
    __device__ __forceinline__ int operator()(int64_t p) const {
        int64_t at = p;
        if (ld != K) {
            const uint32_t t = static_cast<uint32_t>(p) / static_cast<uint32_t>(K);
            at = t * ld + (static_cast<uint32_t>(p) - t * static_cast<uint32_t>(K));
        }
        const int64_t id = wide ? reinterpret_cast<const int64_t *>(ids)[at]
                                : static_cast<int64_t>(reinterpret_cast<const int32_t *>(ids)[at]);
        return id >= 0 && id < E ? static_cast<int>(id) : E;
    }
};

// hist[block][e]: the pairs of expert e in the block's chunk.
__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(SortIds ids, int64_t n, int chunk,
                                                                 int32_t *__restrict__ hist) {
    __shared__ int cnt[kMaxExperts];
    const int E = ids.E;
    for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int64_t p1 = min(n, p0 + chunk);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kSortThreads) {
        const int e = ids(p);
        if (e < E) atomicAdd(&cnt[e], 1);   // whole numbers: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[static_cast<int64_t>(blockIdx.x) * E + e] = cnt[e];
}

// Lanes of the wave that hold the same value (bits of it compared).
__device__ __forceinline__ uint64_t match_lanes(int v, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t s = __ballot((v >> b) & 1);
        m &= ((v >> b) & 1) ? s : ~s;
    }
    return m;
}

// Places of one chunk's pairs. Each wave takes a contiguous part of the
// chunk in groups of 64 and keeps its own counter per expert in LDS, so the
// pairs of an expert keep their order: within a group the place follows from
// the lanes before it that hold the same expert.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortIds ids, int64_t n, int chunk, int bits,
                                                                    const int32_t *__restrict__ hist,
                                                                    int32_t *__restrict__ offsets,
                                                                    int32_t *__restrict__ order,
                                                                    int32_t *__restrict__ slots) {
    extern __shared__ int lds[];
    const int E = ids.E;
    int *cnt = lds;                              // [kSortWaves][E]
    int *total = lds + kSortWaves * E;           // [E] pairs of the expert, then its first place
    int *before = total + E;                     // [E] pairs of the expert in the chunks before this one
    __shared__ int wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int per_wave = chunk / kSortWaves;     // a multiple of 64
    const int64_t w0 = p0 + static_cast<int64_t>(wave) * per_wave;
    int *mine = cnt + wave * E;

    // what the counts need is requested before the counters are cleared: the
    // first group's experts (kept for the second pass over them), and the
    // pairs of the other chunks, as counts or, kOther at most, one by one
    constexpr int kOther = kSortSelf / kSortThreads;
    const int e_first = w0 + lane < n ? ids(w0 + lane) : E;
    const int parts = max(1, kSortThreads / E), part = tid / E, e_part = tid - part * E;
    int t = 0, b = 0, other[kOther];
    if (hist) {
        if (part < parts)
            for (int q = part; q < static_cast<int>(gridDim.x); q += parts) {
                const int h = hist[static_cast<int64_t>(q) * E + e_part];
                t += h;
                b += q < static_cast<int>(blockIdx.x) ? h : 0;
            }
    } else {
#pragma unroll
        for (int i = 0; i < kOther; ++i) {
            const int64_t p = tid + i * kSortThreads;
            other[i] = p < n && (p < p0 || p >= p0 + chunk) ? ids(p) : E;
        }
    }
    for (int i = tid; i < (kSortWaves + 2) * E; i += kSortThreads) lds[i] = 0;
    __syncthreads();
    for (int64_t g = w0; g < w0 + per_wave && g < n; g += 64) {
        const int e = g == w0 ? e_first : g + lane < n ? ids(g + lane) : E;
        if (e < E) atomicAdd(&mine[e], 1);
    }
    if (hist) {
        if (part < parts) {
            atomicAdd(&total[e_part], t);
            atomicAdd(&before[e_part], b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kOther; ++i)
            if (other[i] < E) atomicAdd(&(tid + i * kSortThreads < p0 ? before : total)[other[i]], 1);
        __syncthreads();
        for (int e = tid; e < E; e += kSortThreads) {
            int sum = total[e] + before[e];
            for (int w = 0; w < kSortWaves; ++w) sum += cnt[w * E + e];
            total[e] = sum;
        }
    }
    __syncthreads();

    // first place of every expert: exclusive sums of the totals (E <= 1024,
    // one expert per thread)
    const int own = tid < E ? total[tid] : 0;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int carry = 0, kept = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) carry += wave_sum[w];
        kept += wave_sum[w];
    }
    if (tid < E) {
        const int first = carry + incl - own;
        int at = first + before[tid];
        int c[kSortWaves];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) c[w] = cnt[w * E + tid];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            cnt[w * E + tid] = at;
            at += c[w];
        }
        if (blockIdx.x == 0) offsets[tid] = first;
    }
    if (blockIdx.x == 0 && tid == 0) offsets[E] = kept;
    __syncthreads();

    for (int64_t g = w0; g < w0 + per_wave && g < n; g += 64) {
        const int64_t p = g + lane;
        const int e = g == w0 ? e_first : p < n ? ids(p) : E;
        const uint64_t same = match_lanes(e, bits);
        const int rank = __popcll(same & ((1ull << lane) - 1ull));
        int at = 0;
        if (e < E) at = mine[e] + rank;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
        if (e < E && rank == 0) mine[e] += __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
        if (p < n) {
            slots[p] = e < E ? at : -1;
            if (e < E) order[at] = static_cast<int32_t>(p);
        }
    }
    // no pair has the places behind the last kept one
    for (int64_t s = kept + static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; s < n;
         s += static_cast<int64_t>(gridDim.x) * kSortThreads)
        order[s] = -1;
}

size_t expert_sort_workspace(int64_t n, int E) {
    const SortPlan p = plan_sort(n);
    return n > kSortSelf ? static_cast<size_t>(p.blocks) * E * 4 : 0;
}

hipError_t launch_expert_sort(int64_t T, int K, int E, const void *ids, int id_bytes, int64_t ld_ids,
                              int32_t *offsets, int32_t *order, int32_t *slots, void *ws, hipStream_t st) {
    const int64_t n = T * K;
    const SortPlan p = plan_sort(n);
    const SortIds s{ids, ld_ids, K, E, id_bytes == 8 ? 1 : 0};
    int bits = 1;
    while ((1 << bits) <= E) ++bits;      // values 0 .. E
    int32_t *hist = n > kSortSelf ? static_cast<int32_t *>(ws) : nullptr;
    if (hist) hipLaunchKernelGGL(sort_hist_kernel, dim3(p.blocks), dim3(kSortThreads), 0, st, s, n, p.chunk, hist);
    hipLaunchKernelGGL(sort_scatter_kernel, dim3(p.blocks), dim3(kSortThreads), (kSortWaves + 2) * E * 4, st, s, n,
                       p.chunk, bits, hist, offsets, order, slots);
    return hipGetLastError();
}

// ------------------------------------------------------------------- rows --
constexpr int kRowThreads = 256;

typedef u32x4_t u32x4_e2_t __attribute__((aligned(2)));   // rows need only their element's alignment
typedef u32x4_t u32x4_e4_t __attribute__((aligned(4)));

// A row element type: bf16 (8 to a 16-byte access) or fp32 (4).
template <int BF16>
struct RowOf {
    static constexpr int V = BF16 ? 8 : 4;
    using Elem = std::conditional_t<BF16 != 0, uint16_t, uint32_t>;
    using Vec = std::conditional_t<BF16 != 0, u32x4_e2_t, u32x4_e4_t>;
    template <int NT = 0>
    static __device__ __forceinline__ u32x4_t load(const char *p) {
        const Vec *src = reinterpret_cast<const Vec *>(p);
        return NT ? __builtin_nontemporal_load(src) : *src;
    }
    template <int NT>
    static __device__ __forceinline__ void store(char *p, u32x4_t v) {
        Vec *dst = reinterpret_cast<Vec *>(p);
        if (NT) __builtin_nontemporal_store(v, dst);
        else *dst = v;
    }
    static __device__ __forceinline__ void unpack(u32x4_t w, float (&v)[V]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (BF16) {
                v[2 * e % V] = bf16_lo(w[e]);
                v[(2 * e + 1) % V] = bf16_hi(w[e]);
            } else {
                v[e] = __uint_as_float(w[e]);
            }
        }
    }
    static __device__ __forceinline__ u32x4_t pack(const float (&v)[V]) {
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = BF16 ? pack_bf16x2(v[2 * e % V], v[(2 * e + 1) % V]) : __float_as_uint(v[e]);
        return w;
    }
    static __device__ __forceinline__ float get(const char *p) {
        const uint32_t w = *reinterpret_cast<const Elem *>(p);
        return __uint_as_float(BF16 ? w << 16 : w);
    }
    static __device__ __forceinline__ void put(char *p, float v) {
        *reinterpret_cast<Elem *>(p) = static_cast<Elem>(BF16 ? pack_bf16x2(v, 0.f) : __float_as_uint(v));
    }
};

// Rows go through in pieces of V elements. The last piece of a row whose
// length is no multiple of V starts where it ends with the row: it overlaps
// the one before (whose elements get the same values twice), and no element
// needs an access of its own. Only rows shorter than V are done element by
// element.

// Without weights the rows' bits are copied.
template <int BF16, int NT>
__global__ __launch_bounds__(kRowThreads) void expert_gather_kernel(int K, int h, const char *__restrict__ X,
                                                                    int64_t ldx, const int32_t *__restrict__ slots,
                                                                    const float *__restrict__ w,
                                                                    char *__restrict__ Xs, int64_t ldxs,
                                                                    int64_t n_rows) {
    using R = RowOf<BF16>;
    constexpr int V = R::V, B = BF16 ? 2 : 4;
    const int64_t t = blockIdx.x;
    const int32_t *slot = slots + t * K;
    auto each = [&](int c, auto f) {
        for (int j = 0; j < K; ++j) {
            const int64_t s = slot[j];
            if (s >= 0 && s < n_rows) f(Xs + (s * ldxs + c) * B, j);
        }
    };
    if (h < V) {
        const int c = threadIdx.x;
        if (c >= h) return;
        const char *src = X + (t * ldx + c) * B;
        if (w) {
            const float x = R::get(src);
            each(c, [&](char *dst, int j) { R::put(dst, w[t * K + j] * x); });
        } else {
            const typename R::Elem x = *reinterpret_cast<const typename R::Elem *>(src);
            each(c, [&](char *dst, int) { *reinterpret_cast<typename R::Elem *>(dst) = x; });
        }
        return;
    }
    for (int c0 = threadIdx.x * V; c0 < h; c0 += kRowThreads * V) {
        const int c = min(c0, h - V);
        const u32x4_t bits = R::load(X + (t * ldx + c) * B);
        if (w) {
            float x[V];
            R::unpack(bits, x);
            each(c, [&](char *dst, int j) {
                const float f = w[t * K + j];
                float y[V];
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = f * x[e];
                R::template store<NT>(dst, R::pack(y));
            });
        } else {
            each(c, [&](char *dst, int) { R::template store<NT>(dst, bits); });
        }
    }
}

// Choices of a token whose rows a thread has in flight. bf16 rows of 2048, 8
// pairs per token, us with 1 / 2 / 4: combine 1 token 3.6 / 3.1 / 2.9, 512
// tokens 6.5 / 5.9 / 5.8; its gradient 1 token 8.1 / 6.2 / 5.6, 512 tokens 12.4 /
// 10.1 / 10.1, 4096 tokens 55.7 / 56.1 / 58.2.
constexpr int kRowsAhead = 2;

template <int BF16, int NT>
__global__ __launch_bounds__(kRowThreads) void expert_combine_kernel(int K, int h, const char *__restrict__ Ys,
                                                                     int64_t ldys, int64_t n_rows,
                                                                     const int32_t *__restrict__ slots,
                                                                     const float *__restrict__ w,
                                                                     char *__restrict__ Y, int64_t ldy) {
    using R = RowOf<BF16>;
    constexpr int V = R::V, B = BF16 ? 2 : 4;
    const int64_t t = blockIdx.x;
    if (h < V) {
        const int c = threadIdx.x;
        if (c >= h) return;
        float y = 0.f;
        for (int j = 0; j < K; ++j) {
            const int64_t s = slots[t * K + j];
            if (s >= 0 && s < n_rows) y = fmaf(w ? w[t * K + j] : 1.f, R::get(Ys + (s * ldys + c) * B), y);
        }
        R::put(Y + (t * ldy + c) * B, y);
        return;
    }
    for (int c0 = threadIdx.x * V; c0 < h; c0 += kRowThreads * V) {
        const int c = min(c0, h - V);
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = 0.f;
        for (int j0 = 0; j0 < K; j0 += kRowsAhead) {
            u32x4_t x[kRowsAhead];
            int64_t s[kRowsAhead];
#pragma unroll
            for (int q = 0; q < kRowsAhead; ++q) {
                s[q] = j0 + q < K ? slots[t * K + j0 + q] : -1;
                if (s[q] >= n_rows) s[q] = -1;
                if (s[q] >= 0) x[q] = R::template load<NT>(Ys + (s[q] * ldys + c) * B);
            }
#pragma unroll
            for (int q = 0; q < kRowsAhead; ++q) {
                if (s[q] < 0) continue;
                float v[V];
                R::unpack(x[q], v);
                const float f = w ? w[t * K + j0 + q] : 1.f;
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = fmaf(f, v[e], y[e]);
            }
        }
        R::template store<NT>(Y + (t * ldy + c) * B, R::pack(y));
    }
}

template <int BF16, int NT>
__global__ __launch_bounds__(kRowThreads) void expert_combine_backward_kernel(
    int K, int h, const char *__restrict__ dY, int64_t lddy, const char *__restrict__ Ys, int64_t ldys,
    const int32_t *__restrict__ slots, const float *__restrict__ w, char *__restrict__ dYs, int64_t lddys,
    int64_t n_rows, float *__restrict__ dw) {
    using R = RowOf<BF16>;
    constexpr int V = R::V, B = BF16 ? 2 : 4, kWaves = kRowThreads / 64;
    __shared__ float part[2][kRowsAhead][kWaves];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < K; j0 += kRowsAhead) {
        float dot[kRowsAhead];
        int64_t s[kRowsAhead];
#pragma unroll
        for (int q = 0; q < kRowsAhead; ++q) {
            dot[q] = 0.f;
            s[q] = j0 + q < K ? slots[t * K + j0 + q] : -1;
            if (s[q] >= n_rows) s[q] = -1;
        }
        if (h < V) {
            const int c = threadIdx.x;
#pragma unroll
            for (int q = 0; q < kRowsAhead; ++q)
                if (s[q] >= 0 && c < h) {
                    const float g = R::get(dY + (t * lddy + c) * B);
                    dot[q] = g * R::get(Ys + (s[q] * ldys + c) * B);
                    R::put(dYs + (s[q] * lddys + c) * B, w[t * K + j0 + q] * g);
                }
        } else {
            for (int c0 = threadIdx.x * V; c0 < h; c0 += kRowThreads * V) {
                const int c = min(c0, h - V), seen = c0 - c;      // the piece's elements that the one before has
                u32x4_t y[kRowsAhead];
                const u32x4_t g_bits = R::load(dY + (t * lddy + c) * B);
#pragma unroll
                for (int q = 0; q < kRowsAhead; ++q)
                    if (s[q] >= 0) y[q] = R::template load<NT>(Ys + (s[q] * ldys + c) * B);
                float g[V];
                R::unpack(g_bits, g);
#pragma unroll
                for (int q = 0; q < kRowsAhead; ++q) {
                    if (s[q] < 0) continue;
                    float v[V], out[V];
                    R::unpack(y[q], v);
                    const float f = w[t * K + j0 + q];
                    if (seen == 0) {
#pragma unroll
                        for (int e = 0; e < V; ++e) dot[q] = fmaf(g[e], v[e], dot[q]);
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) dot[q] = e < seen ? dot[q] : fmaf(g[e], v[e], dot[q]);
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) out[e] = f * g[e];
                    R::template store<NT>(dYs + (s[q] * lddys + c) * B, R::pack(out));
                }
            }
        }
        // two buffers in turn: a group's sums are read while the next one's are written
        float(*mine)[kWaves] = part[(j0 / kRowsAhead) & 1];
#pragma unroll
        for (int q = 0; q < kRowsAhead; ++q) {
            if (j0 + q >= K) break;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) dot[q] += __shfl_xor(dot[q], o);
            if (lane == 0) mine[q][wave] = dot[q];
        }
        __syncthreads();
        if (threadIdx.x < kRowsAhead && j0 + threadIdx.x < K) {
            float d = 0.f;
            for (int i = 0; i < kWaves; ++i) d += mine[threadIdx.x][i];
            dw[t * K + j0 + threadIdx.x] = d;
        }
    }
}

// Above this many bytes of sorted rows the kernels read and write them past
// the caches (the last-level one holds 256 MB, and what a step does between
// two uses of the same rows is more than that). bf16 rows of 2048, 8 pairs per
// token, us without / with: rows not in the caches, 4096 tokens (134 MB)
// gather 30.4 / 25.8, combine 33.5 / 25.9, its gradient 59.0 / 55.7; 2500
// tokens (82 MB) 16.6 / 16.9, 20.5 / 18.9, 43.0 / 41.5; the same buffers again
// and again, 4096 tokens 23.4 / 25.1, 23.4 / 24.7, 50.2 / 54.3, 2500 tokens 15.5
// / 16.0, 16.2 / 18.6, 31.9 / 40.0. A token's own row in the backward kernel is
// read topk times and stays cached.
constexpr int64_t kRowStreamBytes = 96ll << 20;
static bool stream_rows(int64_t pairs, int64_t h, int elem) { return pairs * h * elem > kRowStreamBytes; }

hipError_t launch_expert_gather(int64_t T, int K, int64_t h, int elem, const void *X, int64_t ldx,
                                const int32_t *slots, const float *w, void *Xs, int64_t ldxs, int64_t n_rows,
                                hipStream_t st) {
    const bool nt = stream_rows(T * K, h, elem);
    auto kernel = elem == 2 ? (nt ? expert_gather_kernel<1, 1> : expert_gather_kernel<1, 0>)
                            : (nt ? expert_gather_kernel<0, 1> : expert_gather_kernel<0, 0>);
    hipLaunchKernelGGL(kernel, dim3(T), dim3(kRowThreads), 0, st, K, static_cast<int>(h),
                       static_cast<const char *>(X), ldx, slots, w, static_cast<char *>(Xs), ldxs, n_rows);
    return hipGetLastError();
}

hipError_t launch_expert_combine(int64_t T, int K, int64_t h, int elem, const void *Ys, int64_t ldys,
                                 int64_t n_rows, const int32_t *slots, const float *w, void *Y, int64_t ldy,
                                 hipStream_t st) {
    const bool nt = stream_rows(T * K, h, elem);
    auto kernel = elem == 2 ? (nt ? expert_combine_kernel<1, 1> : expert_combine_kernel<1, 0>)
                            : (nt ? expert_combine_kernel<0, 1> : expert_combine_kernel<0, 0>);
    hipLaunchKernelGGL(kernel, dim3(T), dim3(kRowThreads), 0, st, K, static_cast<int>(h),
                       static_cast<const char *>(Ys), ldys, n_rows, slots, w, static_cast<char *>(Y), ldy);
    return hipGetLastError();
}

hipError_t launch_expert_combine_backward(int64_t T, int K, int64_t h, int elem, const void *dY, int64_t lddy,
                                          const void *Ys, int64_t ldys, const int32_t *slots, const float *w,
                                          void *dYs, int64_t lddys, int64_t n_rows, float *dw, hipStream_t st) {
    const bool nt = stream_rows(T * K, h, elem);
    auto kernel = elem == 2 ? (nt ? expert_combine_backward_kernel<1, 1> : expert_combine_backward_kernel<1, 0>)
                            : (nt ? expert_combine_backward_kernel<0, 1> : expert_combine_backward_kernel<0, 0>);
    hipLaunchKernelGGL(kernel, dim3(T), dim3(kRowThreads), 0, st, K, static_cast<int>(h),
                       static_cast<const char *>(dY), lddy, static_cast<const char *>(Ys), ldys, slots, w,
                       static_cast<char *>(dYs), lddys, n_rows, dw);
    return hipGetLastError();
}

}  // namespace logra
