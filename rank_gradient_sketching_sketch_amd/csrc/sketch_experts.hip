// The sketch over the experts of a layer, S_e (+)= dY_e^T (X_e A_e^T) for
// every expert e, in one call.
//
// An expert layer has one projection per expert and each sees its own
// tokens: rows offsets[e] .. offsets[e + 1] of dY (sorted by expert), and of
// X either the same rows or, through the sort's order, row order[i] / topk of
// the unsorted activations (then the sorted copy of X need not exist). The
// sketch of each is the one of sketch_bf16.hip with its own sign matrix A_e,
// two products:
//   P_e = c X_e Sigma_e^T   (rows x r, contraction over k),
//   S_e (+)= dY_e^T P_e     (d x r, contraction over the expert's rows).
// The row counts live on the device, so the grids cover the most that any
// counts could need and each workgroup finds its expert from the offsets.
//
// P is kept as two bf16 terms, P = hi + lo with hi = bf16(P) and
// lo = bf16(P - hi): their sum is off by 2^-16 of P at most (each rounding is
// 2^-8 of what it rounds), so S has nearly the precision of fp32 products
// although dY^T P runs on the bf16 matrix cores (dY is bf16 exactly). One bf16
// term alone would leave 2^-8.
#include "common.hpp"
#include "launch.hpp"
#include "signs.hpp"

namespace logra {

constexpr int kEsTokens = 32;          // rows of a block of P

// Expert e's rows in the sorted arrays, bounds brought into 0 .. N in case
// they are not.
struct EsRange {
    int begin, count;
};
__device__ __forceinline__ EsRange es_range(const int32_t *offsets, int e, int N) {
    const int a = min(max(offsets[e], 0), N), b = min(max(offsets[e + 1], 0), N);
    return EsRange{a, max(0, b - a)};
}

// What every wave works out from the offsets: the expert that holds unit u
// when expert e holds units(count_e) consecutive ones, and the sums before it.
struct EsPlace {
    int expert, index;      // expert -1: no expert holds u; index: the unit's number within it
    int blocks, extras;     // blocks of P and partial sketches of the experts before
};

__device__ __forceinline__ int es_items(int count, int chunk) { return count > chunk ? (count + chunk - 1) / chunk : 1; }

// by_items: units are items (es_items), else 32-row blocks of P. All lanes
// of the wave call it.
__device__ __forceinline__ EsPlace es_find(const int32_t *offsets, int E, int N, int chunk, int u, bool by_items) {
    const int lane = threadIdx.x & 63;
    int before_u = 0, before_b = 0, before_x = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        int nb = 0, nx = 0, nu = 0;
        if (e < E) {
            const int count = es_range(offsets, e, N).count;
            nb = (count + kEsTokens - 1) / kEsTokens;
            nx = es_items(count, chunk) - 1;
            nu = by_items ? nx + 1 : nb;
        }
        int iu = nu, ib = nb, ix = nx;       // inclusive sums over the lanes
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int a = __shfl_up(iu, o), b = __shfl_up(ib, o), c = __shfl_up(ix, o);
            if (lane >= o) {
                iu += a;
                ib += b;
                ix += c;
            }
        }
        const uint64_t past = __ballot(before_u + iu > u);
        if (past) {
            const int l = __builtin_ctzll(past);
            EsPlace p;
            p.expert = e0 + l;
            p.index = u - (before_u + __shfl(iu - nu, l));
            p.blocks = before_b + __shfl(ib - nb, l);
            p.extras = before_x + __shfl(ix - nx, l);
            return p;
        }
        before_u += __shfl(iu, 63);
        before_b += __shfl(ib, 63);
        before_x += __shfl(ix, 63);
    }
    return EsPlace{-1, 0, 0, 0};
}

__device__ __forceinline__ uint64_t es_key(const ExpertSketchArgs &a, int e) {
    const uint64_t id = a.first_id + static_cast<uint64_t>(e) * a.id_stride;
    return splitmix_finalize((a.prefix ^ id) + kGolden);
}

// The row of X that sorted row i reads; -1 where there is none.
__device__ __forceinline__ int64_t es_x_row(const ExpertSketchArgs &a, int i) {
    int64_t row = i;
    if (a.order) {
        const int p = a.order[i];
        row = p < 0 ? -1 : p / a.topk;
    }
    return row < a.x_rows ? row : -1;
}

// ---------------------------------------------------------- bf16, stage 1 --
// A workgroup owns one 32-row block of P and 128 (or r) columns over the
// whole of k; its eight waves split the k range and add their tiles through
// LDS in wave order, as stage 1 of the one-matrix sketch does.
constexpr int kEsWaves = 8, kEsWords = 8;

template <int R>
__global__ __launch_bounds__(512) void es_project_kernel(ExpertSketchArgs a, int chunk, int K,
                                                         uint16_t *__restrict__ P) {
    constexpr int RT = R < 128 ? R : 128, NB = RT / 16, MB = 2;
    constexpr int kTileLd = kEsTokens + 4;
    constexpr int kTable = kEsWaves * kEsWords * RT * 8, kTiles = kEsWaves * RT * kTileLd * 4;
    __shared__ __attribute__((aligned(16))) char smem[kTable > kTiles ? kTable : kTiles];
    uint64_t *table = reinterpret_cast<uint64_t *>(smem);
    float *tile = reinterpret_cast<float *>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int l0 = blockIdx.y * RT;
    const EsPlace at = es_find(a.offsets, a.E, static_cast<int>(a.N), chunk, blockIdx.x, false);
    if (at.expert < 0) return;
    const EsRange rows = es_range(a.offsets, at.expert, static_cast<int>(a.N));
    const int n = min(kEsTokens, rows.count - at.index * kEsTokens);       // rows of this block
    const uint64_t key = es_key(a, at.expert);

    const uint16_t *xrow[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int i = 16 * mb + i16;
        const int64_t r = i < n ? es_x_row(a, rows.begin + at.index * kEsTokens + i) : -1;
        xrow[mb] = r < 0 ? nullptr : static_cast<const uint16_t *>(a.X) + r * a.ldx;
    }
    const int nkb = (K + 63) >> 6;
    const int bpw = (nkb + kEsWaves - 1) / kEsWaves;
    const int kb0 = min(nkb, wave * bpw), kb1 = min(nkb, kb0 + bpw);
    const int s_begin = 2 * kb0, s_end = min((K + 31) >> 5, 2 * kb1);
    auto xload = [&](int s, int mb) -> u32x4_t {
        const int k = 32 * s + 8 * g;
        return xrow[mb] && s < s_end && k < K ? load_u32x4(xrow[mb] + k) : zero_u32x4();
    };
    uint64_t *wt = table + wave * (kEsWords * RT);
    auto refill = [&](int first) {
        for (int idx = lane; idx < kEsWords * RT; idx += 64) {
            const int bb = idx / RT, col = idx - bb * RT;
            const int b = first + bb;
            wt[idx] = b < kb1 ? sign_word(key, static_cast<uint32_t>(l0 + col), static_cast<uint32_t>(b)) : 0ull;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    };
    f32x4_t acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = zero_f32x4();
    const uint32_t one_pair = opaque_u32(0x3F803F80u);
    u32x4_t xa[MB], xn[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) xa[mb] = xload(s_begin, mb);
    int first = kb0;
    if (s_begin < s_end) refill(first);
    for (int s = s_begin; s < s_end; ++s) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) xn[mb] = xload(s + 1, mb);
        const int b = s >> 1;
        if (b >= first + kEsWords) {
            first += kEsWords;
            refill(first);
        }
        const uint64_t *wrow = wt + (b - first) * RT + i16;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint64_t w = wrow[16 * nb];
            const uint32_t dw = (s & 1) ? static_cast<uint32_t>(w >> 32) : static_cast<uint32_t>(w);
            const u32x4_t bf = signs8_to_bf16(__builtin_amdgcn_ubfe(dw, 8 * g, 8), one_pair);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) acc[mb][nb] = mfma_bf16(xa[mb], bf, acc[mb][nb]);
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) xa[mb] = xn[mb];
    }
    __syncthreads();      // every wave is done with its word table
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            *reinterpret_cast<f32x4_t *>(&tile[(wave * RT + 16 * nb + i16) * kTileLd + 16 * mb + 4 * g]) = acc[mb][nb];
    __syncthreads();
    // eight rows of one column per thread: 16 bytes of each term
    for (int q = tid; q < RT * 4; q += 512) {
        const int col = q >> 2, t = 8 * (q & 3);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kEsWaves; ++w) {
            const float *src = &tile[(w * RT + col) * kTileLd + t];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += src[e];
        }
        u32x4_t hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = a.c * v[2 * e], y = a.c * v[2 * e + 1];
            hi[e] = pack_bf16x2(x, y);
            lo[e] = pack_bf16x2(x - bf16_lo(hi[e]), y - bf16_hi(hi[e]));
        }
        uint16_t *dst = P + (static_cast<int64_t>(blockIdx.x) * 2 * R + l0 + col) * kEsTokens + t;
        *reinterpret_cast<u32x4_t *>(dst) = hi;
        *reinterpret_cast<u32x4_t *>(dst + R * kEsTokens) = lo;
    }
}

// ---------------------------------------------------------- bf16, stage 2 --
// A workgroup owns one item (at most `chunk` rows of one expert) and kEsRows
// rows of its S, all r columns: dY is read once and S written once. Four
// waves split the columns; each step of 32 rows brings the dY tile through
// LDS (read transposed, the A operand) and P's fragments from the L2.
constexpr int kEsRows = 64;

typedef short es_i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) es_i16x4_t es_lds_i16x4_t;
__device__ __forceinline__ u32x2_t es_read_tr(const uint16_t *p) {
    const es_i16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((es_lds_i16x4_t *)p);
    return __builtin_bit_cast(u32x2_t, v);
}

template <int R>
__global__ __launch_bounds__(256) void es_fold_kernel(ExpertSketchArgs a, int chunk, int D, int64_t p_blocks,
                                                      int64_t max_extras, const uint16_t *__restrict__ P,
                                                      float *__restrict__ parts) {
    constexpr int WN = R / 16 < 4 ? R / 16 : 4;         // waves across the columns
    constexpr int WM = 4 / WN;                          // waves across the rows
    constexpr int NB = R / 16 / WN, MB = kEsRows / 16 / WM;
    constexpr int kRow = kEsRows;                       // bf16 per LDS row
    __shared__ __attribute__((aligned(16))) uint16_t lds[2][kEsTokens * kRow];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i16 = lane & 15, g = lane >> 4;
    const EsPlace at = es_find(a.offsets, a.E, static_cast<int>(a.N), chunk, blockIdx.y, true);
    if (at.expert < 0) return;
    const EsRange rows = es_range(a.offsets, at.expert, static_cast<int>(a.N));
    const int r0 = at.index * chunk;
    const int n = min(chunk, rows.count - r0);
    const int d0 = blockIdx.x * kEsRows;
    const int64_t block0 = static_cast<int64_t>(at.blocks) + r0 / kEsTokens;
    const int steps = min(static_cast<int64_t>((n + kEsTokens - 1) / kEsTokens), max(static_cast<int64_t>(0), p_blocks - block0));
    // where the tile goes: the first item of an expert to S, the others to a
    // partial sketch each, added to S by es_reduce_kernel
    float *dst = a.S + static_cast<int64_t>(at.expert) * D * R;
    bool add = a.accumulate != 0;
    if (at.index > 0) {
        const int64_t x = static_cast<int64_t>(at.extras) + at.index - 1;
        if (x >= max_extras) return;
        dst = parts + x * D * R;
        add = false;
    } else if (n <= 0 && add) {
        return;
    }

    const uint16_t *dy = static_cast<const uint16_t *>(a.dY) + (static_cast<int64_t>(rows.begin) + r0) * a.lddy;
    const int lt = tid >> 3, lc = 8 * (tid & 7);        // this thread's row and columns of a step's tile
    const bool col_ok = d0 + lc < D;
    auto gload = [&](int s) -> u32x4_t {
        const int t = kEsTokens * s + lt;
        return col_ok && t < n ? load_u32x4(dy + t * a.lddy + d0 + lc) : zero_u32x4();
    };
    const uint16_t *pb = P + block0 * 2 * R * kEsTokens;
    f32x4_t acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = zero_f32x4();
    u32x4_t next = gload(0);
    for (int s = 0; s < steps; ++s) {
        uint16_t *buf = lds[s & 1];
        *reinterpret_cast<u32x4_t *>(&buf[lt * kRow + lc]) = next;
        next = gload(s + 1);
        u32x4_t hi[NB], lo[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint16_t *src = pb + (static_cast<int64_t>(s) * 2 * R + 16 * (wn * NB + nb) + i16) * kEsTokens + 8 * g;
            hi[nb] = load_u32x4(src);
            lo[nb] = load_u32x4(src + R * kEsTokens);
        }
        __syncthreads();
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const uint16_t *p = buf + (8 * g + (i16 >> 2)) * kRow + 16 * (wm + mb * WM) + 4 * (i16 & 3);
            const u32x2_t x = es_read_tr(p), y = es_read_tr(p + 4 * kRow);
            const u32x4_t av = {x.x, x.y, y.x, y.y};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                acc[mb][nb] = mfma_bf16(av, lo[nb], acc[mb][nb]);
                acc[mb][nb] = mfma_bf16(av, hi[nb], acc[mb][nb]);
            }
        }
    }
    // lane (i16, g) of block (mb, nb): rows 4 g .. +3, column i16
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = d0 + 16 * (wm + mb * WM) + 4 * g + q;
                if (row >= D) continue;
                float *p = dst + static_cast<int64_t>(row) * R + 16 * (wn * NB + nb) + i16;
                *p = add ? *p + acc[mb][nb][q] : acc[mb][nb][q];
            }
}

// S_e += the partial sketches of expert e, in their order.
__global__ __launch_bounds__(256) void es_reduce_kernel(ExpertSketchArgs a, int chunk, int64_t size,
                                                        int64_t max_extras, const float *__restrict__ parts) {
    // expert e's partial sketches follow those of the experts before it
    const int e = blockIdx.y;
    const int own = es_items(es_range(a.offsets, e, static_cast<int>(a.N)).count, chunk) - 1;
    if (own == 0) return;
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < e; e0 += 64)
        if (e0 + lane < e) before += es_items(es_range(a.offsets, e0 + lane, static_cast<int>(a.N)).count, chunk) - 1;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    float *S = a.S + static_cast<int64_t>(e) * size;
    const float *p = parts + static_cast<int64_t>(before) * size;
    const int n = static_cast<int>(min(static_cast<int64_t>(own), max(static_cast<int64_t>(0), max_extras - before)));
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < size;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        f32x4_t v = *reinterpret_cast<const f32x4_t *>(S + i);
        for (int q = 0; q < n; ++q) v += *reinterpret_cast<const f32x4_t *>(p + q * size + i);
        *reinterpret_cast<f32x4_t *>(S + i) = v;
    }
}

// ------------------------------------------------------------------- fp32 --
// As sketch_f32.hip: fp32 FMAs over LDS tiles of 32 x 32, sums in index
// order. P is N x r, row i of the sorted rows in row i.
__global__ __launch_bounds__(256) void es_project_f32_kernel(ExpertSketchArgs a, int chunk, int K, float *__restrict__ P) {
    __shared__ float xs[32][65];
    __shared__ uint64_t words[32];
    __shared__ int64_t row_of[32];
    const int R = a.R, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const EsPlace at = es_find(a.offsets, a.E, static_cast<int>(a.N), chunk, blockIdx.x, false);
    if (at.expert < 0) return;
    const EsRange rows = es_range(a.offsets, at.expert, static_cast<int>(a.N));
    const int i0 = rows.begin + at.index * 32, n = min(32, rows.count - at.index * 32);
    const int l0 = blockIdx.y * 32, l = l0 + tx;
    const uint64_t key = es_key(a, at.expert);
    if (threadIdx.x < 32)
        row_of[threadIdx.x] = static_cast<int>(threadIdx.x) < n ? es_x_row(a, i0 + threadIdx.x) : -1;
    __syncthreads();
    const float *X = static_cast<const float *>(a.X);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < K; j0 += 64) {
        for (int e = 0; e < 8; ++e) {
            const int idx = threadIdx.x + 256 * e, t = idx >> 6, j = idx & 63;
            const int64_t row = row_of[t];
            xs[t][j] = row >= 0 && j0 + j < K ? X[row * a.ldx + j0 + j] : 0.f;
        }
        if (threadIdx.x < 32)
            words[threadIdx.x] = sign_word(key, static_cast<uint32_t>(l0 + threadIdx.x), static_cast<uint32_t>(j0 >> 6));
        __syncthreads();
        const uint64_t w = words[tx];
        const int jn = min(64, K - j0);
        for (int j = 0; j < jn; ++j) {
            const float sg = ((w >> j) & 1ull) ? -1.f : 1.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = fmaf(sg, xs[ty + 8 * q][j], acc[q]);
        }
        __syncthreads();
    }
    if (l < R)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (ty + 8 * q < n) P[static_cast<int64_t>(i0 + ty + 8 * q) * R + l] = a.c * acc[q];
}

__global__ __launch_bounds__(256) void es_fold_f32_kernel(ExpertSketchArgs a, int D, const float *__restrict__ P) {
    __shared__ float ds[32][33];
    __shared__ float ps[32][33];
    const int R = a.R, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const EsRange rows = es_range(a.offsets, blockIdx.z, static_cast<int>(a.N));
    const int d0 = blockIdx.x * 32, l0 = blockIdx.y * 32;
    const float *dY = static_cast<const float *>(a.dY);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t0 = 0; t0 < rows.count; t0 += 32) {
        for (int e = 0; e < 4; ++e) {
            const int idx = threadIdx.x + 256 * e, t = idx >> 5, c = idx & 31;
            const int64_t i = static_cast<int64_t>(rows.begin) + t0 + t;
            const bool in = t0 + t < rows.count;
            ds[t][c] = in && d0 + c < D ? dY[i * a.lddy + d0 + c] : 0.f;
            ps[t][c] = in && l0 + c < R ? P[i * R + l0 + c] : 0.f;
        }
        __syncthreads();
        const int tn = min(32, rows.count - t0);
        for (int t = 0; t < tn; ++t) {
            const float p = ps[t][tx];
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = fmaf(ds[t][ty + 8 * q], p, acc[q]);
        }
        __syncthreads();
    }
    float *S = a.S + static_cast<int64_t>(blockIdx.z) * D * R;
    if (l0 + tx < R)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = d0 + ty + 8 * q;
            if (i < D) {
                float *dst = S + static_cast<int64_t>(i) * R + l0 + tx;
                *dst = (a.accumulate ? *dst : 0.f) + acc[q];
            }
        }
}

// ------------------------------------------------------------------ plans --
ExpertSketchPlan plan_expert_sketch(int64_t N, int E, int64_t d, int64_t k, int R, int bf16) {
    ExpertSketchPlan p;
    (void)k;
    p.p_blocks = N / kEsTokens + (N < E ? N : E);
    if (!bf16) {
        p.chunk = 1 << 30;
        p.items = E;
        p.p_bytes = static_cast<size_t>(N) * R * 4;
        p.total = p.p_bytes;
        return p;
    }
    int64_t chunk = 2 * N / E;
    chunk = (chunk < 1024 ? 1024 : chunk + 31) / 32 * 32;
    p.chunk = static_cast<int>(chunk);
    p.extras = N / p.chunk;
    p.items = E + p.extras;
    p.p_bytes = static_cast<size_t>(p.p_blocks) * 2 * R * kEsTokens * 2;
    p.total = p.p_bytes + static_cast<size_t>(p.extras) * d * R * 4;
    return p;
}

template <int R>
static hipError_t expert_sketch_bf16_r(const ExpertSketchArgs &a, hipStream_t st) {
    const ExpertSketchPlan p = plan_expert_sketch(a.N, a.E, a.d, a.k, R, 1);
    uint16_t *P = static_cast<uint16_t *>(a.ws);
    float *parts = reinterpret_cast<float *>(static_cast<char *>(a.ws) + p.p_bytes);
    const int D = static_cast<int>(a.d), K = static_cast<int>(a.k);
    if (p.p_blocks > 0)
        hipLaunchKernelGGL(es_project_kernel<R>, dim3(p.p_blocks, R < 128 ? 1 : R / 128), dim3(512), 0, st, a,
                           p.chunk, K, P);
    hipLaunchKernelGGL(es_fold_kernel<R>, dim3((D + kEsRows - 1) / kEsRows, p.items), dim3(256), 0, st, a, p.chunk, D,
                       p.p_blocks, p.extras, P, parts);
    if (p.extras > 0) {
        const int64_t size = a.d * R;
        const int64_t wgs = (size + 4095) / 4096;
        hipLaunchKernelGGL(es_reduce_kernel, dim3(wgs < 64 ? wgs : 64, a.E), dim3(256), 0, st, a, p.chunk, size,
                           p.extras, parts);
    }
    return hipGetLastError();
}

hipError_t launch_expert_sketch(const ExpertSketchArgs &a, int bf16, hipStream_t st) {
    if (!bf16) {
        const ExpertSketchPlan p = plan_expert_sketch(a.N, a.E, a.d, a.k, a.R, 0);
        float *P = static_cast<float *>(a.ws);
        const unsigned lt = (a.R + 31) / 32;
        if (p.p_blocks > 0)
            hipLaunchKernelGGL(es_project_f32_kernel, dim3(p.p_blocks, lt), dim3(256), 0, st, a, p.chunk,
                               static_cast<int>(a.k), P);
        hipLaunchKernelGGL(es_fold_f32_kernel, dim3((a.d + 31) / 32, lt, a.E), dim3(256), 0, st, a,
                           static_cast<int>(a.d), P);
        return hipGetLastError();
    }
    switch (a.R) {
    case 32: return expert_sketch_bf16_r<32>(a, st);
    case 64: return expert_sketch_bf16_r<64>(a, st);
    case 128: return expert_sketch_bf16_r<128>(a, st);
    case 256: return expert_sketch_bf16_r<256>(a, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace logra
