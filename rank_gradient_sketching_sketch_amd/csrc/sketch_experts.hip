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
// P is kept in fp32 and taken apart by the second product into three bf16
// terms, P = p0 + p1 + p2 with p0 = bf16(P), p1 = bf16(P - p0),
// p2 = bf16(P - p0 - p1): each rounding is 2^-8 of what it rounds, so their
// sum is within 2^-24 of P (unless P is so small that a term is subnormal, or
// rounds to infinity in bf16) and S has the precision of fp32 products although
// dY^T P runs on the bf16 matrix cores (dY is bf16 exactly). One term would
// leave 2^-8 per product, two 2^-16. Storing the terms instead of the value
// would cost half as many bytes again on the path that bounds that product.
//
// 4096 tokens, 8 of 128 experts (uneven: 1 to 1300 rows each), d = 768,
// k = 2048, r = 256: projection 44 us, second product 55 us, partial sketches
// 6 us, 100 us in all. The bytes that cannot be left out (X, dY, S) take 32 us
// at the rate of a copy, the 73 GFLOP of the matrix instructions 61 us at the
// rate of a large library product. Of the projection, some 22 us are the loop
// over k (14 to 19 of them matrix instructions), 7 us the way to its first row
// and 2 us P's 33 MB written; with even experts it takes 35 us, the rest is
// the last units' latency. The second product takes 42 us with even experts:
// 20 us are S's 100 MB written, which comes on top of 22 us of matrix
// instructions because workgroups that start together finish together.
// That is with S overwritten; added to, it takes the call to 164 us, since
// each row of S is loaded, waited for and stored before the next one.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "fold_body.hpp"
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
// The same for an expert that all lanes of the wave name.
__device__ __forceinline__ EsRange es_range_uniform(const int32_t *offsets, int e, int N) {
    const EsRange r = es_range(offsets, e, N);
    return EsRange{__builtin_amdgcn_readfirstlane(r.begin), __builtin_amdgcn_readfirstlane(r.count)};
}

// Buffer views: loads at or past num_records return zero, so kEsOob masks
// one. (Loads under a condition instead would leave the number of requests in
// flight unknown to the compiler, which then waits for all of them.)
constexpr uint32_t kEsOob = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t es_view(const void *p, uint32_t bytes) {
    // in scalar registers whatever the compiler knows of them: a view in
    // vector registers costs a loop over the lanes at every use
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a)));
    const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32)));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000);
}
__device__ __forceinline__ u32x4_t es_load(__amdgpu_buffer_rsrc_t v, uint32_t off) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(v, off, 0, 0));
}

// A unit of the projection: up to unit_rows rows of one expert. All lanes of
// the wave work it out from the offsets: the full units of all experts come
// first, then each expert's last, shorter one, so that long ones do not start
// last.
struct EsUnit {
    int expert;             // -1: there are fewer units
    int index;              // the unit's number within its expert
    int blocks;             // 32-row blocks of P of the experts before
    int part;               // of a short unit: which of the `split` parts of its columns
    EsRange rows;           // the expert's sorted rows
};
__device__ __forceinline__ EsUnit es_unit(const int32_t *offsets, int E, int N, int u, int unit_rows, int split) {
    const int lane = threadIdx.x & 63;
    EsUnit p{-1, 0, 0, 0, {0, 0}};
    int before = 0;
    for (int pass = 0; pass < 2 && p.expert < 0; ++pass) {
        int blocks = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const EsRange r = e0 + lane < E ? es_range(offsets, e0 + lane, N) : EsRange{0, 0};
            const int count = r.count;
            const int nb = (count + kEsTokens - 1) / kEsTokens, full = count / unit_rows;
            const int nu = pass == 0 ? full : count % unit_rows ? split : 0;
            int iu = nu, ib = nb;            // inclusive sums over the lanes
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int a = __shfl_up(iu, o), b = __shfl_up(ib, o);
                if (lane >= o) {
                    iu += a;
                    ib += b;
                }
            }
            const uint64_t past = __ballot(before + iu > u);
            if (past) {
                const int l = __builtin_ctzll(past);
                p.expert = e0 + l;
                const int q = u - before - __builtin_amdgcn_readlane(iu - nu, l);
                p.index = pass == 0 ? q : __builtin_amdgcn_readlane(full, l);
                p.part = pass == 0 ? -1 : q;
                p.blocks = blocks + __builtin_amdgcn_readlane(ib - nb, l);
                p.rows = EsRange{__builtin_amdgcn_readlane(r.begin, l), __builtin_amdgcn_readlane(count, l)};
                break;
            }
            before += __builtin_amdgcn_readlane(iu, 63);
            blocks += __builtin_amdgcn_readlane(ib, 63);
        }
    }
    // the same in all lanes: kept in scalar registers
    return EsUnit{__builtin_amdgcn_readfirstlane(p.expert), __builtin_amdgcn_readfirstlane(p.index),
                  __builtin_amdgcn_readfirstlane(p.blocks), __builtin_amdgcn_readfirstlane(p.part),
                  {__builtin_amdgcn_readfirstlane(p.rows.begin), __builtin_amdgcn_readfirstlane(p.rows.count)}};
}

// The items of the second product, written by one workgroup of the
// projection's launch: at most `chunk` rows of one expert each, at least one
// per expert, in classes of falling length (the order within a class has no
// part in the results). The first item of an expert goes to S, the others to
// a partial sketch each.
struct EsItem {
    int expert;             // -1: there are fewer items
    int begin, rows;        // sorted rows
    int block;              // first block of P
    int part;               // partial sketch, -1 for S, -2 for S of an expert without partial ones
    int pad[3];
};
struct EsParts {            // the partial sketches of an expert that has some
    int expert;
    int first, count;       // count 0: there are fewer such experts
};
constexpr int kEsClasses = 16;

__device__ __forceinline__ int es_items(int count, int chunk) { return count > chunk ? (count + chunk - 1) / chunk : 1; }

__device__ __forceinline__ void es_build_items(const int32_t *offsets, int E, int N, int chunk, int max_items,
                                               EsItem *__restrict__ items, EsParts *__restrict__ experts, int *lds) {
    // lds: kMaxExperts sums of blocks, of partial sketches and of experts that
    // have some (and the sum of these), a counter per class and their total
    int *sum_b = lds, *sum_x = lds + kMaxExperts, *sum_m = lds + 2 * kMaxExperts, *slot = sum_m + kMaxExperts + 1;
    const int tid = threadIdx.x, lane = tid & 63, n_threads = blockDim.x;
    if (tid < kEsClasses) slot[tid] = 0;
    for (int e = tid; e < E; e += n_threads) {
        const int count = es_range(offsets, e, N).count;
        sum_b[e] = (count + kEsTokens - 1) / kEsTokens;
        sum_x[e] = es_items(count, chunk) - 1;
    }
    __syncthreads();
    if (tid < 64) {          // exclusive sums, by one wave
        int before_b = 0, before_x = 0, before_m = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const int nb = e < E ? sum_b[e] : 0, nx = e < E ? sum_x[e] : 0;
            const uint64_t multi = __ballot(nx > 0);
            int ib = nb, ix = nx;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int a = __shfl_up(ib, o), b = __shfl_up(ix, o);
                if (lane >= o) {
                    ib += a;
                    ix += b;
                }
            }
            if (e < E) {
                sum_b[e] = before_b + ib - nb;
                sum_x[e] = before_x + ix - nx;
                sum_m[e] = before_m + __popcll(multi & ((1ull << lane) - 1ull));
            }
            before_m += __popcll(multi);
            before_b += __builtin_amdgcn_readlane(ib, 63);
            before_x += __builtin_amdgcn_readlane(ix, 63);
        }
        if (lane == 0) sum_m[E] = before_m;
    }
    __syncthreads();
    // class 0: the longest
    auto class_of = [&](int rows) {
        return kEsClasses - 1 - static_cast<int>(static_cast<int64_t>(rows > 0 ? rows - 1 : 0) * kEsClasses / chunk);
    };
    for (int e = tid; e < E; e += n_threads) {
        const int count = es_range(offsets, e, N).count, n = es_items(count, chunk);
        if (n > 1) atomicAdd(&slot[class_of(chunk)], n - 1);
        atomicAdd(&slot[class_of(count - (n - 1) * chunk)], 1);
    }
    __syncthreads();
    if (tid == 0) {
        int at = 0;
        for (int c = 0; c < kEsClasses; ++c) {
            const int n = slot[c];
            slot[c] = at;
            at += n;
        }
        slot[kEsClasses] = at;
    }
    __syncthreads();
    const int max_parts = min(E, max_items - E);      // experts with partial sketches, at most
    for (int i = slot[kEsClasses] + tid; i < max_items; i += n_threads) items[i].expert = -1;
    for (int e = tid; e < E; e += n_threads) {
        const EsRange r = es_range(offsets, e, N);
        const int n = es_items(r.count, chunk);
        for (int i = 0; i < n; ++i) {
            const int rows = min(chunk, r.count - i * chunk);
            const int at = atomicAdd(&slot[class_of(rows)], 1);
            if (at < max_items)
                items[at] = EsItem{e, r.begin + i * chunk, rows, sum_b[e] + i * (chunk / kEsTokens),
                                   i > 0 ? sum_x[e] + i - 1 : n > 1 ? -1 : -2, {0, 0, 0}};
        }
        if (n > 1 && sum_m[e] < max_parts) experts[sum_m[e]] = EsParts{e, sum_x[e], n - 1};
    }
    for (int i = sum_m[E] + tid; i < max_parts; i += n_threads) experts[i].count = 0;
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
// A block of P is 32 rows x r, stored as the second product's operand: per 32
// columns four runs of 1 KB, one for each load of a wave there. Lane (i, h)
// of it takes rows 16 kb + 8 h + 4 q .. +3 of column i, kb and q the run's
// number. Returns where four rows from 4 rows4 of a column are.
__device__ __forceinline__ int es_p_at(int col, int rows4) {
    const int kb = rows4 >> 2, h = (rows4 >> 1) & 1, q = rows4 & 1;
    return ((((col >> 5) * 2 + kb) * 2 + q) * 64 + h * 32 + (col & 31)) * 4;
}

// A workgroup owns one 32-row block of P and RT of its columns over the
// whole of k; its eight waves split the k range and add their tiles through
// LDS in wave order, as stage 1 of the one-matrix sketch does.
constexpr int kEsWaves = 8, kEsWords = 8;
constexpr int kEsAhead = 3;         // sign words' columns of X in flight

template <int RT>
__global__ __launch_bounds__(512) void es_project_kernel(ExpertSketchArgs a, int chunk, int K, int64_t p_blocks,
                                                         int max_items,
                                                         EsItem *__restrict__ items, EsParts *__restrict__ experts,
                                                         float *__restrict__ P) {
    constexpr int NB = RT / 16, MB = 2;
    constexpr int kTileLd = kEsTokens + 4;
    constexpr int kTable = kEsWaves * kEsWords * RT * 8, kTiles = kEsWaves * RT * kTileLd * 4;
    __shared__ __attribute__((aligned(16))) char smem[kTable > kTiles ? kTable : kTiles];
    uint64_t *table = reinterpret_cast<uint64_t *>(smem);
    float *tile = reinterpret_cast<float *>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    // workgroup ids are dealt round-robin over the XCDs: the column tiles of a
    // block go to one XCD, whose L2 then holds its rows of X
    const int j = blockIdx.x / kXcds, tiles = a.R / RT;
    const int number = j / tiles * kXcds + static_cast<int>(blockIdx.x % kXcds), l0 = j % tiles * RT;
    if (number == 0) {
        if (l0 == 0)
            es_build_items(a.offsets, a.E, static_cast<int>(a.N), chunk, max_items, items, experts,
                           reinterpret_cast<int *>(smem));
        return;
    }
    const EsUnit at = es_unit(a.offsets, a.E, static_cast<int>(a.N), number - 1, kEsTokens, 1);
    if (at.expert < 0) return;
    const EsRange rows = at.rows;
    const int n = min(kEsTokens, rows.count - at.index * kEsTokens);       // rows of this block
    const uint64_t key = es_key(a, at.expert);

    const __amdgpu_buffer_rsrc_t xv = es_view(a.X, static_cast<uint32_t>(a.x_rows * a.ldx * 2));
    uint32_t xoff[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int i = 16 * mb + i16;
        const int64_t r = i < n ? es_x_row(a, rows.begin + at.index * kEsTokens + i) : -1;
        xoff[mb] = r < 0 ? kEsOob : static_cast<uint32_t>((r * a.ldx + 8 * g) * 2);
    }
    const int nkb = (K + 63) >> 6;
    const int bpw = (nkb + kEsWaves - 1) / kEsWaves;
    const int kb0 = min(nkb, wave * bpw), kb1 = min(nkb, kb0 + bpw);
    // the columns of sign word b, 32 each half
    auto xload = [&](int b, u32x4_t (&x)[2][MB]) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const int k = 64 * b + 32 * half;
                x[half][mb] = es_load(xv, (xoff[mb] + 2u * k) | (b < kb1 && k + 8 * g < K ? 0u : kEsOob));
            }
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
    u32x4_t x[kEsAhead][2][MB];
#pragma unroll
    for (int q = 0; q < kEsAhead; ++q) xload(kb0 + q, x[q]);
    int first = kb0;
    if (kb0 < kb1) refill(first);
    auto word_step = [&](int b, u32x4_t (&xb)[2][MB]) {
        if (b >= first + kEsWords) {
            first += kEsWords;
            refill(first);
        }
        const uint64_t *wrow = wt + (b - first) * RT + i16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint64_t w = wrow[16 * nb];
                const uint32_t dw = half ? static_cast<uint32_t>(w >> 32) : static_cast<uint32_t>(w);
                const u32x4_t bf = signs8_to_bf16(__builtin_amdgcn_ubfe(dw, 8 * g, 8), one_pair);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) acc[mb][nb] = mfma_bf16(xb[half][mb], bf, acc[mb][nb]);
            }
        }
    };
    for (int b0 = kb0; b0 < kb1; b0 += kEsAhead) {
#pragma unroll
        for (int q = 0; q < kEsAhead; ++q) {
            if (b0 + q < kb1) word_step(b0 + q, x[q]);
            xload(b0 + q + kEsAhead, x[q]);
        }
    }
    __syncthreads();      // every wave is done with its word table
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            *reinterpret_cast<f32x4_t *>(&tile[(wave * RT + 16 * nb + i16) * kTileLd + 16 * mb + 4 * g]) = acc[mb][nb];
    __syncthreads();
    const int64_t block = static_cast<int64_t>(at.blocks) + at.index;
    if (block >= p_blocks) return;
    for (int q = tid; q < RT * 8; q += 512) {      // four rows of one column
        const int col = q % RT, t = 4 * (q / RT);
        f32x4_t v = zero_f32x4();
#pragma unroll
        for (int w = 0; w < kEsWaves; ++w) v += *reinterpret_cast<const f32x4_t *>(&tile[(w * RT + col) * kTileLd + t]);
        *reinterpret_cast<f32x4_t *>(P + block * a.R * kEsTokens + es_p_at(l0 + col, t / 4)) = a.c * v;
    }
}

// The same product for calls with many rows and r >= 128: up to 64 rows of
// one expert and all r columns per workgroup, so that X is read once, on
// 32x32x16 matrix instructions (short units may take half the columns, NB =
// 1). Each of the eight waves holds all 64 rows of 32 NB columns; they split
// the columns and k, and the k parts are added through LDS in order. X goes through LDS in steps of 64 columns of k per part, two
// buffers, requested a step ahead; each lane hashes the one sign word of its
// column and step, a step ahead. Row blocks without rows are skipped.
constexpr int kEsWideRows = 64;
constexpr int kEsXRow = 72;            // bf16 per LDS row of 64 (16 bytes of padding against bank conflicts)
constexpr int kEsTileLd = kEsWideRows + 4;

template <int R>
struct EsWide {
    static constexpr int WN = R / 64, WK = 8 / WN;      // waves across the columns, across k
    static constexpr int X_BUF = WK * kEsWideRows * kEsXRow;            // elements of one buffer
    static constexpr int TILE_BYTES = (WK - 1) * R * kEsTileLd * 4;
    static constexpr int LDS_BYTES = 4 * X_BUF > TILE_BYTES ? 4 * X_BUF : TILE_BYTES;
};

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// D = A(32x16 bf16) * B(16x32 bf16) + C. Lane L holds A[L%32][8*(L/32) .. +7],
// B[8*(L/32) .. +7][L%32] and D[8*(i/4) + 4*(L/32) + i%4][L%32], i = 0 .. 15.
__device__ __forceinline__ f32x16_t mfma_bf16_32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                  0, 0, 0);
}

// Byte `sel` of a sign word (its number in bytes 0 and 2 of sel, 0x0C in the
// others) as eight bf16 +-1: the byte goes to both halves of a dword, then one
// packed shift brings two of its bits to the sign positions.
__device__ __forceinline__ u32x4_t es_signs(uint64_t word, uint32_t sel, uint32_t one) {
    const uint32_t z = __builtin_amdgcn_perm(static_cast<uint32_t>(word >> 32), static_cast<uint32_t>(word), sel);
    const u16x2_t v = __builtin_bit_cast(u16x2_t, z);
    u32x4_t r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const u16x2_t sh = {static_cast<unsigned short>(15 - 2 * q), static_cast<unsigned short>(14 - 2 * q)};
        r[q] = (__builtin_bit_cast(uint32_t, v << sh) & 0x80008000u) | one;
    }
    return r;
}

template <int R, int NB>
__device__ __forceinline__ void es_project_unit(const ExpertSketchArgs &a, const EsUnit &at, int col0, int K,
                                                int64_t p_blocks, float *__restrict__ P, char *smem,
                                                uint64_t (*words)[64]) {
    using Sh = EsWide<R>;
    constexpr int WN = Sh::WN, WK = Sh::WK, MB = kEsWideRows / 32;
    uint16_t *xs = reinterpret_cast<uint16_t *>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wk = wave / WN;
    const int i32 = lane & 31, h = lane >> 5;
    const EsRange rows = at.rows;
    const int r0 = at.index * kEsWideRows;
    const int n = min(kEsWideRows, rows.count - r0);
    const int blocks = __builtin_amdgcn_readfirstlane((n + 31) >> 5);
    const int l0 = col0 + 32 * NB * wn;

    // the row of X whose 16-byte pieces this thread moves
    const int xr = tid >> 3, xc = 8 * (tid & 7);
    const __amdgpu_buffer_rsrc_t xv = es_view(a.X, static_cast<uint32_t>(a.x_rows * a.ldx * 2));
    const int64_t row = xr < n ? es_x_row(a, rows.begin + r0 + xr) : -1;
    const uint32_t xoff = row < 0 ? kEsOob : static_cast<uint32_t>((row * a.ldx + xc) * 2);
    auto xload = [&](int i, u32x4_t (&x)[WK]) {
#pragma unroll
        for (int p = 0; p < WK; ++p) {
            const int k = 64 * (WK * i + p);
            x[p] = es_load(xv, (xoff + 2u * k) | (k + xc < K ? 0u : kEsOob));
        }
    };
    // columns of k past K are zeros in X, so their signs do not matter
    const uint64_t first_word = es_key(a, at.expert) + ((static_cast<uint64_t>(l0 + lane % (32 * NB)) << 32) + 1ull) * kGolden;
    auto word_at = [&](int i) { return splitmix_finalize(first_word + static_cast<uint64_t>(WK * i + wk) * kGolden); };
    f32x16_t acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[mb][nb][e] = 0.f;
    const uint32_t one_pair = opaque_u32(0x3F803F80u);
    const int steps = (K + 64 * WK - 1) / (64 * WK);
    // the loop over k with M row blocks
    auto run = [&](auto m_blocks) {
        constexpr int M = decltype(m_blocks)::value;
        u32x4_t x[WK];
        xload(0, x);
        uint64_t word = word_at(0);
        auto step = [&](int i) {
            uint16_t *buf = xs + (i & 1) * Sh::X_BUF;
#pragma unroll
            for (int p = 0; p < WK; ++p)
                *reinterpret_cast<u32x4_t *>(buf + (p * kEsWideRows + xr) * kEsXRow + xc) = x[p];
            words[wave][lane] = word;
            xload(i + 1, x);
            lds_barrier();
            const uint16_t *mine = buf + (wk * kEsWideRows + i32) * kEsXRow + 8 * h;
            uint64_t w[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) w[nb] = words[wave][32 * nb + i32];
            word = word_at(i + 1);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                u32x4_t av[M];
#pragma unroll
                for (int mb = 0; mb < M; ++mb)
                    av[mb] = *reinterpret_cast<const u32x4_t *>(mine + 32 * mb * kEsXRow + 16 * kb);
                const uint32_t sel = 0x0C000C00u + 0x00010001u * (2 * kb + h);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const u32x4_t bf = es_signs(w[nb], sel, one_pair);
#pragma unroll
                    for (int mb = 0; mb < M; ++mb) acc[mb][nb] = mfma_bf16_32(av[mb], bf, acc[mb][nb]);
                }
            }
        };
        for (int i = 0; i < steps; ++i) step(i);
    };
    if (blocks == 1) run(std::integral_constant<int, 1>());
    else run(std::integral_constant<int, 2>());
    // The k parts are added in order, each 32 x 32 block (mb, nb) by one of the
    // WK waves that hold a part of it: lane (i32, h) holds rows
    // 32 mb + 8 q + 4 h .. +3 of its column i32, q = 0 .. 3.
    float *tile = reinterpret_cast<float *>(smem);
    auto at_tile = [&](int part, int mb, int nb, int q) {
        return reinterpret_cast<f32x4_t *>(
            &tile[(part * R + 32 * NB * wn + 32 * nb + i32) * kEsTileLd + 32 * mb + 8 * q + 4 * h]);
    };
    auto piece = [&](int mb, int nb, int q) {
        return f32x4_t{acc[mb][nb][4 * q], acc[mb][nb][4 * q + 1], acc[mb][nb][4 * q + 2], acc[mb][nb][4 * q + 3]};
    };
    // wave wk finishes the blocks (mb, nb) with (NB mb + nb) % WK == wk; of the
    // others' parts, part p lies in slot (p - wk - 1) mod WK
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int owner = (NB * mb + nb) % WK;
            if (owner == wk) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) *at_tile((wk + WK - owner - 1) % WK, mb, nb, q) = piece(mb, nb, q);
        }
    __syncthreads();
    const int64_t block0 = static_cast<int64_t>(at.blocks) + MB * at.index;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        if (mb >= blocks || block0 + mb >= p_blocks) break;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if ((NB * mb + nb) % WK != wk) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4_t v = zero_f32x4();
#pragma unroll
                for (int part = 0; part < WK; ++part)
                    v += part == wk ? piece(mb, nb, q) : *at_tile((part + WK - wk - 1) % WK, mb, nb, q);
                *reinterpret_cast<f32x4_t *>(P + (block0 + mb) * R * kEsTokens + es_p_at(l0 + 32 * nb + i32, 2 * q + h)) =
                    a.c * v;
            }
        }
    }
}

template <int R>
__global__ __launch_bounds__(512, R == 256 ? 4 : 2) void es_project_wide_kernel(ExpertSketchArgs a, int chunk, int K,
                                                                 int64_t p_blocks, int max_items, int split,
                                                                 EsItem *__restrict__ items,
                                                                 EsParts *__restrict__ experts,
                                                                 float *__restrict__ P) {
    __shared__ __attribute__((aligned(16))) char smem[EsWide<R>::LDS_BYTES];
    __shared__ uint64_t words[8][64];
    if (blockIdx.x == 0) {
        es_build_items(a.offsets, a.E, static_cast<int>(a.N), chunk, max_items, items, experts,
                       reinterpret_cast<int *>(smem));
        return;
    }
    const EsUnit at = es_unit(a.offsets, a.E, static_cast<int>(a.N), blockIdx.x - 1, kEsWideRows, split);
    if (at.expert < 0) return;
    if (at.part < 0 || split == 1) es_project_unit<R, 2>(a, at, 0, K, p_blocks, P, smem, words);
    else es_project_unit<R, 1>(a, at, at.part * (R / 2), K, p_blocks, P, smem, words);
}

// ---------------------------------------------------------- bf16, stage 2 --
// A workgroup owns one item (at most `chunk` rows of one expert) and kEsRows
// rows of its S, all r columns: dY is read once and S written once. The waves
// split the columns; each step of 32 rows brings the dY tile through LDS (read
// transposed, the A operand) and P from the L2, each piece of the next step
// requested as soon as this step has taken it apart.
constexpr int kEsRows = 128;

// Eight values of P as MFMA fragments of their three terms.
constexpr int kEsTerms = 3;
__device__ __forceinline__ void es_split(u32x4_t lo, u32x4_t hi, u32x4_t (&p)[kEsTerms]) {
    // what a term leaves, x - term, by a two-element dot product with (-1, 0)
    // or (0, -1): one instruction instead of a shift and a subtraction. The
    // constants stay in registers: folded into the instruction, (-1, 0) was
    // built as the inline constant -1.0, which the hardware reads as (0, -1).
    const bf16x2_t minus_lo = __builtin_bit_cast(bf16x2_t, opaque_u32(0x0000BF80u));
    const bf16x2_t minus_hi = __builtin_bit_cast(bf16x2_t, opaque_u32(0xBF800000u));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float x = __uint_as_float(e < 2 ? lo[2 * e] : hi[2 * e - 4]);
        float y = __uint_as_float(e < 2 ? lo[2 * e + 1] : hi[2 * e - 3]);
#pragma unroll
        for (int q = 0; q < kEsTerms; ++q) {
            const uint32_t w = pack_bf16x2(x, y);
            p[q][e] = w;
            x = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), minus_lo, x, false);
            y = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), minus_hi, y, false);
        }
    }
}

template <int R>
__global__ __launch_bounds__(256, 2) void es_fold_kernel(ExpertSketchArgs a, int D, int tiles, int max_items,
                                                         int64_t p_blocks, int64_t max_extras, int stream,
                                                         const EsItem *__restrict__ items,
                                                         const float *__restrict__ P, float *__restrict__ parts) {
    constexpr int WN = R / 32 < 4 ? R / 32 : 4;         // waves across the columns
    constexpr int WM = 4 / WN;                          // waves across the rows
    constexpr int NB = R / 32 / WN, MB = kEsRows / 32 / WM;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2][kEsTokens * kEsRows];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i32 = lane & 31, h = lane >> 5;
    // workgroup ids are dealt round-robin over the XCDs: the tiles of an item
    // go to one XCD, whose L2 then holds its P
    const int j = blockIdx.x / kXcds;
    const int number = j / tiles * kXcds + static_cast<int>(blockIdx.x % kXcds), d0 = j % tiles * kEsRows;
    if (number >= max_items) return;
    const EsItem item = items[number];
    if (item.expert < 0) return;
    const int n = item.rows;
    const int64_t block0 = item.block;
    const int steps = static_cast<int>(min(static_cast<int64_t>((n + kEsTokens - 1) / kEsTokens),
                                           max(static_cast<int64_t>(0), p_blocks - block0)));
    float *dst = a.S + static_cast<int64_t>(item.expert) * D * R;
    bool add = a.accumulate != 0;
    if (item.part >= 0) {       // added to S by es_reduce_kernel
        if (item.part >= max_extras) return;
        dst = parts + static_cast<int64_t>(item.part) * D * R;
        add = false;
    } else if (n <= 0 && add) {
        return;
    }

    f32x16_t acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[mb][nb][e] = 0.f;
    if (steps > 0) {
        // A dY tile in LDS: row t, 16-column block b at block b ^ swizzle(t)
        // of the row, so that the rows a transposed read touches at once lie
        // in different banks.
        const uint16_t *dy = static_cast<const uint16_t *>(a.dY) + static_cast<int64_t>(item.begin) * a.lddy;
        const uint32_t ld_bytes = static_cast<uint32_t>(a.lddy * 2);
        const int lt = tid >> 4, lc = tid & 15;         // this thread's rows (lt, lt + 16) and 8-column piece
        auto swizzle = [](int t) { return (t & 3) | ((t >> 1) & 4); };
        const uint32_t goff = d0 + 8 * lc < D ? lt * ld_bytes + 2 * (d0 + 8 * lc) : kEsOob;
        // (the views of a step's 32 rows start at their first one: an item may be longer than a view reaches)
        auto gload = [&](int s, u32x4_t (&v)[2]) {
            const uint32_t left = static_cast<uint32_t>(min(kEsTokens, max(0, n - kEsTokens * s)));
            const __amdgpu_buffer_rsrc_t view = es_view(dy + static_cast<int64_t>(s) * kEsTokens * a.lddy, left * ld_bytes);
            v[0] = es_load(view, goff);
            v[1] = es_load(view, goff + 16 * ld_bytes);
        };
        constexpr uint32_t kStep = R * kEsTokens * 4;   // bytes of P per step
        const __amdgpu_buffer_rsrc_t pview = es_view(P + block0 * R * kEsTokens, static_cast<uint32_t>(steps) * kStep);
        const uint32_t poff = wn * NB * 4096 + lane * 16;
        auto pload = [&](uint32_t at_step, int nb, int kb, u32x4_t (&v)[2]) {
            const uint32_t off = poff + at_step + 4096 * nb + 2048 * kb;
            v[0] = es_load(pview, off);
            v[1] = es_load(pview, off + 1024);
        };
        u32x4_t next0[2], next1[2], pv[2][NB][2];
        gload(0, next0);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) pload(0, nb, kb, pv[kb][nb]);
        gload(1, next1);
        auto step = [&](int s, u32x4_t (&next)[2]) {
            uint16_t *buf = lds[s & 1];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = lt + 16 * q;
                *reinterpret_cast<u32x4_t *>(&buf[t * kEsRows + 16 * ((lc >> 1) ^ swizzle(t)) + 8 * (lc & 1)]) = next[q];
            }
            gload(s + 2, next);
            lds_barrier();
            const uint32_t ahead = static_cast<uint32_t>(s + 1) * kStep;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                // 16 rows t = 16 kb ..: lanes of group g16 read columns 16 (g16 & 1) of a
                // 32-column block, rows 8 (g16 >> 1) ..
                u32x4_t av[MB];
                const int t = 16 * kb + 8 * h + ((lane & 15) >> 2);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    const int b16 = 2 * (wm * MB + mb) + ((lane >> 4) & 1);
                    const uint16_t *src = buf + t * kEsRows + 16 * (b16 ^ swizzle(t)) + 4 * (lane & 3);
                    const u32x2_t x = lds_read_tr(src), y = lds_read_tr(src + 4 * kEsRows);
                    av[mb] = u32x4_t{x.x, x.y, y.x, y.y};
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    u32x4_t p[kEsTerms];
                    es_split(pv[kb][nb][0], pv[kb][nb][1], p);
                    pload(ahead, nb, kb, pv[kb][nb]);
                    __builtin_amdgcn_sched_barrier(0);      // the request stays a step ahead of its use
#pragma unroll
                    for (int q = kEsTerms - 1; q >= 0; --q)
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) acc[mb][nb] = mfma_bf16_32(av[mb], p[q], acc[mb][nb]);
                }
            }
        };
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            step(s, next0);
            step(s + 1, next1);
        }
        if (s < steps) step(s, next0);
    }
    // lane (i32, h) of block (mb, nb): rows 8 q + 4 h + e of column i32
    float *out = dst + static_cast<int64_t>(d0) * R + 32 * wn * NB + i32;
    auto each = [&](auto f) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const int row = 32 * (wm * MB + mb) + 8 * (q >> 2) + 4 * h + (q & 3);
                if (d0 + row < D)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) f(out + row * R + 32 * nb, acc[mb][nb][q]);
            }
    };
    if (add) each([](float *p, float v) { *p += v; });
    else if (stream && item.part == -2) each([](float *p, float v) { __builtin_nontemporal_store(v, p); });
    else each([](float *p, float v) { *p = v; });
}

// S_e += the partial sketches of expert e, in their order; a row of workgroups
// per expert that has some.
__global__ __launch_bounds__(256) void es_reduce_kernel(ExpertSketchArgs a, int64_t size, int64_t max_extras,
                                                        const EsParts *__restrict__ experts,
                                                        const float *__restrict__ parts) {
    const EsParts own = experts[blockIdx.y];
    if (own.count == 0) return;
    float *S = a.S + static_cast<int64_t>(own.expert) * size;
    const float *p = parts + static_cast<int64_t>(own.first) * size;
    const int n = static_cast<int>(min(static_cast<int64_t>(own.count), max(static_cast<int64_t>(0), max_extras - own.first)));
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < size;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        f32x4_t v = *reinterpret_cast<const f32x4_t *>(S + i);
        int q = 0;
        for (; q + 4 <= n; q += 4) {        // four requests at once
            f32x4_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const f32x4_t *>(p + (q + j) * size + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v += w[j];
        }
        for (; q < n; ++q) v += *reinterpret_cast<const f32x4_t *>(p + q * size + i);
        *reinterpret_cast<f32x4_t *>(S + i) = v;
    }
}

// ------------------------------------------------------------------- fp32 --
// Both products on the fp32 matrix instructions (fp32 products and sums), any
// shape. P is N x r, row i of the sorted rows in row i. A workgroup owns a
// tile of the result and its waves split the contraction, adding their tiles
// through LDS in wave order. Operands come straight from memory: the calls
// this path is for are short, and what bounds them is the latency of a few
// loads, which more waves over fewer steps hide best.
constexpr int kEsF32Waves = 8;
constexpr int kEsUnitsAtOnce = 1 << 16;     // units of a grid's row: a launch has fewer than 2^32 threads in x

// D = A(16x4) * B(4x16) + C. Lane L holds A[L%16][L/16], B[L/16][L%16] and
// D[4*(L/16) .. +3][L%16].
__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

typedef f32x4_t f32x4_a4_t __attribute__((aligned(4)));     // rows need only their element's alignment

// Adds the waves' tiles of MT x NT blocks in wave order and calls
// store(row, column, value) for every element (row and column in the tile).
template <int MT, int NT, class Store>
__device__ __forceinline__ void es_f32_join(f32x4_t (&acc)[MT][NT], float *lds, Store store) {
    constexpr int kLd = 16 * MT + 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<f32x4_t *>(&lds[(wave * 16 * NT + 16 * n + i16) * kLd + 16 * m + 4 * g]) = acc[m][n];
    __syncthreads();
    for (int q = tid; q < 16 * MT * 16 * NT; q += 64 * kEsF32Waves) {
        const int row = q / (16 * NT), col = q - row * 16 * NT;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kEsF32Waves; ++w) v += lds[(w * 16 * NT + col) * kLd + row];
        store(row, col, v);
    }
}

template <int T>
__global__ __launch_bounds__(64 * kEsF32Waves) void es_project_f32_kernel(ExpertSketchArgs a, int K,
                                                                          float *__restrict__ P) {
    constexpr int MT = T, NT = T, kRows = 16 * T;
    __shared__ __attribute__((aligned(16))) float lds[kEsF32Waves * 16 * NT * (16 * MT + 4)];
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the column tiles of a block of rows go to one XCD, as in the bf16 kernel
    const int j = blockIdx.x / kXcds, tiles = (a.R + 16 * NT - 1) / (16 * NT);
    const int number = blockIdx.z * kEsUnitsAtOnce + j / tiles * kXcds + static_cast<int>(blockIdx.x % kXcds);
    const int l0 = j % tiles * 16 * NT;
    const EsUnit at = es_unit(a.offsets, a.E, static_cast<int>(a.N), number, kRows, 1);
    if (at.expert < 0) return;
    const EsRange rows = at.rows;
    const int i0 = rows.begin + at.index * kRows, n = min(kRows, rows.count - at.index * kRows);
    const uint64_t key = es_key(a, at.expert);
    const float *xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t row = 16 * m + i16 < n ? es_x_row(a, i0 + 16 * m + i16) : -1;
        xrow[m] = row < 0 ? nullptr : static_cast<const float *>(a.X) + row * a.ldx;
    }
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[m][q] = zero_f32x4();
    // 64 columns of k per step; piece q of a lane is columns 16 q + 4 g .. +3, so
    // that the lane's four loads are one row's and its four products' k agree
    // between X and the signs
    for (int b = wave; b < (K + 63) / 64; b += kEsF32Waves) {
        f32x4_t x[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int k = 64 * b + 16 * q + 4 * g;
                x[m][q] = zero_f32x4();
                if (xrow[m] && k + 4 <= K) x[m][q] = *reinterpret_cast<const f32x4_a4_t *>(xrow[m] + k);
                else if (xrow[m])
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k + e < K) x[m][q][e] = xrow[m][k + e];
            }
        uint64_t w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            w[t] = sign_word(key, static_cast<uint32_t>(l0 + 16 * t + i16), static_cast<uint32_t>(b)) >> (4 * g);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t bit = static_cast<uint32_t>(w[t] >> (16 * q)) << (31 - e);
                    const float sign = __uint_as_float((bit & 0x80000000u) | 0x3F800000u);
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[m][t] = mfma_f32(x[m][q][e], sign, acc[m][t]);
                }
    }
    const int R = a.R;
    es_f32_join(acc, lds, [&](int row, int col, float v) {
        if (row < n && l0 + col < R) P[static_cast<int64_t>(i0 + row) * R + l0 + col] = a.c * v;
    });
}

template <int T>
__global__ __launch_bounds__(64 * kEsF32Waves) void es_fold_f32_kernel(ExpertSketchArgs a, int D,
                                                                       const float *__restrict__ P) {
    __shared__ __attribute__((aligned(16))) float lds[kEsF32Waves * 16 * T * (16 * T + 4)];
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const EsRange rows = es_range_uniform(a.offsets, blockIdx.z, static_cast<int>(a.N));
    if (rows.count == 0 && a.accumulate) return;
    const int R = a.R, d0 = blockIdx.x * 16 * T, l0 = blockIdx.y * 16 * T;
    const float *dY = static_cast<const float *>(a.dY);
    f32x4_t acc[T][T];
#pragma unroll
    for (int m = 0; m < T; ++m)
#pragma unroll
        for (int n = 0; n < T; ++n) acc[m][n] = zero_f32x4();
    constexpr int U = T > 2 ? 2 : 4;       // steps of four rows in flight
    for (int t0 = 4 * U * wave; t0 < rows.count; t0 += 4 * U * kEsF32Waves) {
        float av[U][T], bv[U][T];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + 4 * u + g;
            const int64_t i = static_cast<int64_t>(rows.begin) + t;
            const bool in = t < rows.count;
#pragma unroll
            for (int q = 0; q < T; ++q) {
                const int d = d0 + 16 * q + i16, l = l0 + 16 * q + i16;
                av[u][q] = in && d < D ? dY[i * a.lddy + d] : 0.f;
                bv[u][q] = in && l < R ? P[i * R + l] : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < T; ++n)
#pragma unroll
                for (int m = 0; m < T; ++m) acc[m][n] = mfma_f32(av[u][m], bv[u][n], acc[m][n]);
    }
    float *S = a.S + static_cast<int64_t>(blockIdx.z) * D * R;
    es_f32_join(acc, lds, [&](int row, int col, float v) {
        if (d0 + row >= D || l0 + col >= R) return;
        float *p = S + static_cast<int64_t>(d0 + row) * R + l0 + col;
        *p = a.accumulate ? *p + v : v;
    });
}

// ------------------------------------------------------------------ plans --
constexpr int64_t kEsF32WideFrom = 256;
// The fp32 projection's tiles are 32 x 32, and 16 x 16 where that would make no
// more than kEsF32SmallWGs workgroups (8 experts: 768 rows, k = 512, r = 32 5.1 us
// against 7.8 with 32 x 32, r = 256 8.2 against 8.5; 2048 rows, k = 2048, r = 256
// 38 against 31).
constexpr int64_t kEsF32SmallWGs = 256;
constexpr int64_t kEsMaxChunk = 1 << 20;   // an item's part of P stays within a view (r <= 256)
// The wide projection is used from kEsWideFrom rows or where the other one
// would take more than kEsWideWGs workgroups (whole call, k = 2048, r = 256:
// 8 experts, 2048 rows 34 us against 37 wide, 4096 rows 45 against 40; 128
// experts, 1024 rows 42 against 41, 2048 rows 51 against 42).
constexpr int64_t kEsWideFrom = 4096, kEsWideWGs = 320;

// The other projection takes 128 columns, or all r, per workgroup; 64 or 32
// where it would have no more than kEsNarrowWGs workgroups (8 experts, k =
// 2048, r = 256: 512 rows 9.1 us with 32 columns, 10.7 with 64, 12.6 with 128;
// 2048 rows 15.2, 11.8, 14.1; 16 experts, 128 rows, k = 1536, r = 64: 6.7 with
// 32 columns, 8.0 with 64).
constexpr int64_t kEsNarrowWGs = 160;

constexpr int64_t kEsReduceWGs = 256;      // per expert, at most
// Where the experts' last, shorter units are few, two workgroups take half the
// columns of each: they fill what the long ones leave (k = 2048, r = 256, kernel
// alone: 128 uneven experts, 32768 rows 48.7 us against 52.7, 4096 rows 15.8
// against 18.6; 256 experts, 8192 rows 26.1 against 23.5; with r = 128, one
// workgroup per compute unit, 128 experts, 33568 rows 42.3 against 40.8).
constexpr int64_t kEsSplitShorts = 128;
// From this many elements of S on (the 32 MB of all L2 caches) what the second
// product finishes is written past them, so that P stays there: 67 -> 62.5 us
// for the 100 MB of the call above.
constexpr int64_t kEsStream = 8ll << 20;

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
    // Rows of an item: the longest one's time grows with them, and every item
    // beyond an expert's first costs d r 4 bytes written and read again. With
    // N / chunk such items the sum of the two is least at sqrt(N d r) times a
    // constant. Whole call in us with 1 / 152, 1 / 110, 1 / 90 of it, uneven
    // experts, d = 768, k = 2048, r = 256: 128 experts, 32768 rows 106, 97, 97;
    // 32 experts, 16384 rows 66, 63, 62; 8 experts, 8192 rows 45, 47, 48.
    int64_t chunk = static_cast<int64_t>(sqrt(static_cast<double>(N) * static_cast<double>(d) * R) / 110.0);
    chunk = (chunk < 256 ? 256 : chunk + 31) / 32 * 32;
    if (chunk > kEsMaxChunk) chunk = kEsMaxChunk;
    p.chunk = static_cast<int>(chunk);
    p.extras = N > 0 ? (N - 1) / p.chunk : 0;
    p.items = E + p.extras;
    p.p_bytes = static_cast<size_t>(p.p_blocks) * R * kEsTokens * 4;
    p.table_bytes = (static_cast<size_t>(p.items) * sizeof(EsItem) + E * sizeof(EsParts) + 255) / 256 * 256;
    p.total = p.table_bytes + p.p_bytes + static_cast<size_t>(p.extras) * d * R * 4;
    return p;
}

template <int R>
static hipError_t expert_sketch_bf16_r(const ExpertSketchArgs &a, hipStream_t st) {
    const ExpertSketchPlan p = plan_expert_sketch(a.N, a.E, a.d, a.k, R, 1);
    char *ws = static_cast<char *>(a.ws);
    EsItem *items = reinterpret_cast<EsItem *>(ws);
    EsParts *experts = reinterpret_cast<EsParts *>(items + p.items);
    float *P = reinterpret_cast<float *>(ws + p.table_bytes);
    float *parts = reinterpret_cast<float *>(ws + p.table_bytes + p.p_bytes);
    const int D = static_cast<int>(a.d), K = static_cast<int>(a.k), n_items = static_cast<int>(p.items);
    bool done = false;
    if constexpr (R >= 128) {
        done = a.N >= kEsWideFrom || p.p_blocks * (R / 128) > kEsWideWGs;
        if (done) {
            const int64_t shorts = a.N < a.E ? a.N : a.E;        // units of fewer rows, at most
            const int split = R == 256 && shorts <= kEsSplitShorts ? 2 : 1;
            const int64_t units = a.N / kEsWideRows + split * shorts;
            hipLaunchKernelGGL(es_project_wide_kernel<R>, dim3(units + 1), dim3(512), 0, st, a, p.chunk, K, p.p_blocks,
                               n_items, split, items, experts, P);
        }
    }
    if (!done) {
        int rt = R < 128 ? R : 128;
        while (rt > 32 && p.p_blocks * (R / rt) <= kEsNarrowWGs) rt /= 2;
        hipLaunchKernelGGL(rt == 32 ? es_project_kernel<32> : rt == 64 ? es_project_kernel<64> : es_project_kernel<128>,
                           dim3((p.p_blocks / kXcds + 1) * kXcds * (R / rt)), dim3(512), 0, st, a, p.chunk, K,
                           p.p_blocks, n_items, items, experts, P);
    }
    const int tiles = (D + kEsRows - 1) / kEsRows;
    hipLaunchKernelGGL(es_fold_kernel<R>, dim3((p.items + kXcds - 1) / kXcds * kXcds * tiles), dim3(256), 0, st, a, D,
                       tiles, n_items, p.p_blocks, p.extras, a.E * a.d * R > kEsStream ? 1 : 0, items, P, parts);
    if (p.extras > 0) {
        const int64_t size = a.d * R;
        const int64_t n = (size + 1023) / 1024;
        hipLaunchKernelGGL(es_reduce_kernel,
                           dim3(n < kEsReduceWGs ? n : kEsReduceWGs, p.extras < a.E ? p.extras : a.E), dim3(256), 0,
                           st, a, size, p.extras, experts, parts);
    }
    return hipGetLastError();
}

hipError_t launch_expert_sketch(const ExpertSketchArgs &a, int bf16, hipStream_t st) {
    if (!bf16) {
        const ExpertSketchPlan p = plan_expert_sketch(a.N, a.E, a.d, a.k, a.R, 0);
        float *P = static_cast<float *>(a.ws);
        const int D = static_cast<int>(a.d), K = static_cast<int>(a.k);
        if (p.p_blocks > 0) {
            const int T = p.p_blocks * ((a.R + 31) / 32) <= kEsF32SmallWGs ? 1 : 2;
            const int64_t units = a.N / (16 * T) + (a.N < a.E ? a.N : a.E);
            hipLaunchKernelGGL(T == 1 ? es_project_f32_kernel<1> : es_project_f32_kernel<2>,
                               dim3(((units < kEsUnitsAtOnce ? units : kEsUnitsAtOnce) + kXcds - 1) / kXcds * kXcds *
                                        ((a.R + 16 * T - 1) / (16 * T)), 1,
                                    (units + kEsUnitsAtOnce - 1) / kEsUnitsAtOnce),
                               dim3(64 * kEsF32Waves), 0, st, a, K, P);
        }
        // tiles of 64 x 64 where they still give each compute unit one, which
        // reads a quarter of what tiles of 32 x 32 read per product
        const bool wide = static_cast<int64_t>((a.R + 63) / 64) * ((D + 63) / 64) * a.E >= kEsF32WideFrom;
        const int tile = wide ? 64 : 32;
        hipLaunchKernelGGL(wide ? es_fold_f32_kernel<4> : es_fold_f32_kernel<2>,
                           dim3((D + tile - 1) / tile, (a.R + tile - 1) / tile, a.E), dim3(64 * kEsF32Waves), 0, st, a,
                           D, P);
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
