// Y = X W^T with operands in e4m3 and a scale for every 128 of the
// contraction, dense or over the experts of a layer:
//   Y[i][n] = sum_b xs[row(i)][b] ws[e][n / 128][b] sum_(k in block b) x[row(i)][k] w[e][n][k]
// row(i) = i, or order[i] / topk: the activations before the sort of
// experts.hip; e is the expert that sorted row i belongs to (offsets).
//
// Weights are the matrix instructions' first operand and rows of x their
// second, so a lane's four results are neighbouring features of one row of Y,
// all with one scale: one product of two scales per 16 x 16 block of results
// and block of k, then a multiply-add per result into fp32 accumulators. The
// accumulators are read by vector instructions every block, so they must live
// in vector registers (a wave can hold 128 of them beside its operands), which
// bounds a wave's share to 128 x 64 results.
//
// Y in bf16: one v_mfma_f32_16x16x128_f8f6f4 contracts a block of 128. These
// instructions add eight neighbouring products at a time with 13 bits below
// the largest one's exponent and cut off what is lower (measured, with
// v_mfma_f32_16x16x32_fp8_fp8 the same), and the groups' sums in fp32: each
// group of eight is off by at most 7 2^-13 of its largest product, 1.5e-5 of
// Y for codes of normal values, a hundredth of Y's rounding to bf16.
// Y in fp32: the codes are made bf16 (exact) and multiplied by
// v_mfma_f32_16x16x32_bf16, whose sums are fp32 (8e-8 of Y measured), at half
// the rate.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace logra {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;

constexpr uint32_t kMmOob = 0x80000000u;      // past every buffer view: loads give zeros
constexpr int kMmK = 128;
constexpr int kMmXcds = 8;

// Operand of 128 k: a lane has 32 of the k of row L % 16 of A or of column
// L % 16 of B (which ones does not matter as long as both have the same), as
// codes or as bf16 values.
template <int WIDE>
struct MmOperand {
    u32x4_t v[WIDE ? 4 : 2];
};
template <int WIDE>
__device__ __forceinline__ MmOperand<WIDE> mm_operand(u32x4_t c0, u32x4_t c1) {
    MmOperand<WIDE> o;
    if constexpr (WIDE) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t c = q < 4 ? c0[q] : c1[q - 4];
            o.v[q / 2][2 * (q % 2)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, false));
            o.v[q / 2][2 * (q % 2) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, true));
        }
    } else {
        o.v[0] = c0;
        o.v[1] = c1;
    }
    return o;
}

// sum_k A[f][k] B[k][r] over 128 k; lane L holds D[4 (L / 16) .. +3][L % 16].
template <int WIDE>
__device__ __forceinline__ f32x4_t mm_product(const MmOperand<WIDE> &a, const MmOperand<WIDE> &b) {
    if constexpr (WIDE) {
        f32x4_t p = zero_f32x4();
#pragma unroll
        for (int q = 0; q < 4; ++q) p = mfma_bf16(a.v[q], b.v[q], p);
        return p;
    } else {
        // formats 0, 0: e4m3; no block scales of its own
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8_t, a), __builtin_bit_cast(i32x8_t, b),
                                                                zero_f32x4(), 0, 0, 0, 0, 0, 0);
    }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_view(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, 0x7FFFFFFF, 0x00020000);
}
__device__ __forceinline__ u32x4_t mm_load16(__amdgpu_buffer_rsrc_t rs, uint32_t off, int step) {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, off, step, 0);
}
__device__ __forceinline__ float mm_load4(__amdgpu_buffer_rsrc_t rs, uint32_t off, int step) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, off, step, 0));
}

// What a workgroup works on: rows row0 .. row0 + rows - 1 of Y, all of one
// expert, and one tile of features.
struct MmTile {
    int expert, rows, tn;
    int64_t row0;
};

// The workgroup's tile of (row tiles of all experts) x (feature tiles).
// Workgroup ids of one XCD (id mod 8) have neighbouring tiles: BAND row tiles
// by as many feature tiles as there are workgroups, so that they read the
// same rows of x and w through the XCD's cache. False: none is left.
template <int BM>
__device__ __forceinline__ bool mm_tile(const MatmulCall &c, int n_tn, int band, MmTile *out) {
    const int lane = threadIdx.x & 63;
    int tiles, per = 1, mine = 0, before = 0;
    if (c.offsets) {
        per = (c.E + 63) / 64;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e >= c.E) break;
            const int64_t a = min(max(static_cast<int64_t>(c.offsets[e]), static_cast<int64_t>(0)), c.M);
            const int64_t b = min(max(static_cast<int64_t>(c.offsets[e + 1]), a), c.M);
            mine += static_cast<int>((b - a + BM - 1) / BM);
        }
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(sum, o);
            if (lane >= o) sum += up;
        }
        before = sum - mine;
        tiles = __builtin_amdgcn_readlane(sum, 63);
    } else {
        tiles = static_cast<int>((c.M + BM - 1) / BM);
    }
    const int64_t G = static_cast<int64_t>(tiles) * n_tn, id = blockIdx.x;
    if (id >= G) return false;
    const int64_t share = G / kMmXcds, rest = G % kMmXcds, x = id % kMmXcds;
    const int64_t q = x * share + (x < rest ? x : rest) + id / kMmXcds;
    const int64_t group = q / (static_cast<int64_t>(band) * n_tn);
    const int64_t in = q - group * band * n_tn;
    const int high = min(static_cast<int64_t>(band), tiles - group * band);    // the last band may be lower
    const int tm = static_cast<int>(group * band + in % high);
    out->tn = static_cast<int>(in / high);
    if (!c.offsets) {
        out->expert = 0;
        out->row0 = static_cast<int64_t>(tm) * BM;
        out->rows = static_cast<int>(min(static_cast<int64_t>(BM), c.M - out->row0));
        return true;
    }
    // the lane whose experts hold the row tile, then the expert
    const int from = __builtin_ctzll(__ballot(before + mine > tm));
    int left = tm - __builtin_amdgcn_readlane(before, from);
    for (int e = from * per;; ++e) {
        const int64_t a = min(max(static_cast<int64_t>(c.offsets[e]), static_cast<int64_t>(0)), c.M);
        const int64_t b = min(max(static_cast<int64_t>(c.offsets[e + 1]), a), c.M);
        const int n = static_cast<int>((b - a + BM - 1) / BM);
        if (left < n) {
            out->expert = e;
            out->row0 = a + static_cast<int64_t>(left) * BM;
            out->rows = static_cast<int>(min(static_cast<int64_t>(BM), b - out->row0));
            return true;
        }
        left -= n;
    }
}

// Row of x (and of its scales) that the tile's row r reads; -1: none.
__device__ __forceinline__ int64_t mm_row(const MatmulCall &c, const MmTile &t, int r) {
    if (r >= t.rows) return -1;
    const int64_t i = t.row0 + r;
    if (!c.order) return i;
    const int p = c.order[i];
    const int row = p / c.topk;
    return p >= 0 && row < c.x_rows ? row : -1;
}

// Rows of x are read at 32-bit offsets from the tile's first row, or from the
// start of x where the order picks them.
__device__ __forceinline__ int64_t mm_base(const MatmulCall &c, const MmTile &t) { return c.order ? 0 : t.row0; }

template <int BF16>
__device__ __forceinline__ void mm_store4(const MatmulCall &c, int64_t row, int n, const f32x4_t v) {
    // feature n is a multiple of four; rows of y need only their element's alignment
    typedef u32x4_t u32x4_m4_t __attribute__((aligned(4)));
    typedef u32x2_t u32x2_m2_t __attribute__((aligned(2)));
    if (n + 4 <= c.N) {
        if (BF16)
            *reinterpret_cast<u32x2_m2_t *>(static_cast<uint16_t *>(c.y) + row * c.ldy + n) =
                u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
            *reinterpret_cast<u32x4_m4_t *>(static_cast<float *>(c.y) + row * c.ldy + n) = __builtin_bit_cast(u32x4_t, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (n + e >= c.N) break;
        if (BF16) static_cast<uint16_t *>(c.y)[row * c.ldy + n + e] = static_cast<uint16_t>(pack_bf16x2(v[e], 0.f));
        else static_cast<float *>(c.y)[row * c.ldy + n + e] = v[e];
    }
}

// ------------------------------------------------------------------ tiles --
// BM rows x BN features by WM x WN waves. LDS holds two stages of 128 k: rows
// of 128 bytes, eight granules of 16, granule q of row r at q ^ sw(r), so that
// the sixteen rows of an operand fall on sixteen different bank groups. Loads
// that write LDS directly fill one stage while the other is multiplied.
//
// Features of a wave are dealt to its blocks so that a pair of blocks gives a
// lane eight neighbouring ones: row r of block b is feature
// 32 (b / 2) + 8 (r / 4) + 4 (b % 2) + r % 4.
__device__ __forceinline__ int mm_swx(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int mm_sww(int r) { return (r >> 1 & 1) | (r >> 3 & 3) << 1; }

template <int BM, int BN, int WM, int WN, int BF16>
__device__ __forceinline__ void mm_tile_body(const MatmulCall &c, const MmTile &t, char *s0, char *s1) {
    constexpr int WIDE = !BF16, WAVES = WM * WN, RT = BM / WM / 16, FT = BN / WN / 16;
    constexpr int XI = BM / 8 / WAVES, WI = BN / 8 / WAVES;      // 1 KB loads of a wave per stage
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && 128 % (16 * FT) == 0, "whole loads, one scale");
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int n0 = t.tn * BN;
    const int64_t base = mm_base(c, t);
    const int kb = (c.K + kMmK - 1) / kMmK, nb = (c.N + 127) / 128;
    const __amdgpu_buffer_rsrc_t x_rs = mm_view(c.x + base * c.ldx);
    const __amdgpu_buffer_rsrc_t xs_rs = mm_view(c.xs + base * kb);
    const __amdgpu_buffer_rsrc_t w_rs = mm_view(c.w + (static_cast<int64_t>(t.expert) * c.N + n0) * c.ldw);
    const int fb = min((n0 + wn * 16 * FT) / 128, nb - 1);        // the wave's block of features
    const __amdgpu_buffer_rsrc_t ws_rs = mm_view(c.ws + (static_cast<int64_t>(t.expert) * nb + fb) * kb);

    // the stage's loads: instruction i of a wave fills eight rows
    uint32_t x_off[XI], w_off[WI];
    int x_q[XI], w_q[WI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int r = 8 * (XI * wave + i) + (lane >> 3);
        const int64_t row = mm_row(c, t, r);
        x_q[i] = (lane & 7) ^ mm_swx(r);
        x_off[i] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * c.ldx + 16 * x_q[i]);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int r = 8 * (WI * wave + i) + (lane >> 3);
        w_q[i] = (lane & 7) ^ mm_sww(r);
        w_off[i] = n0 + r >= c.N ? kMmOob : static_cast<uint32_t>(static_cast<int64_t>(r) * c.ldw + 16 * w_q[i]);
    }
    // scales: of a lane's rows (one per 16-row block), and of the wave's features
    uint32_t xs_off[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int64_t row = mm_row(c, t, wm * 16 * RT + 16 * j + i16);
        xs_off[j] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * kb * 4);
    }
    float xs[2][RT], ws[2];
    auto issue = [&](int b, auto stage_c) {
        constexpr int S = decltype(stage_c)::value;
        char *st = S ? s1 : s0;
        const int left = c.K - b * kMmK;        // <= 0 behind the last block: all of it zeros
        const int step = left > 0 ? b * kMmK : 0, at = left > 0 ? 4 * b : 0;
#pragma unroll
        for (int j = 0; j < RT; ++j) xs[S][j] = mm_load4(xs_rs, left > 0 ? xs_off[j] : kMmOob, at);
        ws[S] = mm_load4(ws_rs, left > 0 ? 0u : kMmOob, at);
#pragma unroll
        for (int i = 0; i < XI; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x_rs, (lds_void_t *)(st + (XI * wave + i) * 1024), 16,
                                                     16 * x_q[i] < left ? x_off[i] : kMmOob, step, 0, 0);
#pragma unroll
        for (int i = 0; i < WI; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rs, (lds_void_t *)(st + BM * kMmK + (WI * wave + i) * 1024), 16,
                                                     16 * w_q[i] < left ? w_off[i] : kMmOob, step, 0, 0);
    };
    f32x4_t acc[FT][RT];
#pragma unroll
    for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[f][j] = zero_f32x4();

    // operands in a stage: rows of one operand lie at constant distances, as
    // what the granules are permuted by is the same for all of a lane's rows
    int x_at[2], w_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int rx = wm * 16 * RT + i16, rw = wn * 16 * FT + 8 * (i16 >> 2) + (i16 & 3);
        x_at[h] = rx * kMmK + (((2 * g + h) ^ mm_swx(rx)) << 4);
        w_at[h] = rw * kMmK + (((2 * g + h) ^ mm_sww(rw)) << 4);
    }
    auto multiply = [&](auto stage_c) {
        constexpr int S = decltype(stage_c)::value;
        const char *X = S ? s1 : s0, *W = X + BM * kMmK;
        MmOperand<WIDE> xf[RT];
        float s[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            xf[j] = mm_operand<WIDE>(load_u32x4(X + x_at[0] + 16 * j * kMmK), load_u32x4(X + x_at[1] + 16 * j * kMmK));
            s[j] = xs[S][j] * ws[S];
        }
        auto w_frag = [&](int f) {
            const char *at = W + (32 * (f / 2) + 4 * (f % 2)) * kMmK;
            return mm_operand<WIDE>(load_u32x4(at + w_at[0]), load_u32x4(at + w_at[1]));
        };
        // the products of one block of features while those of the one before
        // are scaled and added
        MmOperand<WIDE> wf[2];
        f32x4_t p[2][RT];
        wf[0] = w_frag(0);
#pragma unroll
        for (int f = 0; f <= FT; ++f) {
            if (f + 1 < FT) wf[(f + 1) & 1] = w_frag(f + 1);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                if (f < FT) p[f & 1][j] = mm_product<WIDE>(wf[f & 1], xf[j]);
                if (f > 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[f - 1][j][e] = fmaf(s[j], p[(f - 1) & 1][j][e], acc[f - 1][j][e]);
                    asm volatile("" : "+v"(acc[f - 1][j]));      // here, not past the block's end
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    // per block: its loads have landed (all of them were issued a block ago)
    // and every wave has read the stage that the next block's loads fill
    auto turn = [&](int b, auto here, auto next) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) expcnt(7) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(b + 1, next);
        multiply(here);
    };
    issue(0, I0{});
    for (int b = 0;; b += 2) {
        turn(b, I0{}, I1{});
        if (b + 1 >= kb) break;
        turn(b + 1, I1{}, I0{});
        if (b + 2 >= kb) break;
    }
    __builtin_amdgcn_s_waitcnt(0x0070);       // the last stage's zeros have landed
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int r = wm * 16 * RT + 16 * j + i16;
        if (r >= t.rows) continue;
#pragma unroll
        for (int f = 0; f < FT; ++f) {
            const int n = n0 + wn * 16 * FT + 32 * (f / 2) + 8 * g + 4 * (f % 2);
            mm_store4<BF16>(c, t.row0 + r, n, acc[f][j]);
        }
    }
}

template <int BM, int BN, int WM, int WN, int BF16>
__global__ __launch_bounds__(64 * WM * WN) void mm_tile_kernel(MatmulCall c, int n_tn, int band) {
    __shared__ __attribute__((aligned(16))) char s0[(BM + BN) * kMmK];
    __shared__ __attribute__((aligned(16))) char s1[(BM + BN) * kMmK];
    MmTile t;
    if (!mm_tile<BM>(c, n_tn, band, &t)) return;
    mm_tile_body<BM, BN, WM, WN, BF16>(c, t, s0, s1);
}

// --------------------------------------------------------------- few rows --
// Up to 16 RT rows: w is read once and sets the time, so it goes from memory
// to the registers of the matrix instructions. A workgroup has 16 features;
// its waves take the blocks of k in turn and their sums are added in LDS.
template <int RT, int WAVES, int BF16>
__global__ __launch_bounds__(64 * WAVES) void mm_rows_kernel(MatmulCall c, int n_tn, int band) {
    constexpr int WIDE = !BF16, BM = 16 * RT, AHEAD = RT > 2 ? 2 : 4;
    __shared__ f32x4_t part[WAVES][RT][64];
    MmTile t;
    if (!mm_tile<BM>(c, n_tn, band, &t)) return;
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = t.tn * 16;
    const int64_t base = mm_base(c, t);
    const int kb = (c.K + kMmK - 1) / kMmK, nb = (c.N + 127) / 128;
    const __amdgpu_buffer_rsrc_t x_rs = mm_view(c.x + base * c.ldx);
    const __amdgpu_buffer_rsrc_t xs_rs = mm_view(c.xs + base * kb);
    const __amdgpu_buffer_rsrc_t w_rs = mm_view(c.w + (static_cast<int64_t>(t.expert) * c.N + n0) * c.ldw);
    const __amdgpu_buffer_rsrc_t ws_rs = mm_view(c.ws + (static_cast<int64_t>(t.expert) * nb + n0 / 128) * kb);
    const uint32_t w_off = n0 + i16 < c.N ? static_cast<uint32_t>(static_cast<int64_t>(i16) * c.ldw + 32 * g) : kMmOob;
    uint32_t x_off[RT], xs_off[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int64_t row = mm_row(c, t, 16 * j + i16);
        x_off[j] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * c.ldx + 32 * g);
        xs_off[j] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * kb * 4);
    }
    f32x4_t acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = zero_f32x4();
    for (int b0 = wave; b0 < kb; b0 += AHEAD * WAVES) {
        u32x4_t w[AHEAD][2], x[AHEAD][RT][2];
        float s[AHEAD][RT], ws[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int b = b0 + a * WAVES, left = c.K - b * kMmK;      // <= 0 behind the last block
            const int step = left > 0 ? b * kMmK : 0, at = left > 0 ? 4 * b : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[a][h] = mm_load16(w_rs, 32 * g + 16 * h < left ? w_off + 16 * h : kMmOob, step);
            ws[a] = mm_load4(ws_rs, left > 0 ? 0u : kMmOob, at);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[a][j][h] = mm_load16(x_rs, 32 * g + 16 * h < left && x_off[j] != kMmOob ? x_off[j] + 16 * h : kMmOob, step);
                s[a][j] = mm_load4(xs_rs, left > 0 ? xs_off[j] : kMmOob, at);
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const MmOperand<WIDE> wo = mm_operand<WIDE>(w[a][0], w[a][1]);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const f32x4_t p = mm_product<WIDE>(wo, mm_operand<WIDE>(x[a][j][0], x[a][j][1]));
                const float f = s[a][j] * ws[a];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(f, p[e], acc[j][e]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) part[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < RT; j += WAVES) {
        f32x4_t sum = part[0][j][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += part[w][j][lane];
        const int r = 16 * j + i16;
        if (r < t.rows && n0 + 4 * g < c.N) mm_store4<BF16>(c, t.row0 + r, n0 + 4 * g, sum);
    }
}

// Row tiles at most: every expert but as many as there are rows may have a
// part of one.
static int64_t mm_row_tiles(int64_t M, int E, int bm) {
    return E ? M / bm + (M < E ? M : E) : (M + bm - 1) / bm;
}

template <int RT, int WAVES>
static void mm_rows(const MatmulCall &c, hipStream_t st) {
    const int n_tn = (c.N + 15) / 16;
    const dim3 grid(static_cast<uint32_t>(mm_row_tiles(c.M, c.offsets ? c.E : 0, 16 * RT) * n_tn)), block(64 * WAVES);
    if (c.y_bf16) hipLaunchKernelGGL((mm_rows_kernel<RT, WAVES, 1>), grid, block, 0, st, c, n_tn, 1);
    else hipLaunchKernelGGL((mm_rows_kernel<RT, WAVES, 0>), grid, block, 0, st, c, n_tn, 1);
}

template <int BM, int BN, int WM, int WN, int BF16>
static void mm_tiles(const MatmulCall &c, int band, hipStream_t st) {
    const int n_tn = (c.N + BN - 1) / BN;
    const dim3 grid(static_cast<uint32_t>(mm_row_tiles(c.M, c.offsets ? c.E : 0, BM) * n_tn)), block(64 * WM * WN);
    hipLaunchKernelGGL((mm_tile_kernel<BM, BN, WM, WN, BF16>), grid, block, 0, st, c, n_tn, band);
}

// A launch has fewer than 2^32 threads; the smallest tiles are 16 x 16 of 256.
bool fp8_matmul_fits(int64_t M, int64_t N, int E) {
    return mm_row_tiles(M, E, 16) < (1ll << 23) / ((N + 15) / 16);
}

hipError_t launch_fp8_matmul(const MatmulCall &c, hipStream_t st) {
    const int64_t per = c.offsets ? (c.M + c.E - 1) / c.E : c.M;     // rows of an expert
    const int band = c.offsets ? 2 : 8;
    if (per <= 16) mm_rows<1, 4>(c, st);
    else if (per <= 32) mm_rows<2, 4>(c, st);
    else if (!c.y_bf16) mm_tiles<128, 128, 2, 2, 0>(c, band, st);
    else if (per <= 128) mm_tiles<128, 128, 2, 2, 1>(c, band, st);
    else mm_tiles<256, 256, 4, 2, 1>(c, band, st);
    return hipGetLastError();
}

}  // namespace logra
