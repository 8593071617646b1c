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
//
// Measured, Y in bf16: 4096 rows, n 18944, k 3584 (556 GFLOP) 280 us, 2.0
// PFLOP/s; 4096 tokens to 8 of 128 experts, n 768, k 2048 (103 GFLOP, 260 MB) 95
// us; one row, n 18944, k 3584 (68 MB) 14 us, 4.8 TB/s.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace logra {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char_t;

constexpr uint32_t kMmOob = 0x80000000u;      // past every buffer view: loads give zeros
constexpr int kMmK = 128;
constexpr int kMmXcds = 8;
constexpr int kMmGrid = 256;                   // one workgroup for each compute unit
constexpr int kMmList = 64;                    // tiles in a workgroup's list
constexpr int kMmTiles = 1 << 23;              // tiles of a product are numbered below this

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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_view(const void *p, int64_t bytes = 0x7FFFFFFF) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             static_cast<int>(min(bytes, static_cast<int64_t>(0x7FFFFFFF))), 0x00020000);
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

// The tiles of a product: row tiles of all experts, times feature tiles.
struct MmPlan {
    int tiles, n_tn, band;        // row tiles, feature tiles
    int per, mine, before;        // experts of a lane, their row tiles, and those before them
};

__device__ __forceinline__ void mm_rows_of(const MatmulCall &c, int e, int64_t *a, int64_t *b) {
    *a = min(max(static_cast<int64_t>(c.offsets[e]), static_cast<int64_t>(0)), c.M);
    *b = min(max(static_cast<int64_t>(c.offsets[e + 1]), *a), c.M);
}

template <int BM>
__device__ __forceinline__ MmPlan mm_plan(const MatmulCall &c, int n_tn, int band) {
    const int lane = threadIdx.x & 63;
    MmPlan p{0, n_tn, band, 1, 0, 0};
    if (!c.offsets) {
        p.tiles = static_cast<int>((c.M + BM - 1) / BM);
        return p;
    }
    p.per = (c.E + 63) / 64;
    for (int i = 0; i < p.per; ++i) {
        const int e = lane * p.per + i;
        if (e >= c.E) break;
        int64_t a, b;
        mm_rows_of(c, e, &a, &b);
        p.mine += static_cast<int>((b - a + BM - 1) / BM);
    }
    // offsets that decrease somewhere give rows to several experts and could give
    // more tiles than can be numbered: those left out are not written
    p.mine = min(p.mine, kMmTiles);
    int sum = p.mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(sum, o);
        if (lane >= o) sum += up;
    }
    p.before = sum - p.mine;
    p.tiles = min(__builtin_amdgcn_readlane(sum, 63), (kMmTiles - 1) / n_tn);
    return p;
}

// Numbers below 2^24 are divided in a few instructions where the compiler sees that they are.
__device__ __forceinline__ uint32_t mm_div(uint32_t a, uint32_t b) { return (a & 0xFFFFFF) / (b & 0xFFFFFF); }

// Tile id (any of 0 .. tiles n_tn - 1; workgroups take ids a grid apart, which
// is a multiple of eight where there are several). Ids of one XCD (id mod 8)
// have neighbouring tiles, `band` row tiles by as many feature tiles as there
// are workgroups, so that they read the same rows of x and w through the XCD's
// cache. Lanes may ask for different ids, all 64 together; no rows: no such
// tile.
template <int BM>
__device__ __forceinline__ MmTile mm_tile(const MatmulCall &c, const MmPlan &p, uint32_t id) {
    const uint32_t n_tn = p.n_tn, G = static_cast<uint32_t>(p.tiles) * n_tn;      // below kMmTiles
    const bool is = id < G;
    if (!is) id = 0;
    const uint32_t share = G / kMmXcds, rest = G % kMmXcds, x = id % kMmXcds;
    const uint32_t q = x * share + min(x, rest) + id / kMmXcds;
    const uint32_t group = mm_div(q, p.band * n_tn), in = q - group * p.band * n_tn;
    const uint32_t high = max(min(p.band, p.tiles - static_cast<int>(group) * p.band), 1);      // the last band may be lower
    const uint32_t tn = mm_div(in, high);
    const int tm = static_cast<int>(group * p.band + in - tn * high);
    MmTile t{0, 0, static_cast<int>(tn), static_cast<int64_t>(tm) * BM};
    if (!c.offsets) {
        if (is) t.rows = static_cast<int>(min(static_cast<int64_t>(BM), c.M - t.row0));
        return t;
    }
    // the first lane whose experts end behind the row tile, then the expert
    int from = 0;
#pragma unroll
    for (int h = 32; h; h >>= 1)
        if (__shfl(p.before + p.mine, from + h - 1) <= tm) from += h;
    int left = tm - __shfl(p.before, from);
    for (int e = from * p.per; e < min((from + 1) * p.per, c.E); ++e) {
        int64_t a, b;
        mm_rows_of(c, e, &a, &b);
        const int n = static_cast<int>((b - a + BM - 1) / BM);
        if (left >= 0 && left < n && is) {
            t.expert = e;
            t.row0 = a + static_cast<int64_t>(left) * BM;
            t.rows = static_cast<int>(min(static_cast<int64_t>(BM), b - t.row0));
        }
        left -= n;
    }
    return t;
}

// A tile that all lanes have alike.
__device__ __forceinline__ MmTile mm_uniform(const MmTile &t) {
    return MmTile{__builtin_amdgcn_readfirstlane(t.expert), __builtin_amdgcn_readfirstlane(t.rows), __builtin_amdgcn_readfirstlane(t.tn),
                  __builtin_amdgcn_readfirstlane(static_cast<int>(t.row0))};
}

// Row of x (and of its scales) that the tile's row r reads, with what the order
// says of it; -1: none.
__device__ __forceinline__ int64_t mm_row(const MatmulCall &c, const MmTile &t, int r, int p) {
    if (r >= t.rows) return -1;
    if (!c.order) return t.row0 + r;
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

// Eight neighbouring features of a row in bf16 (n a multiple of eight).
__device__ __forceinline__ void mm_store8(const MatmulCall &c, int64_t row, int n, const f32x4_t a, const f32x4_t b) {
    typedef u32x4_t u32x4_m2_t __attribute__((aligned(2)));
    uint16_t *dst = static_cast<uint16_t *>(c.y) + row * c.ldy + n;
    const u32x4_t v = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
    if (n + 8 <= c.N) {
        *reinterpret_cast<u32x4_m2_t *>(dst) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (n + e < c.N) dst[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e % 2)));
}

// ------------------------------------------------------------------ tiles --
// BM rows x BN features by WM x WN waves. LDS is a ring of D stages of 128 k:
// rows of 128 bytes, eight granules of 16, granule q of row r at q ^ sw(r), so
// that the sixteen rows of an operand fall on sixteen different bank groups;
// lanes 16 g .. read granules g and 4 + g (with 2 g and 2 g + 1 the reads took
// twice as long: the LDS takes lanes of several g together).
//
// Features of a wave are dealt to its blocks so that a pair of blocks gives a
// lane eight neighbouring ones: row r of block b is feature
// 32 (b / 2) + 8 (r / 4) + 4 (b % 2) + r % 4.
//
// A workgroup goes from tile to tile, and its loads run D - 1 blocks ahead of
// its products, into the next tile too: its first blocks come while the last
// ones of this tile are multiplied and its results are written. Nothing on the
// way waits for a load of its own: a list in LDS holds the workgroup's next
// tiles, and what the order says of a tile's rows comes into LDS a tile ahead.
// (With both looked up where a tile began, 32768 rows of 128 experts, n 768, k
// 2048, took 97 us, as many rows of one expert 67.)
__device__ __forceinline__ int mm_swx(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int mm_sww(int r) { return (r >> 1 & 1) | (r >> 3 & 3) << 1; }

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_t mm_words(const void *p, int64_t bytes = 0x7FFFFFFF) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return i32x4_t{__builtin_amdgcn_readfirstlane(static_cast<int>(a)), __builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32 & 0xFFFF)),
                   __builtin_amdgcn_readfirstlane(static_cast<int>(min(bytes, static_cast<int64_t>(0x7FFFFFFF)))), 0x00020000};
}

__device__ __forceinline__ i32x4_t mm_scalar(i32x4_t v) {
    return i32x4_t{__builtin_amdgcn_readfirstlane(v[0]), __builtin_amdgcn_readfirstlane(v[1]), __builtin_amdgcn_readfirstlane(v[2]),
                   __builtin_amdgcn_readfirstlane(v[3])};
}

// 16 bytes per lane from the view at off + step straight into LDS at `to`
// (lane order; out of the view: zeros). Written out so that the compiler does
// not wait for all of them at the next LDS read, as it does for the builtin
// where it cannot tell the stages apart: who reads waits (mm_wait) before.
__device__ __forceinline__ void mm_fetch(i32x4_t view, uint32_t to, uint32_t off, int step) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(mm_scalar(view)), "s"(__builtin_amdgcn_readfirstlane(step))
                 : "m0", "memory");
}

// The same of 4 bytes per lane.
__device__ __forceinline__ void mm_fetch4(i32x4_t view, uint32_t to, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(mm_scalar(view))
                 : "m0", "memory");
}

// At most N vector memory operations of the wave are left, its LDS reads are
// done; then all waves of the workgroup are here.
template <int N>
__device__ __forceinline__ void mm_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int BM, int BN, int WM, int WN, int D>
struct MmShape {
    static constexpr int WAVES = WM * WN, RT = BM / WM / 16, FT = BN / WN / 16;
    static constexpr int STAGE = (BM + BN) * kMmK;
    // scales of eight blocks of k: of the rows, then of the features' blocks
    static constexpr int SCALES = BM * 32 + BN / 4;
    static constexpr int XI = BM / 8 / WAVES, WI = BN / 8 / WAVES;       // 1 KB loads of a wave for a block
    static constexpr int SI = (BM / 32 + WAVES - 1) / WAVES;             // and for eight blocks' scales
    // the next tiles, and the order's entries of two tiles' rows
    static constexpr int LIST = D * (STAGE + SCALES), ROWS = LIST + kMmList * 16, ROWS_EACH = (BM < 64 ? 64 : BM) * 4;
    static constexpr int LDS = ROWS + 2 * ROWS_EACH;
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && 128 % (16 * FT) == 0, "whole loads, one scale");
    static_assert(LDS <= 160 * 1024 && (D - 2) * (XI + WI) < 64, "what a compute unit has, what a wait can count");
};

template <int BM, int BN, int WM, int WN, int D, int BF16>
__global__ __launch_bounds__(64 * WM * WN) void mm_tile_kernel(MatmulCall c, int n_tn, int band) {
    using Sh = MmShape<BM, BN, WM, WN, D>;
    constexpr int WIDE = !BF16, RT = Sh::RT, FT = Sh::FT, XI = Sh::XI, WI = Sh::WI, SI = Sh::SI;
    __shared__ __attribute__((aligned(16))) char lds[Sh::LDS];
    const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t *)lds)), scales = ring + D * Sh::STAGE;
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int kb = (c.K + kMmK - 1) / kMmK, nb = (c.N + 127) / 128;
    // tiles first .. first + count - 1 of this workgroup into the list
    auto list_tiles = [&](int first, int count) {
        const MmTile t = mm_tile<BM>(c, mm_plan<BM>(c, n_tn, band), blockIdx.x + gridDim.x * static_cast<uint32_t>(first + lane));
        if (lane < count)
            *reinterpret_cast<i32x4_t *>(lds + Sh::LIST + (first + lane) % kMmList * 16) = i32x4_t{t.expert, t.rows, t.tn, static_cast<int>(t.row0)};
    };
    auto tile = [&](int i) {
        const i32x4_t v = *reinterpret_cast<const i32x4_t *>(lds + Sh::LIST + i % kMmList * 16);
        return mm_uniform(MmTile{v[0], v[1], v[2], v[3]});
    };
    auto fetch_rows = [&](int i) {
        const MmTile t = tile(i);
        if (c.order && wave < (BM + 63) / 64 && t.rows)
            mm_fetch4(mm_words(c.order + t.row0, 4 * t.rows), ring + Sh::ROWS + i % 2 * Sh::ROWS_EACH + wave * 256, 4 * (64 * wave + lane));
    };

    // what is fetched: tile, block, and their places in the two rings
    int f_i = 0, f_b = 0, f_stage = 0, f_place = 0;
    bool f_more;
    i32x4_t x_rs, xs_rs, w_rs, ws_rs;
    uint32_t x_off[XI], w_off[WI], xs_off[SI], ws_off;
    auto enter = [&]() {
        // the list's half whose tiles are done; the others read it 16 tiles on
        if (f_i % (kMmList / 2) == 16 && wave == 0) list_tiles(f_i + 16, kMmList / 2);
        // its rows were asked for a tile before: with so few blocks they may not be here
        if (c.order && kb < D) mm_wait<0>();
        const MmTile t = tile(f_i);
        f_more = t.rows > 0;
        if (!f_more) return;
        const int *order = reinterpret_cast<const int *>(lds + Sh::ROWS + f_i % 2 * Sh::ROWS_EACH);
        fetch_rows(f_i + 1);
        const int n0 = t.tn * BN;
        const int64_t base = mm_base(c, t);
        x_rs = mm_words(c.x + base * c.ldx);
        // x without rows: one row's length, as a step behind a view of nothing would
        // make its end wrap around
        xs_rs = mm_words(c.xs + base * kb, max(c.x_rows - base, static_cast<int64_t>(1)) * kb * 4);
        w_rs = mm_words(c.w + (static_cast<int64_t>(t.expert) * c.N + n0) * c.ldw);
        const int64_t fb = static_cast<int64_t>(t.expert) * nb + n0 / 128;      // the tile's first block of features
        ws_rs = mm_words(c.ws + fb * kb, (static_cast<int64_t>(c.E) * nb - fb) * kb * 4);
        // instruction i of a wave fills eight rows
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int r = 8 * (XI * wave + i) + (lane >> 3);
            const int64_t row = mm_row(c, t, r, order[r]);
            x_off[i] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * c.ldx + 16 * ((lane & 7) ^ mm_swx(r)));
        }
#pragma unroll
        for (int i = 0; i < WI; ++i) {
            const int r = 8 * (WI * wave + i) + (lane >> 3);
            w_off[i] = n0 + r >= c.N ? kMmOob : static_cast<uint32_t>(static_cast<int64_t>(r) * c.ldw + 16 * ((lane & 7) ^ mm_sww(r)));
        }
        // scales: two lanes a row
#pragma unroll
        for (int i = 0; i < SI; ++i) {
            const int r = 32 * (SI * wave + i) + (lane >> 1);
            const int64_t row = r < BM ? mm_row(c, t, r, order[r]) : -1;
            xs_off[i] = row < 0 ? kMmOob : static_cast<uint32_t>(((row - base) * kb + 4 * (lane & 1)) * 4);
        }
        ws_off = static_cast<uint32_t>(((lane >> 1) * kb + 4 * (lane & 1)) * 4);
    };
    // The loads of a block in XI + WI pieces (behind the last tile: zeros, so
    // that every wait finds as many), and the scales before every eighth.
    auto fetch_scales = [&]() {
        if ((f_b & 7) != 0 || !f_more) return;
        const uint32_t to = scales + f_place * Sh::SCALES;
#pragma unroll
        for (int i = 0; i < SI; ++i)
            if (SI * Sh::WAVES * 32 == BM || SI * wave + i < BM / 32)
                mm_fetch(xs_rs, to + (SI * wave + i) * 1024, xs_off[i], 4 * f_b);
        if (wave == Sh::WAVES - 1 && lane < BN / 64) mm_fetch(ws_rs, to + BM * 32, ws_off, 4 * f_b);
    };
    auto fetch_piece = [&](int i) {
        const uint32_t to = ring + f_stage * Sh::STAGE;
        const int left = f_more ? c.K - f_b * kMmK : 0;
        if (i < XI) {
            const int q = 16 * ((lane & 7) ^ mm_swx(8 * (XI * wave + i) + (lane >> 3)));
            mm_fetch(x_rs, to + (XI * wave + i) * 1024, q < left ? x_off[i] : kMmOob, f_b * kMmK);
        } else {
            const int q = 16 * ((lane & 7) ^ mm_sww(8 * (WI * wave + i - XI) + (lane >> 3)));
            mm_fetch(w_rs, to + BM * kMmK + (WI * wave + i - XI) * 1024, q < left ? w_off[i - XI] : kMmOob, f_b * kMmK);
        }
    };
    auto fetched = [&]() {
        f_stage = f_stage + 1 == D ? 0 : f_stage + 1;
        if (!f_more) return;
        ++f_b;
        if ((f_b & 7) == 0 || f_b == kb) f_place = f_place + 1 == D ? 0 : f_place + 1;
        if (f_b == kb) {
            f_b = 0;
            ++f_i;
            enter();
        }
    };

    // operands in a stage: rows of one operand lie at constant distances, as
    // what the granules are permuted by is the same for all of a lane's rows
    int x_at[2], w_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int rx = wm * 16 * RT + i16, rw = wn * 16 * FT + 8 * (i16 >> 2) + (i16 & 3);
        x_at[h] = rx * kMmK + (((g + 4 * h) ^ mm_swx(rx)) << 4);
        w_at[h] = (BM + rw) * kMmK + (((g + 4 * h) ^ mm_sww(rw)) << 4);
    }
    const int xs_at = (wm * 16 * RT + i16) * 32, ws_at = BM * 32 + wn * 16 * FT / 128 * 32;
    f32x4_t acc[FT][RT];
    auto clear = [&]() {
#pragma unroll
        for (int f = 0; f < FT; ++f)
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[f][j] = zero_f32x4();
    };
    // One block: the operands' LDS reads first, then the products of one block
    // of features while those of the one before are scaled and added, with the
    // loads of the block to come between them.
    auto multiply = [&](const char *st, const char *sc) {
        MmOperand<WIDE> xf[RT], wf[2];
        const char *X0 = st + x_at[0], *X1 = st + x_at[1], *W0 = st + w_at[0], *W1 = st + w_at[1];
        auto w_frag = [&](int f) {
            const int at = (32 * (f / 2) + 4 * (f % 2)) * kMmK;
            return mm_operand<WIDE>(load_u32x4(W0 + at), load_u32x4(W1 + at));
        };
        wf[0] = w_frag(0);
#pragma unroll
        for (int j = 0; j < RT; ++j) xf[j] = mm_operand<WIDE>(load_u32x4(X0 + 16 * j * kMmK), load_u32x4(X1 + 16 * j * kMmK));
        float s[RT];
        const float ws = *reinterpret_cast<const float *>(sc + ws_at);
#pragma unroll
        for (int j = 0; j < RT; ++j) s[j] = ws * *reinterpret_cast<const float *>(sc + xs_at + 16 * j * 32);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int EACH = FT > 2 ? (2 * (XI + WI) + FT - 1) / FT : (XI + WI + FT - 1) / FT;     // pieces a time
        f32x4_t p[2][RT];
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
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = f * EACH; i < (f + 1) * EACH && i < XI + WI; ++i) fetch_piece(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto write = [&](const MmTile &o) {
        const int n0 = o.tn * BN + wn * 16 * FT;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int r = wm * 16 * RT + 16 * j + i16;
            if (r >= o.rows) continue;
#pragma unroll
            for (int f = 0; f < FT; f += 2) {
                const int n = n0 + 16 * f + 8 * g;
                if constexpr (BF16) mm_store8(c, o.row0 + r, n, acc[f][j], acc[f + 1][j]);
                else {
                    mm_store4<0>(c, o.row0 + r, n, acc[f][j]);
                    mm_store4<0>(c, o.row0 + r, n + 4, acc[f + 1][j]);
                }
            }
        }
    };

    if (wave == 0) list_tiles(0, kMmList);
    __syncthreads();
    if (c.order) {
        fetch_rows(0);
        mm_wait<0>();
    }
    enter();
    if (!f_more) return;
    for (int i = 0; i < D - 1; ++i) {
        fetch_scales();
#pragma unroll
        for (int q = 0; q < XI + WI; ++q) fetch_piece(q);
        fetched();
    }
    clear();
    int i = 0, b = 0, stage = 0, place = 0;
    for (;;) {
        // this block's loads have landed (D - 2 blocks' are younger), and every
        // wave has read the block before, whose stage is filled next
        mm_wait<(D - 2) * (XI + WI)>();
        fetch_scales();
        multiply(lds + stage * Sh::STAGE, lds + D * Sh::STAGE + place * Sh::SCALES + (b & 7) * 4);
        fetched();
        stage = stage + 1 == D ? 0 : stage + 1;
        ++b;
        if ((b & 7) == 0 || b == kb) place = place + 1 == D ? 0 : place + 1;
        if (b == kb) {
            write(tile(i));
            if (!tile(++i).rows) break;
            clear();
            b = 0;
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0070);       // the zeros behind the last tile have landed: the LDS is free
}

// --------------------------------------------------------------- few rows --
// Up to 16 RT rows: w is read once and sets the time, so it goes from memory
// to the registers of the matrix instructions. A workgroup has 16 FT features;
// its waves take the blocks of k in turn, AHEAD of them at a time, and their
// sums are added in LDS.
template <int RT, int FT, int WAVES, int AHEAD, int BF16>
__global__ __launch_bounds__(64 * WAVES) void mm_rows_kernel(MatmulCall c, int n_tn) {
    constexpr int WIDE = !BF16, BM = 16 * RT;
    __shared__ f32x4_t part[WAVES][FT][RT][64];
    const MmTile t = mm_uniform(mm_tile<BM>(c, mm_plan<BM>(c, n_tn, 1), blockIdx.x));
    if (!t.rows) return;
    const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = t.tn * 16 * FT;
    const int64_t base = mm_base(c, t);
    const int kb = (c.K + kMmK - 1) / kMmK, nb = (c.N + 127) / 128;
    const __amdgpu_buffer_rsrc_t x_rs = mm_view(c.x + base * c.ldx);
    const __amdgpu_buffer_rsrc_t xs_rs = mm_view(c.xs + base * kb);
    const __amdgpu_buffer_rsrc_t w_rs = mm_view(c.w + (static_cast<int64_t>(t.expert) * c.N + n0) * c.ldw);
    const __amdgpu_buffer_rsrc_t ws_rs = mm_view(c.ws + (static_cast<int64_t>(t.expert) * nb + n0 / 128) * kb);
    uint32_t w_off[FT], x_off[RT], xs_off[RT];
#pragma unroll
    for (int f = 0; f < FT; ++f)
        w_off[f] = n0 + 16 * f + i16 < c.N ? static_cast<uint32_t>(static_cast<int64_t>(16 * f + i16) * c.ldw + 32 * g) : kMmOob;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int r = 16 * j + i16;
        const int64_t row = mm_row(c, t, r, c.order && r < t.rows ? c.order[t.row0 + r] : 0);
        x_off[j] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * c.ldx + 32 * g);
        xs_off[j] = row < 0 ? kMmOob : static_cast<uint32_t>((row - base) * kb * 4);
    }
    f32x4_t acc[FT][RT];
#pragma unroll
    for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[f][j] = zero_f32x4();
    for (int b0 = wave; b0 < kb; b0 += AHEAD * WAVES) {
        u32x4_t w[AHEAD][FT][2], x[AHEAD][RT][2];
        float s[AHEAD][RT], ws[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int b = b0 + a * WAVES, left = c.K - b * kMmK;      // <= 0 behind the last block
            const int step = left > 0 ? b * kMmK : 0, at = left > 0 ? 4 * b : 0;
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[a][f][h] = mm_load16(w_rs, 32 * g + 16 * h < left && w_off[f] != kMmOob ? w_off[f] + 16 * h : kMmOob, step);
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
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const MmOperand<WIDE> xo = mm_operand<WIDE>(x[a][j][0], x[a][j][1]);
                const float m = s[a][j] * ws[a];
#pragma unroll
                for (int f = 0; f < FT; ++f) {
                    const f32x4_t p = mm_product<WIDE>(mm_operand<WIDE>(w[a][f][0], w[a][f][1]), xo);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[f][j][e] = fmaf(m, p[e], acc[f][j][e]);
                }
            }
    }
#pragma unroll
    for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int j = 0; j < RT; ++j) part[wave][f][j][lane] = acc[f][j];
    __syncthreads();
    for (int q = wave; q < RT * FT; q += WAVES) {
        const int f = q / RT, j = q % RT;
        f32x4_t sum = part[0][f][j][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += part[w][f][j][lane];
        const int r = 16 * j + i16, n = n0 + 16 * f + 4 * g;
        if (r < t.rows && n < c.N) mm_store4<BF16>(c, t.row0 + r, n, sum);
    }
}

// Row tiles at most: every expert but as many as there are rows may have a
// part of one.
static int64_t mm_row_tiles(int64_t M, int E, int bm) {
    return E ? M / bm + (M < E ? M : E) : (M + bm - 1) / bm;
}

template <int RT, int FT, int WAVES, int AHEAD, int BF16>
static void mm_rows(const MatmulCall &c, hipStream_t st) {
    const int n_tn = (c.N + 16 * FT - 1) / (16 * FT);
    const dim3 grid(static_cast<uint32_t>(mm_row_tiles(c.M, c.offsets ? c.E : 0, 16 * RT) * n_tn)), block(64 * WAVES);
    hipLaunchKernelGGL((mm_rows_kernel<RT, FT, WAVES, AHEAD, BF16>), grid, block, 0, st, c, n_tn);
}

template <int BM, int BN, int WM, int WN, int D, int BF16>
static void mm_tiles(const MatmulCall &c, int band, hipStream_t st) {
    const int n_tn = (c.N + BN - 1) / BN;
    const int64_t tiles = mm_row_tiles(c.M, c.offsets ? c.E : 0, BM) * n_tn;
    const dim3 grid(static_cast<uint32_t>(tiles < kMmGrid ? tiles : kMmGrid)), block(64 * WM * WN);
    hipLaunchKernelGGL((mm_tile_kernel<BM, BN, WM, WN, D, BF16>), grid, block, 0, st, c, n_tn, band);
}

// Those of 32 x 128 at least can be numbered.
bool fp8_matmul_fits(int64_t M, int64_t N, int E) { return mm_row_tiles(M, E, 32) < kMmTiles / ((N + 127) / 128); }

// Which kernel: the one expected to be done first. A product's tiles go to the
// compute units in rounds, and a round takes a start (the results' stores) and a
// step per block of k; both were measured for each shape (us; fp32 results take
// the shapes up to 128 x 256, whose steps are half as long again, each by about
// as much: 8192 rows, n 8960, k 1536 244, in 128 x 128 296). The rows kernels read w past the LDS and split k over the waves:
// their time follows the blocks a compute unit has to stream. Measured, us:
//   n 18944, k 3584: 4096 rows 275 in 256 x 256 tiles, 335 in 128 x 256; 256 rows
//   49 and 34; 128 rows 33 in 128 x 256, 24 in 128 x 128; 64 rows 23 in 128 x 128,
//   20 in 64 x 128; 24 rows 20 in 64 x 128, 17 in 32 x 128, 24.6 in rows of 32.
//   n 1536, k 8960: 512 rows 51 in 128 x 128, 43 in 64 x 128, 36 in 32 x 128; 64
//   rows 36 in 32 x 128, 16 in rows of 32.
//   128 experts, 8 choices, n 768, k 2048: 4096 tokens 95 in 128 x 256, 112 in 256
//   x 256 and in 128 x 128; 1024 tokens 53, 73 and 61; 256 tokens 44 in 32 x 128,
//   50 in 128 x 256, 69 in rows of 16; 16 tokens 23 and 23 in rows; 4 tokens 14
//   and 12. n 2048, k 768: 64 tokens 39 in 32 x 128, 70 in rows; one token 9 and 7.
struct MmShapeTime {
    int bm, bn;
    double step, start;
};
constexpr MmShapeTime kMmTimes[] = {{32, 128, 0.55, 0.8}, {64, 128, 0.66, 1.3}, {128, 128, 0.78, 2.0}, {128, 256, 1.12, 4.0}, {256, 256, 1.72, 7.0}};

hipError_t launch_fp8_matmul(const MatmulCall &c, hipStream_t st) {
    const double kb = (c.K + kMmK - 1) / kMmK;
    const int band = c.offsets ? 2 : 8;
    // Experts that have rows, were they chosen by chance, and their row tiles:
    // one at least, half of one left over where they have many.
    const double used = c.offsets ? c.E * (1 - exp(-static_cast<double>(c.M) / c.E)) : 1;
    const auto row_tiles = [&](int bm) {
        const double r = c.M / (used * bm);
        return c.offsets ? used * (r + 0.5 + 0.5 * exp(-2 * r)) : static_cast<double>((c.M + bm - 1) / bm);
    };
    double best, fill;
    if (c.offsets) {
        const double wgs = row_tiles(16) * ((c.N + 31) / 32);
        const bool fits = mm_row_tiles(c.M, c.E, 16) < kMmTiles / ((c.N + 31) / 32);
        best = fits ? 2.5 + wgs * (0.0045 * ceil(kb / 16) + 0.00045 * kb) : INFINITY;
        fill = 3.5;         // offsets, order and rows, one after the other
    } else if (c.M <= 16) {
        // one block of features for a workgroup while few rows make few loads
        // of x (n 18944, k 3584: 1 row 13.6 us with one, 15.2 with two; 16 rows
        // 19.8 and 18.5) or there are few workgroups (n 1536, k 8960: 1 row 8.7
        // and 12.1)
        if (c.N < 8192 || c.M <= 8) c.y_bf16 ? mm_rows<1, 1, 4, 8, 1>(c, st) : mm_rows<1, 1, 4, 8, 0>(c, st);
        else c.y_bf16 ? mm_rows<1, 2, 4, 4, 1>(c, st) : mm_rows<1, 2, 4, 4, 0>(c, st);
        return hipGetLastError();
    } else {
        const double wgs = row_tiles(32) * ((c.N + 15) / 16);
        const bool fits = mm_row_tiles(c.M, 0, 32) < kMmTiles / ((c.N + 15) / 16);
        best = fits ? kb * (wgs < 180 ? 0.15 : 0.00085 * wgs) : INFINITY;
        fill = 1.2;
    }
    int which = -1;
    for (int i = 0; i < (c.y_bf16 ? 5 : 4); ++i) {
        const MmShapeTime &m = kMmTimes[i];
        const double rounds = ceil(row_tiles(m.bm) * ((c.N + m.bn - 1) / m.bn) / kMmGrid);
        const double time = fill + rounds * (kb * m.step + m.start);
        if (time < best) {
            best = time;
            which = i;
        }
    }
    switch (which) {
    case -1:
        if (c.offsets) c.y_bf16 ? mm_rows<1, 2, 4, 4, 1>(c, st) : mm_rows<1, 2, 4, 4, 0>(c, st);
        else c.y_bf16 ? mm_rows<2, 1, 4, 4, 1>(c, st) : mm_rows<2, 1, 4, 4, 0>(c, st);
        break;
    case 0: c.y_bf16 ? mm_tiles<32, 128, 1, 4, 6, 1>(c, band, st) : mm_tiles<32, 128, 1, 4, 6, 0>(c, band, st); break;
    case 1: c.y_bf16 ? mm_tiles<64, 128, 1, 4, 5, 1>(c, band, st) : mm_tiles<64, 128, 1, 4, 5, 0>(c, band, st); break;
    case 2: c.y_bf16 ? mm_tiles<128, 128, 4, 2, 4, 1>(c, band, st) : mm_tiles<128, 128, 4, 2, 4, 0>(c, band, st); break;
    case 3: c.y_bf16 ? mm_tiles<128, 256, 2, 4, 3, 1>(c, band, st) : mm_tiles<128, 256, 2, 4, 3, 0>(c, band, st); break;
    default: mm_tiles<256, 256, 4, 2, 2, 1>(c, band, st);
    }
    return hipGetLastError();
}

}  // namespace logra
