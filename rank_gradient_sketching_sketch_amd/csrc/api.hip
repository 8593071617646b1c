// C ABI of liblogra.so: argument validation, per-step key derivation, work
// planning and kernel dispatch. Declarations and the contract of every entry
// point are in include/logra.h. Nothing here allocates memory or keeps state:
// every buffer, workspace included, comes from the caller.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "../../include/logra.h"
#include "launch.hpp"
#include "signs.hpp"

using namespace logra;

namespace {

// key = h(h(h(seed) ^ step) ^ matrix_id), h(x) = first SplitMix64 output of x.
uint64_t stream_key(uint64_t seed, uint64_t step, uint64_t matrix_id) {
    auto h = [](uint64_t x) { return splitmix_finalize(x + kGolden); };
    return h(h(h(seed) ^ step) ^ matrix_id);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool bf16_rank_ok(int64_t r) { return r == 32 || r == 64 || r == 128 || r == 256; }

bool matrix_ok(const logra_matrix *m) {
    return m && m->d > 0 && m->k > 0 && m->r > 0 && m->d <= (1ll << 30) && m->k <= (1ll << 30);
}

logra_status from_hip(hipError_t e) { return e == hipSuccess ? LOGRA_OK : LOGRA_ERR_HIP; }

float inv_sqrt_rank(int64_t r) { return 1.0f / sqrtf(static_cast<float>(r)); }

size_t sqnorm_ws_bytes(const logra_matrix *m, int compute_dtype) {
    if (compute_dtype == LOGRA_BF16) {
        const SqnormPlan p = plan_sqnorm_bf16(m->d, m->k, static_cast<int>(m->r));
        return p.partial_bytes + p.gram_bytes;
    }
    return static_cast<size_t>(apply_blocks_f32(m->d)) * sizeof(float);
}

// Buffer views address at most 2^31 bytes.
bool fits_view(int64_t rows, int64_t ld, int64_t elem) { return rows * ld * elem < (1ll << 31); }

// Launch options with their defaults filled in (NULL = all defaults).
struct Opts {
    int sketch_concurrency = 1;
    int apply_concurrency = 1;
    int backward_fold = 0;
    FoldWait wait;
};

bool read_opts(const logra_launch_opts *o, Opts *out) {
    Opts r;
    if (o) {
        if (o->backward_fold < 0 || o->backward_fold > 2) return false;
        r.backward_fold = o->backward_fold;
        if (o->sketch_concurrency < 0 || o->sketch_concurrency > 256) return false;
        if (o->apply_concurrency < 0 || o->apply_concurrency > 256) return false;
        if (o->sketch_concurrency > 0) r.sketch_concurrency = o->sketch_concurrency;
        if (o->apply_concurrency > 0) r.apply_concurrency = o->apply_concurrency;
        if (o->fold_wait_limit != 0) r.wait.spin_limit = o->fold_wait_limit;
        r.wait.timeouts = o->fold_timeouts;
    }
    *out = r;
    return true;
}

}  // namespace

// Scratch of logra_update_sqnorm_noalloc, for callers that cannot allocate:
// every device the library runs on holds its own copy until the process
// ends, and every call on that device shares it. In host code `scratch`
// names a host-side stand-in, never the device memory: the device address
// comes from hipGetSymbolAddress, once per device, and is kept in
// scratch_addr (a cache of a fixed address, written at most once per device
// with the value every caller would write).
constexpr size_t kNoallocScratchBytes = LOGRA_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char scratch[kNoallocScratchBytes];
constexpr int kMaxDevices = 64;
static std::atomic<void *> scratch_addr[kMaxDevices];

// The device address of this device's scratch, or null (with the HIP error
// in *err) if the current device cannot be queried.
static void *device_scratch(hipError_t *err) {
    int dev = -1;
    *err = hipGetDevice(&dev);
    if (*err != hipSuccess) return nullptr;
    if (dev < 0 || dev >= kMaxDevices) {
        *err = hipErrorInvalidDevice;
        return nullptr;
    }
    void *p = scratch_addr[dev].load(std::memory_order_acquire);
    if (p) return p;
    *err = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (*err != hipSuccess || !p) {
        if (*err == hipSuccess) *err = hipErrorInvalidSymbol;
        return nullptr;
    }
    scratch_addr[dev].store(p, std::memory_order_release);
    return p;
}

extern "C" {

int logra_abi_version(void) { return LOGRA_ABI_VERSION; }

const char *logra_status_string(int status) {
    switch (status) {
    case LOGRA_OK: return "LOGRA_OK";
    case LOGRA_ERR_INVALID_ARGUMENT: return "LOGRA_ERR_INVALID_ARGUMENT";
    case LOGRA_ERR_UNSUPPORTED: return "LOGRA_ERR_UNSUPPORTED";
    case LOGRA_ERR_WORKSPACE: return "LOGRA_ERR_WORKSPACE";
    case LOGRA_ERR_HIP: return "LOGRA_ERR_HIP";
    default: return "LOGRA_UNKNOWN_STATUS";
    }
}

logra_status logra_sign_words(const logra_matrix *m, uint64_t *words, void *stream) {
    if (!matrix_ok(m) || !words) return LOGRA_ERR_INVALID_ARGUMENT;
    if (m->r > (1ll << 20)) return LOGRA_ERR_UNSUPPORTED;
    const uint64_t key = stream_key(m->seed, m->step, m->matrix_id);
    return from_hip(launch_sign_words(key, static_cast<int>(m->r), static_cast<int>(m->k), words,
                                      static_cast<hipStream_t>(stream)));
}

size_t logra_sketch_workspace_bytes(const logra_matrix *m, int64_t T, int act_dtype) {
    if (!matrix_ok(m) || T < 0) return 0;
    if (T == 0) return 0;
    if (act_dtype == LOGRA_BF16) {
        if (!bf16_rank_ok(m->r)) return 0;
        const Stage1Plan p = plan_stage1_bf16(T, m->k, static_cast<int>(m->r));
        const FoldPlan f = plan_fold_bf16(T, m->d, static_cast<int>(m->r));
        return p.p_bytes + f.xbuf_bytes + f.sync_bytes;
    }
    if (act_dtype == LOGRA_F32) return workspace_sketch_f32(T, m->r);
    return 0;
}

static logra_status check_sketch(const logra_matrix *m, int64_t T, int act_dtype) {
    if (!matrix_ok(m) || T < 0) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype != LOGRA_F32 && act_dtype != LOGRA_BF16) return LOGRA_ERR_UNSUPPORTED;
    if (T > (1ll << 30)) return LOGRA_ERR_UNSUPPORTED;
    if (act_dtype == LOGRA_BF16) {
        if (!bf16_rank_ok(m->r) || m->d % 8 || m->k % 8) return LOGRA_ERR_UNSUPPORTED;
        // the projection (ceil(T/32) blocks of 32 tokens x r, bf16) is read
        // through a 32-bit buffer view
        if (!fits_view(T + 32, m->r, 2)) return LOGRA_ERR_UNSUPPORTED;
    } else if (m->r > 1024) {
        return LOGRA_ERR_UNSUPPORTED;
    }
    return LOGRA_OK;
}

static logra_status check_project(const logra_matrix *m, int64_t T, int act_dtype, const void *X,
                                  int64_t ldx, const void *ws, size_t ws_bytes) {
    if (T == 0) return LOGRA_OK;
    if (!X || ldx < m->k) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype == LOGRA_BF16 && (ldx % 8 || !aligned16(X))) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype == LOGRA_BF16 && !fits_view(T, ldx, 2)) return LOGRA_ERR_UNSUPPORTED;
    const size_t need = logra_sketch_workspace_bytes(m, T, act_dtype);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    return LOGRA_OK;
}

static logra_status check_fold(const logra_matrix *m, int64_t T, int act_dtype, const void *dY,
                               int64_t lddy, const float *S, const void *ws, size_t ws_bytes) {
    if (!S || !aligned16(S)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (T == 0) return LOGRA_OK;
    if (!dY || lddy < m->d) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype == LOGRA_BF16 && (lddy % 8 || !aligned16(dY))) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype == LOGRA_BF16 && (!fits_view(T + 32, lddy, 2) || !fits_view(m->d, m->r, 4 * 16)))
        return LOGRA_ERR_UNSUPPORTED;
    const size_t need = logra_sketch_workspace_bytes(m, T, act_dtype);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    return LOGRA_OK;
}

static hipError_t do_project(const logra_matrix *m, int64_t T, int act_dtype, const void *X,
                             int64_t ldx, void *ws, const Opts &o, hipStream_t st) {
    if (T == 0) return hipSuccess;
    const uint64_t key = stream_key(m->seed, m->step, m->matrix_id);
    const float c = inv_sqrt_rank(m->r);
    const int r = static_cast<int>(m->r);
    if (act_dtype == LOGRA_BF16)
        return launch_project_bf16(r, T, m->d, m->k, key, c, static_cast<const uint16_t *>(X), ldx, ws,
                                   o.sketch_concurrency, st);
    return launch_project_f32(r, T, m->k, key, c, static_cast<const float *>(X), ldx, ws, st);
}

static hipError_t do_fold(const logra_matrix *m, int64_t T, int act_dtype, const void *dY,
                          int64_t lddy, float *S, int accumulate, void *ws, const Opts &o, hipStream_t st) {
    if (T == 0) return accumulate ? hipSuccess : launch_fill_zero(S, m->d * m->r, st);
    const int r = static_cast<int>(m->r);
    if (act_dtype == LOGRA_BF16)
        return launch_fold_bf16(r, T, m->d, m->k, static_cast<const uint16_t *>(dY), lddy, S,
                                accumulate ? 1 : 0, ws, o.wait, st);
    return launch_fold_f32(r, T, m->d, static_cast<const float *>(dY), lddy, S, accumulate ? 1 : 0,
                           ws, st);
}

logra_status logra_sketch_project(const logra_matrix *m, int64_t T, int act_dtype, const void *X,
                                  int64_t ldx, void *ws, size_t ws_bytes, const logra_launch_opts *opts,
                                  void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_sketch(m, T, act_dtype);
    if (e == LOGRA_OK) e = check_project(m, T, act_dtype, X, ldx, ws, ws_bytes);
    if (e != LOGRA_OK) return e;
    return from_hip(do_project(m, T, act_dtype, X, ldx, ws, o, static_cast<hipStream_t>(stream)));
}

logra_status logra_sketch_fold(const logra_matrix *m, int64_t T, int act_dtype, const void *dY,
                               int64_t lddy, float *S, int accumulate, void *ws,
                               size_t ws_bytes, const logra_launch_opts *opts, void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_sketch(m, T, act_dtype);
    if (e == LOGRA_OK) e = check_fold(m, T, act_dtype, dY, lddy, S, ws, ws_bytes);
    if (e != LOGRA_OK) return e;
    return from_hip(do_fold(m, T, act_dtype, dY, lddy, S, accumulate, ws, o,
                            static_cast<hipStream_t>(stream)));
}

size_t logra_sketch_parts_bytes(const logra_matrix *m, int64_t T, int act_dtype) {
    if (check_sketch(m, T, act_dtype) != LOGRA_OK || T == 0 || act_dtype != LOGRA_BF16) return 0;
    return fold_parts_bytes_bf16(T, m->d, static_cast<int>(m->r));
}

logra_status logra_sketch_fold_parts(const logra_matrix *m, int64_t T, int act_dtype, const void *dY,
                                     int64_t lddy, float *S, float *parts, size_t parts_bytes, int phase,
                                     void *ws, size_t ws_bytes, const logra_launch_opts *opts,
                                     void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (phase & ~(LOGRA_FOLD_FIRST | LOGRA_FOLD_LAST)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_sketch(m, T, act_dtype);
    if (e == LOGRA_OK) e = check_fold(m, T, act_dtype, dY, lddy, S, ws, ws_bytes);
    if (e != LOGRA_OK) return e;
    const size_t need = logra_sketch_parts_bytes(m, T, act_dtype);
    if (need > 0) {
        if (!parts || parts_bytes < need) return LOGRA_ERR_WORKSPACE;
        if (!aligned16(parts)) return LOGRA_ERR_INVALID_ARGUMENT;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int accumulate = (phase & LOGRA_FOLD_FIRST) ? 0 : 1;
    if (need == 0) return from_hip(do_fold(m, T, act_dtype, dY, lddy, S, accumulate, ws, o, st));
    return from_hip(launch_fold_parts_ws_bf16(static_cast<int>(m->r), T, m->d, m->k,
                                              static_cast<const uint16_t *>(dY), lddy, S, parts, phase, ws, st));
}

logra_status logra_sketch_accumulate(const logra_matrix *m, int64_t T, int act_dtype,
                                     const void *X, int64_t ldx, const void *dY, int64_t lddy,
                                     float *S, int accumulate, void *ws, size_t ws_bytes,
                                     const logra_launch_opts *opts, void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_sketch(m, T, act_dtype);
    if (e == LOGRA_OK) e = check_fold(m, T, act_dtype, dY, lddy, S, ws, ws_bytes);
    if (e == LOGRA_OK) e = check_project(m, T, act_dtype, X, ldx, ws, ws_bytes);
    if (e != LOGRA_OK) return e;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t h = do_project(m, T, act_dtype, X, ldx, ws, o, st);
    if (h != hipSuccess) return LOGRA_ERR_HIP;
    return from_hip(do_fold(m, T, act_dtype, dY, lddy, S, accumulate, ws, o, st));
}

// Arguments of the backward product shared by both entry points.
static logra_status check_dx(const logra_matrix *m, int64_t T, int act_dtype, const void *dY, int64_t lddy,
                             const void *W, int64_t ldw, const void *dX, int64_t lddx) {
    if (!matrix_ok(m) || T < 0) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype != LOGRA_BF16) return LOGRA_ERR_UNSUPPORTED;
    if (m->d % 8 || m->k % 8 || T > (1ll << 30)) return LOGRA_ERR_UNSUPPORTED;
    if (!W || ldw < m->k || ldw % 8 || !aligned16(W)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!fits_view(m->d, ldw, 2)) return LOGRA_ERR_UNSUPPORTED;
    if (T == 0) return LOGRA_OK;
    if (!dY || lddy < m->d || lddy % 8 || !aligned16(dY)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!dX || lddx < m->k || lddx % 8 || !aligned16(dX)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!fits_view(T, lddy, 2) || !fits_view(T, lddx, 2)) return LOGRA_ERR_UNSUPPORTED;
    return LOGRA_OK;
}

logra_status logra_backward_dx(const logra_matrix *m, int64_t T, int act_dtype, const void *dY, int64_t lddy,
                               const void *W, int64_t ldw, void *dX, int64_t lddx,
                               const logra_launch_opts *opts, void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    const logra_status e = check_dx(m, T, act_dtype, dY, lddy, W, ldw, dX, lddx);
    if (e != LOGRA_OK || T == 0) return e;
    // the r = 256 instance of the launch, the one the fused call runs at the
    // 7B shapes, so the two time the same product code
    return from_hip(launch_dx_bf16(256, T, m->d, m->k, static_cast<const uint16_t *>(dY), lddy,
                                   static_cast<const uint16_t *>(W), ldw, static_cast<uint16_t *>(dX), lddx,
                                   nullptr, 0, nullptr, 0, 0, o.wait, static_cast<hipStream_t>(stream)));
}

logra_status logra_backward_dx_sketch(const logra_matrix *m, int64_t T, int act_dtype, const void *dY,
                                      int64_t lddy, const void *W, int64_t ldw, void *dX, int64_t lddx,
                                      float *S, int accumulate, void *ws, size_t ws_bytes,
                                      const logra_launch_opts *opts, void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_dx(m, T, act_dtype, dY, lddy, W, ldw, dX, lddx);
    if (e == LOGRA_OK) e = check_sketch(m, T, act_dtype);
    if (e == LOGRA_OK) e = check_fold(m, T, act_dtype, dY, lddy, S, ws, ws_bytes);
    if (e != LOGRA_OK) return e;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (T == 0) return accumulate ? LOGRA_OK : from_hip(launch_fill_zero(S, m->d * m->r, st));
    const int r = static_cast<int>(m->r);
    const Stage1Plan p = plan_stage1_bf16(T, m->k, r);
    const uint16_t *dy = static_cast<const uint16_t *>(dY);
    const bool fuse = o.backward_fold == 1 || (o.backward_fold == 0 && dx_fuse_pays(T, m->d, m->k, r));
    if (fuse)
        return from_hip(launch_dx_bf16(r, T, m->d, m->k, dy, lddy, static_cast<const uint16_t *>(W), ldw,
                                       static_cast<uint16_t *>(dX), lddx, static_cast<const uint16_t *>(ws),
                                       p.t_blocks, S, accumulate ? 1 : 0, 1, o.wait, st));
    // the fold would outlast the product beside it: the product, then the fold
    if (launch_dx_bf16(r, T, m->d, m->k, dy, lddy, static_cast<const uint16_t *>(W), ldw,
                       static_cast<uint16_t *>(dX), lddx, nullptr, 0, nullptr, 0, 0, o.wait, st) != hipSuccess)
        return LOGRA_ERR_HIP;
    return from_hip(launch_fold_bf16(r, T, m->d, m->k, dy, lddy, S, accumulate ? 1 : 0, ws, o.wait, st));
}

size_t logra_sqnorm_workspace_bytes(const logra_matrix *m, int compute_dtype) {
    if (!matrix_ok(m)) return 0;
    if (compute_dtype != LOGRA_F32 && compute_dtype != LOGRA_BF16) return 0;
    return sqnorm_ws_bytes(m, compute_dtype);
}

static logra_status check_apply_common(const logra_matrix *m, int compute_dtype, const float *S,
                                       float beta2, float eps) {
    if (!matrix_ok(m) || !S) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!(beta2 >= 0.f && beta2 <= 1.f) || !(eps >= 0.f)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (compute_dtype == LOGRA_BF16) {
        if (!bf16_rank_ok(m->r) || m->k % 8) return LOGRA_ERR_UNSUPPORTED;
    } else if (compute_dtype == LOGRA_F32) {
        if (m->r > 1024) return LOGRA_ERR_UNSUPPORTED;
    } else {
        return LOGRA_ERR_UNSUPPORTED;
    }
    if (!aligned16(S)) return LOGRA_ERR_INVALID_ARGUMENT;
    return LOGRA_OK;
}

static ApplyArgs base_args(const logra_matrix *m, const float *S, float beta2, float eps) {
    ApplyArgs a;
    a.R = static_cast<int>(m->r);
    a.D = m->d;
    a.K = m->k;
    a.key = stream_key(m->seed, m->step, m->matrix_id);
    a.c = inv_sqrt_rank(m->r);
    a.S = S;
    a.beta2 = beta2;
    a.eps = eps;
    return a;
}

static logra_status update_sqnorm_parts(const logra_matrix *m, int compute_dtype, const float *S,
                                        const float *v, float beta2, float eps, float *v_new,
                                        float *rowsq, float *sqnorm, void *ws, size_t ws_bytes,
                                        void *stream, int parts);

logra_status logra_update_sqnorm(const logra_matrix *m, int compute_dtype, const float *S,
                                 const float *v, float beta2, float eps, float *v_new,
                                 float *rowsq, float *sqnorm, void *ws, size_t ws_bytes,
                                 void *stream) {
    return update_sqnorm_parts(m, compute_dtype, S, v, beta2, eps, v_new, rowsq, sqnorm, ws, ws_bytes, stream,
                               kSqnormGram | kSqnormRows);
}

logra_status logra_update_sqnorm_prepared(const logra_matrix *m, int compute_dtype, const float *S,
                                          const float *v, float beta2, float eps, float *v_new,
                                          float *rowsq, float *sqnorm, void *ws, size_t ws_bytes,
                                          void *stream) {
    return update_sqnorm_parts(m, compute_dtype, S, v, beta2, eps, v_new, rowsq, sqnorm, ws, ws_bytes, stream,
                               kSqnormRows);
}

logra_status logra_sqnorm_prepare(const logra_matrix *m, int compute_dtype, void *ws, size_t ws_bytes,
                                  void *stream) {
    if (!matrix_ok(m)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (compute_dtype == LOGRA_BF16) {
        if (!bf16_rank_ok(m->r) || m->k % 8) return LOGRA_ERR_UNSUPPORTED;
    } else if (compute_dtype == LOGRA_F32) {
        if (m->r > 1024) return LOGRA_ERR_UNSUPPORTED;
    } else {
        return LOGRA_ERR_UNSUPPORTED;
    }
    const size_t need = sqnorm_ws_bytes(m, compute_dtype);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    if (compute_dtype != LOGRA_BF16) return LOGRA_OK;   // the fp32 pass has nothing to prepare
    ApplyArgs a = base_args(m, nullptr, 0.f, 0.f);
    return from_hip(launch_sqnorm_bf16(a, ws, static_cast<hipStream_t>(stream), kSqnormGram));
}

static logra_status update_sqnorm_parts(const logra_matrix *m, int compute_dtype, const float *S,
                                        const float *v, float beta2, float eps, float *v_new,
                                        float *rowsq, float *sqnorm, void *ws, size_t ws_bytes,
                                        void *stream, int parts) {
    logra_status stt = check_apply_common(m, compute_dtype, S, beta2, eps);
    if (stt != LOGRA_OK) return stt;
    if (!v || !v_new || !sqnorm || v_new == v) return LOGRA_ERR_INVALID_ARGUMENT;
    const size_t need = sqnorm_ws_bytes(m, compute_dtype);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ApplyArgs a = base_args(m, S, beta2, eps);
    a.v_in = v;
    a.v_new_out = v_new;
    a.rowsq_out = rowsq;
    a.sqnorm = sqnorm;
    if (compute_dtype == LOGRA_BF16) return from_hip(launch_sqnorm_bf16(a, ws, st, parts));
    a.partials = static_cast<float *>(ws);
    if (launch_apply_f32(0, a, st) != hipSuccess) return LOGRA_ERR_HIP;
    return from_hip(launch_sqnorm_final(a.partials, apply_blocks_f32(m->d), sqnorm, st));
}

logra_status logra_update_sqnorm_noalloc(const logra_matrix *m, int compute_dtype, const float *S,
                                         const float *v, float beta2, float eps, float *v_new,
                                         float *rowsq, float *sqnorm, void *stream) {
    // the same validation as logra_update_sqnorm, before the scratch is touched
    logra_status stt = check_apply_common(m, compute_dtype, S, beta2, eps);
    if (stt != LOGRA_OK) return stt;
    if (!v || !v_new || !sqnorm || v_new == v) return LOGRA_ERR_INVALID_ARGUMENT;
    const size_t need = sqnorm_ws_bytes(m, compute_dtype);
    if (need > kNoallocScratchBytes) return LOGRA_ERR_WORKSPACE;
    hipError_t e = hipSuccess;
    void *ws = device_scratch(&e);
    if (!ws) return LOGRA_ERR_HIP;
    return update_sqnorm_parts(m, compute_dtype, S, v, beta2, eps, v_new, rowsq, sqnorm, ws, kNoallocScratchBytes,
                               stream, kSqnormGram | kSqnormRows);
}

// Workspace slice of matrix i of a batch: the single-matrix layout, each
// slice 256-byte aligned.
static size_t batch_slice_bytes(const logra_matrix *m, int compute_dtype) {
    return (sqnorm_ws_bytes(m, compute_dtype) + 255) / 256 * 256;
}

size_t logra_sqnorm_batch_workspace_bytes(int n, const logra_matrix *ms, int compute_dtype) {
    if (n < 1 || n > LOGRA_MAX_BATCH || !ms) return 0;
    if (compute_dtype != LOGRA_F32 && compute_dtype != LOGRA_BF16) return 0;
    size_t total = 0;
    for (int i = 0; i < n; ++i) {
        if (!matrix_ok(&ms[i])) return 0;
        total += batch_slice_bytes(&ms[i], compute_dtype);
    }
    return total;
}

logra_status logra_update_sqnorm_batch(int n, const logra_matrix *ms, int compute_dtype,
                                       const float *const *S, const float *const *v, float beta2,
                                       float eps, float *const *v_new, float *const *rowsq,
                                       float *sqnorm, void *ws, size_t ws_bytes, void *stream) {
    if (n < 1 || n > LOGRA_MAX_BATCH || !ms || !S || !v || !v_new || !sqnorm)
        return LOGRA_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < n; ++i) {
        const logra_status e = check_apply_common(&ms[i], compute_dtype, S[i], beta2, eps);
        if (e != LOGRA_OK) return e;
        if (ms[i].r != ms[0].r) return LOGRA_ERR_INVALID_ARGUMENT;
        if (!v[i] || !v_new[i] || v_new[i] == v[i]) return LOGRA_ERR_INVALID_ARGUMENT;
    }
    if (!aligned16(sqnorm)) return LOGRA_ERR_INVALID_ARGUMENT;
    const size_t need = logra_sqnorm_batch_workspace_bytes(n, ms, compute_dtype);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char *base = static_cast<char *>(ws);
    if (compute_dtype == LOGRA_F32) {
        // the fp32 twin: the single-matrix passes one after another
        for (int i = 0; i < n; ++i) {
            ApplyArgs a = base_args(&ms[i], S[i], beta2, eps);
            a.v_in = v[i];
            a.v_new_out = v_new[i];
            a.rowsq_out = rowsq ? rowsq[i] : nullptr;
            a.sqnorm = sqnorm + i;
            a.partials = reinterpret_cast<float *>(base);
            if (launch_apply_f32(0, a, st) != hipSuccess) return LOGRA_ERR_HIP;
            if (launch_sqnorm_final(a.partials, apply_blocks_f32(ms[i].d), a.sqnorm, st) != hipSuccess)
                return LOGRA_ERR_HIP;
            base += batch_slice_bytes(&ms[i], compute_dtype);
        }
        return LOGRA_OK;
    }
    SqnormBatch b;
    b.n = n;
    b.beta2 = beta2;
    b.eps = eps;
    b.sqnorm = sqnorm;
    int wg = 0;
    for (int i = 0; i < n; ++i) {
        const SqnormPlan p = plan_sqnorm_bf16(ms[i].d, ms[i].k, static_cast<int>(ms[i].r));
        SqnormItem &it = b.item[i];
        it.S = S[i];
        it.v = v[i];
        it.v_new = v_new[i];
        it.rowsq = rowsq ? rowsq[i] : nullptr;
        it.slots = reinterpret_cast<uint64_t *>(base);
        it.M = reinterpret_cast<uint16_t *>(base + p.partial_bytes);
        it.key = stream_key(ms[i].seed, ms[i].step, ms[i].matrix_id);
        it.c = inv_sqrt_rank(ms[i].r);
        it.D = static_cast<int>(ms[i].d);
        it.K = static_cast<int>(ms[i].k);
        it.bpw = p.rows_per_block / 16;
        it.wg_begin = wg;
        it.n_wg = p.n_blocks;
        wg += p.n_blocks;
        base += batch_slice_bytes(&ms[i], compute_dtype);
    }
    return from_hip(launch_sqnorm_batch_bf16(static_cast<int>(ms[0].r), b, st));
}

logra_status logra_rowadam_apply(const logra_matrix *m, int compute_dtype, const float *S,
                                 const float *v_new, void *W, int w_dtype, int64_t ldw,
                                 float lr, float scale, float eps, const logra_launch_opts *opts,
                                 void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status stt = check_apply_common(m, compute_dtype, S, 0.f, eps);
    if (stt != LOGRA_OK) return stt;
    if (!v_new || !W) return LOGRA_ERR_INVALID_ARGUMENT;
    if (w_dtype != LOGRA_F32 && w_dtype != LOGRA_BF16) return LOGRA_ERR_UNSUPPORTED;
    if (ldw < m->k) return LOGRA_ERR_INVALID_ARGUMENT;
    if (compute_dtype == LOGRA_BF16 && (ldw % 8 || !aligned16(W))) return LOGRA_ERR_INVALID_ARGUMENT;
    if (compute_dtype == LOGRA_BF16 && !fits_view(m->d, ldw, w_dtype == LOGRA_BF16 ? 2 : 4))
        return LOGRA_ERR_UNSUPPORTED;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ApplyArgs a = base_args(m, S, 0.f, eps);
    a.v_new_in = v_new;
    a.lr_scale = lr * scale;
    a.W = W;
    a.w_bf16 = w_dtype == LOGRA_BF16 ? 1 : 0;
    a.ldw = ldw;
    return from_hip(compute_dtype == LOGRA_BF16 ? launch_rowadam_bf16(a, o.apply_concurrency, st)
                                                : launch_apply_f32(1, a, st));
}

// ------------------------------------------------------------- two-sided --

// Step value of the projections' streams (side s uses this + s): one the
// sign matrices of a run never take.
constexpr uint64_t kTsProjectionStep = 0xFFFFFFFFFFFFFF00ull;

static logra_status check_ts(const logra_matrix *m) {
    if (!matrix_ok(m)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (m->r != 32 || m->d % 8 || m->k % 8 || m->d < 32 || m->k < 32) return LOGRA_ERR_UNSUPPORTED;
    // the folds' exchange buffers are addressed through 32-bit views
    if (!fits_view(m->d, m->r, 4 * 16) || !fits_view(m->k, m->r, 4 * 16)) return LOGRA_ERR_UNSUPPORTED;
    return LOGRA_OK;
}

size_t logra_ts_projection_bytes(const logra_matrix *m, int side) {
    if (check_ts(m) != LOGRA_OK || (side != 0 && side != 1)) return 0;
    return ts_projection_layout(side ? m->k : m->d).total;
}

logra_status logra_ts_make_projection(const logra_matrix *m, int side, void *proj, size_t proj_bytes,
                                      void *stream) {
    if (side != 0 && side != 1) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_ts(m);
    if (e != LOGRA_OK) return e;
    if (!proj || !aligned16(proj)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (proj_bytes < logra_ts_projection_bytes(m, side)) return LOGRA_ERR_WORKSPACE;
    const uint64_t key = stream_key(m->seed, kTsProjectionStep + static_cast<uint64_t>(side), m->matrix_id);
    return from_hip(launch_ts_projection(key, side ? m->k : m->d, proj, static_cast<hipStream_t>(stream)));
}

size_t logra_ts_sketch_workspace_bytes(const logra_matrix *m, int64_t T) {
    if (check_ts(m) != LOGRA_OK || T <= 0 || T > (1ll << 30)) return 0;
    return ts_sketch_layout(T, m->d, m->k).total;
}

logra_status logra_ts_sketch_accumulate(const logra_matrix *m, int64_t T, const void *X, int64_t ldx,
                                        const void *dY, int64_t lddy, const void *proj_P, const void *proj_Q,
                                        float *S_L, float *S_R, int accumulate, void *ws, size_t ws_bytes,
                                        const logra_launch_opts *opts, void *stream) {
    Opts o;
    if (!read_opts(opts, &o)) return LOGRA_ERR_INVALID_ARGUMENT;
    logra_status e = check_ts(m);
    if (e != LOGRA_OK) return e;
    if (T < 0) return LOGRA_ERR_INVALID_ARGUMENT;
    if (T > (1ll << 30)) return LOGRA_ERR_UNSUPPORTED;
    if (!S_L || !S_R || S_L == S_R || !aligned16(S_L) || !aligned16(S_R)) return LOGRA_ERR_INVALID_ARGUMENT;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (T == 0) {
        if (accumulate) return LOGRA_OK;
        if (launch_fill_zero(S_R, m->d * m->r, st) != hipSuccess) return LOGRA_ERR_HIP;
        return from_hip(launch_fill_zero(S_L, m->k * m->r, st));
    }
    if (!X || !dY || !proj_P || !proj_Q || !aligned16(proj_P) || !aligned16(proj_Q)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (ldx < m->k || ldx % 8 || !aligned16(X)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (lddy < m->d || lddy % 8 || !aligned16(dY)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!fits_view(T + 32, ldx, 2) || !fits_view(T + 32, lddy, 2)) return LOGRA_ERR_UNSUPPORTED;
    const size_t need = logra_ts_sketch_workspace_bytes(m, T);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    return from_hip(launch_ts_sketch(T, m->d, m->k, static_cast<const uint16_t *>(X), ldx,
                                     static_cast<const uint16_t *>(dY), lddy, proj_P, proj_Q, S_L, S_R,
                                     accumulate ? 1 : 0, ws, o.wait, st));
}

size_t logra_ts_update_workspace_bytes(const logra_matrix *m) {
    if (check_ts(m) != LOGRA_OK) return 0;
    return ts_update_layout(m->d, m->k).total;
}

logra_status logra_ts_update(const logra_matrix *m, const float *S_L, const float *S_R, const void *proj_P,
                             float *m_L, float *v_L, float *m_R, float *v_R, float beta1, float beta2, float eps,
                             float *sqnorm, void *ws, size_t ws_bytes, void *stream) {
    logra_status e = check_ts(m);
    if (e != LOGRA_OK) return e;
    const void *ptrs[] = {S_L, S_R, proj_P, m_L, v_L, m_R, v_R};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!sqnorm) return LOGRA_ERR_INVALID_ARGUMENT;
    const void *outs[] = {m_L, v_L, m_R, v_R};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (outs[i] == outs[j]) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!(beta1 >= 0.f && beta1 <= 1.f) || !(beta2 >= 0.f && beta2 <= 1.f) || !(eps >= 0.f))
        return LOGRA_ERR_INVALID_ARGUMENT;
    const size_t need = logra_ts_update_workspace_bytes(m);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    return from_hip(launch_ts_update(m->d, m->k, S_L, S_R, proj_P, m_L, v_L, m_R, v_R, beta1, beta2, eps, sqnorm,
                                     ws, static_cast<hipStream_t>(stream)));
}

logra_status logra_ts_apply(const logra_matrix *m, const void *ws, size_t ws_bytes, void *W, int w_dtype,
                            int64_t ldw, float lr, float scale, void *stream) {
    logra_status e = check_ts(m);
    if (e != LOGRA_OK) return e;
    if (!W) return LOGRA_ERR_INVALID_ARGUMENT;
    if (w_dtype != LOGRA_F32 && w_dtype != LOGRA_BF16) return LOGRA_ERR_UNSUPPORTED;
    if (ldw < m->k || ldw % 8 || !aligned16(W)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!isfinite(lr) || !isfinite(scale)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!fits_view(m->d, ldw, w_dtype == LOGRA_BF16 ? 2 : 4)) return LOGRA_ERR_UNSUPPORTED;
    const size_t need = logra_ts_update_workspace_bytes(m);
    if (!ws || ws_bytes < need || !aligned16(ws)) return LOGRA_ERR_WORKSPACE;
    return from_hip(launch_ts_apply(m->d, m->k, ws, W, w_dtype == LOGRA_BF16 ? 1 : 0, ldw, lr * scale,
                                    static_cast<hipStream_t>(stream)));
}

// ---- global gradient norm and clipping ----

namespace {

bool aligned_to(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A list as the launching calls take it.
bool grad_list_ok(const logra_grad_list *g) {
    return g && g->n >= 0 && g->chunks >= 0 && (g->n == 0 || (g->table && aligned16(g->table)));
}

bool grad_ws_ok(const logra_grad_list *g, const void *ws, size_t ws_bytes) {
    const size_t need = logra_grad_workspace_bytes(g);
    return need == 0 || (ws && ws_bytes >= need && aligned16(ws));
}

struct GradSpan {
    uint64_t begin, end;
    bool operator<(const GradSpan &o) const { return begin < o.begin; }
};

}  // namespace

size_t logra_grad_table_bytes(int64_t n) {
    return n < 0 || n > (1 << 20) ? 0 : static_cast<size_t>(n) * sizeof(GradEntry);
}

logra_status logra_grad_list_pack(int64_t n, const logra_grad_tensor *tensors, void *table_host, size_t table_bytes,
                                  logra_grad_list *list) {
    if (n < 0 || n > (1 << 20) || !list || (n > 0 && (!tensors || !table_host)) || !aligned_to(table_host, 8))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (table_bytes < logra_grad_table_bytes(n)) return LOGRA_ERR_WORKSPACE;
    constexpr int64_t kMost = 1ll << 40;
    // the address ranges, in the table's memory before the table takes it
    GradSpan *span = static_cast<GradSpan *>(table_host);
    int64_t n_span = 0;
    for (int64_t i = 0; i < n; ++i) {
        const logra_grad_tensor &t = tensors[i];
        if (t.rows < 0 || t.cols < 0 || t.ld < t.cols) return LOGRA_ERR_INVALID_ARGUMENT;
        if (t.dtype != LOGRA_F32 && t.dtype != LOGRA_BF16) return LOGRA_ERR_UNSUPPORTED;
        if (t.rows == 0 || t.cols == 0) continue;
        const int64_t el = t.dtype == LOGRA_BF16 ? 2 : 4;
        if (!t.data || !aligned_to(t.data, el)) return LOGRA_ERR_INVALID_ARGUMENT;
        if (t.rows > kMost || t.cols > kMost || t.ld > kMost || t.rows > kMost / t.cols || t.rows > kMost / t.ld)
            return LOGRA_ERR_UNSUPPORTED;
        const uint64_t a = reinterpret_cast<uint64_t>(t.data);
        span[n_span++] = GradSpan{a, a + static_cast<uint64_t>(((t.rows - 1) * t.ld + t.cols) * el)};
    }
    std::sort(span, span + n_span);
    for (int64_t i = 1; i < n_span; ++i)
        if (span[i].begin < span[i - 1].end) return LOGRA_ERR_INVALID_ARGUMENT;
    GradEntry *table = static_cast<GradEntry *>(table_host);
    logra_grad_list out = {};
    uint64_t hash = 0xCBF29CE484222325ull;      // FNV-1a over rows and cols
    auto mix = [&](int64_t v) {
        for (int b = 0; b < 64; b += 8) hash = (hash ^ ((static_cast<uint64_t>(v) >> b) & 0xFF)) * 0x100000001B3ull;
    };
    for (int64_t i = 0; i < n; ++i) {
        const logra_grad_tensor &t = tensors[i];
        GradEntry e;
        e.addr = reinterpret_cast<uint64_t>(t.data);
        e.rows = t.rows;
        e.cols = t.cols;
        e.ld = t.rows == 1 ? t.cols : t.ld;
        e.bf16 = t.dtype == LOGRA_BF16;
        e.first = out.chunks;
        if (t.rows > 0 && t.cols > 0) {
            if (t.cols <= kGradChunk) {
                e.rows_per_chunk = static_cast<int32_t>(kGradChunk / t.cols);
                e.chunks = (t.rows + e.rows_per_chunk - 1) / e.rows_per_chunk;
            } else {
                const int64_t segs = (t.cols + kGradChunk - 1) / kGradChunk;
                e.seg_len = static_cast<int32_t>(((t.cols + segs - 1) / segs + 7) / 8 * 8);
                e.segs_per_row = static_cast<int32_t>((t.cols + e.seg_len - 1) / e.seg_len);
                e.chunks = t.rows * e.segs_per_row;
            }
        }
        out.chunks += e.chunks;
        out.elements += t.rows * t.cols;
        if (out.elements > (kMost << 4)) return LOGRA_ERR_UNSUPPORTED;
        mix(t.rows);
        mix(t.cols);
        table[i] = e;
    }
    out.n = static_cast<int32_t>(n);
    out.shapes = hash;
    *list = out;
    return LOGRA_OK;
}

size_t logra_grad_workspace_bytes(const logra_grad_list *list) {
    return list && list->chunks >= 0 ? grad_workspace(list->n, list->chunks, list->elements) : 0;
}

logra_status logra_grad_norm(const logra_grad_list *list, float *norm, void *ws, size_t ws_bytes, void *stream) {
    if (!grad_list_ok(list) || !norm || !aligned_to(norm, 4)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!grad_ws_ok(list, ws, ws_bytes)) return LOGRA_ERR_WORKSPACE;
    return from_hip(launch_grad_norm(static_cast<const GradEntry *>(list->table), list->n, list->chunks,
                                     list->elements, static_cast<double *>(ws), norm, static_cast<hipStream_t>(stream)));
}

logra_status logra_grad_clip(const logra_grad_list *list, const logra_grad_list *out, float max_norm, float *norm,
                             float *coef, void *ws, size_t ws_bytes, void *stream) {
    if (!grad_list_ok(list) || !norm || !coef || norm == coef) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(norm, 4) || !aligned_to(coef, 4) || !(max_norm >= 0.f)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!out) out = list;
    if (!grad_list_ok(out) || out->n != list->n || out->chunks != list->chunks || out->shapes != list->shapes)
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (!grad_ws_ok(list, ws, ws_bytes)) return LOGRA_ERR_WORKSPACE;
    return from_hip(launch_grad_clip(static_cast<const GradEntry *>(list->table),
                                     static_cast<const GradEntry *>(out->table), list->n, list->chunks,
                                     list->elements, max_norm, static_cast<double *>(ws), norm, coef, static_cast<hipStream_t>(stream)));
}

// ---- rows sorted by expert, and back ----

namespace {

constexpr int64_t kMaxPairs = 1ll << 26, kMaxExpertTokens = 1ll << 23, kMaxExpertDim = 1ll << 22;

logra_status check_pairs(int64_t T, int topk) {
    if (T < 0 || topk < 1) return LOGRA_ERR_INVALID_ARGUMENT;
    if (topk > kMaxTopK || T > kMaxExpertTokens || T * topk > kMaxPairs) return LOGRA_ERR_UNSUPPORTED;
    return LOGRA_OK;
}

// One array of rows: n of them, h wide.
bool rows_ok(const void *p, int64_t ld, int64_t n, int64_t h, int dtype) {
    return n == 0 || (p && ld >= h && aligned_to(p, dtype == LOGRA_BF16 ? 2 : 4));
}

logra_status check_rows(int64_t T, int topk, int64_t h, int dtype, const int32_t *slots, const float *w,
                        int64_t n_rows) {
    const logra_status e = check_pairs(T, topk);
    if (e != LOGRA_OK) return e;
    if (h < 1 || n_rows < 0) return LOGRA_ERR_INVALID_ARGUMENT;
    if ((dtype != LOGRA_F32 && dtype != LOGRA_BF16) || h > (1ll << 30)) return LOGRA_ERR_UNSUPPORTED;
    if (T > 0 && (!slots || !aligned_to(slots, 4) || !aligned_to(w, 4))) return LOGRA_ERR_INVALID_ARGUMENT;
    return LOGRA_OK;
}

int elem_bytes(int dtype) { return dtype == LOGRA_BF16 ? 2 : 4; }

}  // namespace

size_t logra_expert_sort_workspace_bytes(int64_t T, int topk, int n_experts) {
    if (check_pairs(T, topk) != LOGRA_OK || n_experts < 1 || n_experts > kMaxExperts) return 0;
    return expert_sort_workspace(T * topk, n_experts);
}

logra_status logra_expert_sort(int64_t T, int topk, int n_experts, const void *ids, int id_bytes, int64_t ld_ids,
                               int32_t *offsets, int32_t *order, int32_t *slots, void *ws, size_t ws_bytes,
                               void *stream) {
    const logra_status e = check_pairs(T, topk);
    if (e != LOGRA_OK) return e;
    if (n_experts < 1 || (id_bytes != 4 && id_bytes != 8) || !offsets || !aligned_to(offsets, 4))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (n_experts > kMaxExperts) return LOGRA_ERR_UNSUPPORTED;
    if (T > 0 && (!ids || !aligned_to(ids, id_bytes) || ld_ids < topk || !order || !aligned_to(order, 4) || !slots ||
                  !aligned_to(slots, 4)))
        return LOGRA_ERR_INVALID_ARGUMENT;
    const size_t need = expert_sort_workspace(T * topk, n_experts);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return LOGRA_ERR_WORKSPACE;
    return from_hip(launch_expert_sort(T, topk, n_experts, ids, id_bytes, ld_ids, offsets, order, slots, ws,
                                       static_cast<hipStream_t>(stream)));
}

logra_status logra_expert_gather(int64_t T, int topk, int64_t h, int dtype, const void *X, int64_t ldx,
                                 const int32_t *slots, const float *w, void *Xs, int64_t ldxs, int64_t n_rows,
                                 void *stream) {
    const logra_status e = check_rows(T, topk, h, dtype, slots, w, n_rows);
    if (e != LOGRA_OK) return e;
    if (!rows_ok(X, ldx, T, h, dtype) || !rows_ok(Xs, ldxs, n_rows, h, dtype)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (T == 0 || n_rows == 0) return LOGRA_OK;
    return from_hip(launch_expert_gather(T, topk, h, elem_bytes(dtype), X, ldx, slots, w, Xs, ldxs, n_rows,
                                         static_cast<hipStream_t>(stream)));
}

logra_status logra_expert_combine(int64_t T, int topk, int64_t h, int dtype, const void *Ys, int64_t ldys,
                                  int64_t n_rows, const int32_t *slots, const float *w, void *Y, int64_t ldy,
                                  void *stream) {
    const logra_status e = check_rows(T, topk, h, dtype, slots, w, n_rows);
    if (e != LOGRA_OK) return e;
    if (!rows_ok(Ys, ldys, n_rows, h, dtype) || !rows_ok(Y, ldy, T, h, dtype)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (T == 0) return LOGRA_OK;
    return from_hip(launch_expert_combine(T, topk, h, elem_bytes(dtype), Ys, ldys, n_rows, slots, w, Y, ldy,
                                          static_cast<hipStream_t>(stream)));
}

logra_status logra_expert_combine_backward(int64_t T, int topk, int64_t h, int dtype, const void *dY, int64_t lddy,
                                           const void *Ys, int64_t ldys, int64_t n_rows, const int32_t *slots,
                                           const float *w, void *dYs, int64_t lddys, float *dw, void *stream) {
    const logra_status e = check_rows(T, topk, h, dtype, slots, w, n_rows);
    if (e != LOGRA_OK) return e;
    if (!rows_ok(dY, lddy, T, h, dtype) || !rows_ok(Ys, ldys, n_rows, h, dtype) ||
        !rows_ok(dYs, lddys, n_rows, h, dtype))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!w || !dw || !aligned_to(dw, 4))) return LOGRA_ERR_INVALID_ARGUMENT;
    if (T == 0) return LOGRA_OK;
    return from_hip(launch_expert_combine_backward(T, topk, h, elem_bytes(dtype), dY, lddy, Ys, ldys, slots, w, dYs,
                                                   lddys, n_rows, dw, static_cast<hipStream_t>(stream)));
}

// ---- the sketch over experts ----

static logra_status check_sketch_experts(const logra_matrix *m, int n_experts, int64_t N, int act_dtype) {
    if (!matrix_ok(m) || n_experts < 1 || N < 0) return LOGRA_ERR_INVALID_ARGUMENT;
    if (act_dtype != LOGRA_F32 && act_dtype != LOGRA_BF16) return LOGRA_ERR_UNSUPPORTED;
    if (n_experts > kMaxExperts || N > kMaxPairs) return LOGRA_ERR_UNSUPPORTED;
    if (m->d > kMaxExpertDim || m->k > kMaxExpertDim) return LOGRA_ERR_UNSUPPORTED;
    if (act_dtype == LOGRA_BF16 ? !bf16_rank_ok(m->r) || m->d % 8 || m->k % 8 : m->r > 1024)
        return LOGRA_ERR_UNSUPPORTED;
    // a launch has fewer than 2^32 threads in a dimension
    const ExpertSketchPlan p =
        plan_expert_sketch(N, n_experts, m->d, m->k, static_cast<int>(m->r), act_dtype == LOGRA_BF16);
    if ((p.items + 8) * ((m->d + 127) / 128) >= (1ll << 24)) return LOGRA_ERR_UNSUPPORTED;
    return LOGRA_OK;
}

size_t logra_sketch_experts_workspace_bytes(const logra_matrix *m, int n_experts, int64_t N, int act_dtype) {
    if (check_sketch_experts(m, n_experts, N, act_dtype) != LOGRA_OK) return 0;
    return plan_expert_sketch(N, n_experts, m->d, m->k, static_cast<int>(m->r), act_dtype == LOGRA_BF16).total;
}

logra_status logra_sketch_experts(const logra_matrix *m, int n_experts, uint64_t id_stride, int64_t N, int act_dtype,
                                  const int32_t *offsets, const int32_t *order, int topk, const void *X, int64_t ldx,
                                  int64_t x_rows, const void *dY, int64_t lddy, float *S, int accumulate, void *ws,
                                  size_t ws_bytes, void *stream) {
    const logra_status e = check_sketch_experts(m, n_experts, N, act_dtype);
    if (e != LOGRA_OK) return e;
    const bool bf16 = act_dtype == LOGRA_BF16;
    if (!offsets || !aligned_to(offsets, 4) || !S || !aligned16(S)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (x_rows < 0 || (order ? topk < 1 || !aligned_to(order, 4) : x_rows < N)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (N > 0) {
        if (!dY || lddy < m->d || (x_rows > 0 && (!X || ldx < m->k))) return LOGRA_ERR_INVALID_ARGUMENT;
        if (bf16 ? lddy % 8 || ldx % 8 || !aligned16(X) || !aligned16(dY) : !aligned_to(X, 4) || !aligned_to(dY, 4))
            return LOGRA_ERR_INVALID_ARGUMENT;
        // X is read through one buffer view, dY through one per 32 rows
        if (bf16 && ((x_rows > 0 && ldx > ((1ll << 31) - 1) / 2 / x_rows) || lddy > (1ll << 24)))
            return LOGRA_ERR_UNSUPPORTED;
    }
    const ExpertSketchPlan p = plan_expert_sketch(N, n_experts, m->d, m->k, static_cast<int>(m->r), bf16);
    if (N == 0 && accumulate) return LOGRA_OK;
    if (p.total > 0 && (!ws || ws_bytes < p.total || !aligned16(ws))) return LOGRA_ERR_WORKSPACE;
    ExpertSketchArgs a;
    a.E = n_experts;
    a.R = static_cast<int>(m->r);
    a.topk = order ? topk : 1;
    a.N = N;
    a.d = m->d;
    a.k = m->k;
    const auto h = [](uint64_t x) { return splitmix_finalize(x + kGolden); };
    a.prefix = h(h(m->seed) ^ m->step);     // expert e's key is h(prefix ^ id), see stream_key
    a.first_id = m->matrix_id;
    a.id_stride = id_stride;
    a.c = inv_sqrt_rank(m->r);
    a.offsets = offsets;
    a.order = order;
    a.X = X;
    a.dY = dY;
    a.ldx = ldx;
    a.x_rows = x_rows;
    a.lddy = lddy;
    a.S = S;
    a.accumulate = accumulate ? 1 : 0;
    a.ws = ws;
    return from_hip(launch_expert_sketch(a, bf16 ? 1 : 0, static_cast<hipStream_t>(stream)));
}

// ---- routing ----

namespace {

bool dtype_ok(int dtype) { return dtype == LOGRA_F32 || dtype == LOGRA_BF16; }

// What routing and its gradient have in common.
logra_status check_route(int64_t T, int n_experts, int topk, int dtype, int score, const void *logits, int64_t ld,
                         const int32_t *ids, const float *w) {
    if (T < 0 || n_experts < 1 || topk < 1 || topk > n_experts) return LOGRA_ERR_INVALID_ARGUMENT;
    if (score != LOGRA_SOFTMAX && score != LOGRA_SIGMOID) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(dtype) || n_experts > kMaxExperts || topk > kMaxTopK || T > kMaxExpertTokens || ld > (1ll << 40))
        return LOGRA_ERR_UNSUPPORTED;
    if (!rows_ok(logits, ld, T, n_experts, dtype)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!ids || !aligned_to(ids, 4) || !w || !aligned_to(w, 4))) return LOGRA_ERR_INVALID_ARGUMENT;
    return LOGRA_OK;
}

void route_call(RouteCall &c, int64_t T, int n_experts, int topk, int dtype, int score, const void *logits, int64_t ld,
                int renormalize, float scale) {
    c.logits = logits;
    c.ld = ld;
    c.T = T;
    c.bf16 = dtype == LOGRA_BF16;
    c.E = n_experts;
    c.K = topk;
    c.sigmoid = score == LOGRA_SIGMOID;
    c.renorm = renormalize != 0;
    c.scale = scale;
}

}  // namespace

logra_status logra_route(int64_t T, int n_experts, int topk, int dtype, const void *logits, int64_t ld, int score,
                         const float *bias, int groups, int topk_groups, int group_best, int renormalize, float scale,
                         int32_t *ids, float *weights, void *stream) {
    const logra_status e = check_route(T, n_experts, topk, dtype, score, logits, ld, ids, weights);
    if (e != LOGRA_OK) return e;
    if (!aligned_to(bias, 4) || groups < 1 || n_experts % groups || topk_groups < 1 || topk_groups > groups ||
        (group_best != 1 && group_best != 2))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (groups > kMaxRouteGroups) return LOGRA_ERR_UNSUPPORTED;
    if (T == 0) return LOGRA_OK;
    RouteCall c;
    route_call(c, T, n_experts, topk, dtype, score, logits, ld, renormalize, scale);
    c.bias = bias;
    c.groups = groups;
    c.kept = topk_groups;
    c.best = group_best;
    c.ids = ids;
    c.weights = weights;
    return from_hip(launch_route(c, static_cast<hipStream_t>(stream)));
}

logra_status logra_route_backward(int64_t T, int n_experts, int topk, int dtype, const void *logits, int64_t ld,
                                  int score, const int32_t *ids, const float *dweights, int renormalize, float scale,
                                  void *dlogits, int64_t ldd, void *stream) {
    const logra_status e = check_route(T, n_experts, topk, dtype, score, logits, ld, ids, dweights);
    if (e != LOGRA_OK) return e;
    if (!rows_ok(dlogits, ldd, T, n_experts, dtype)) return LOGRA_ERR_INVALID_ARGUMENT;
    if (ldd > (1ll << 40)) return LOGRA_ERR_UNSUPPORTED;
    if (T == 0) return LOGRA_OK;
    RouteCall c;
    route_call(c, T, n_experts, topk, dtype, score, logits, ld, renormalize, scale);
    c.ids = const_cast<int32_t *>(ids);
    return from_hip(launch_route_backward(c, dweights, dlogits, ldd, static_cast<hipStream_t>(stream)));
}

// ---- products in 8 bits ----

logra_status logra_fp8_quantize(int64_t batch, int64_t rows, int64_t cols, int dtype, const void *x, int64_t ldx,
                                int block_rows, int transpose, void *codes, int64_t ldc, float *scales,
                                void *stream) {
    if (batch < 0 || rows < 0 || cols < 0 || (block_rows != 1 && block_rows != 128) || (transpose && block_rows == 1))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(dtype)) return LOGRA_ERR_UNSUPPORTED;
    if (batch == 0 || rows == 0 || cols == 0) return LOGRA_OK;
    constexpr int64_t kMost = 1ll << 40;
    if (batch > kMost || rows > kMost || cols > (1ll << 30) || ldx > kMost / rows || ldc > kMost / rows ||
        ldc > kMost / cols || batch > kMost / rows)
        return LOGRA_ERR_UNSUPPORTED;
    if (!x || ldx < cols || !aligned_to(x, elem_bytes(dtype)) || !codes || ldc < (transpose ? rows : cols) || !scales ||
        !aligned_to(scales, 4))
        return LOGRA_ERR_INVALID_ARGUMENT;
    // a launch has fewer than 2^32 threads: 16 of them a row's block, 256 a block of 128 rows
    const int64_t kb = (cols + 127) / 128;
    const int64_t blocks = block_rows == 1 ? batch * rows / 16 + 1 : batch * ((rows + 127) / 128);
    if (blocks >= (1ll << 24) / kb) return LOGRA_ERR_UNSUPPORTED;
    QuantizeCall c;
    c.batch = batch;
    c.rows = rows;
    c.cols = cols;
    c.x = x;
    c.ldx = ldx;
    c.bf16 = dtype == LOGRA_BF16;
    c.block_rows = block_rows;
    c.turned = transpose != 0;
    c.codes = static_cast<uint8_t *>(codes);
    c.ldc = ldc;
    c.scales = scales;
    return from_hip(launch_fp8_quantize(c, static_cast<hipStream_t>(stream)));
}

logra_status logra_fp8_matmul(int64_t M, int64_t n, int64_t k, int n_experts, const int32_t *offsets,
                              const int32_t *order, int topk, const void *x, int64_t ldx, int64_t x_rows,
                              const float *x_scales, const void *w, int64_t ldw, const float *w_scales, int y_dtype,
                              void *y, int64_t ldy, void *stream) {
    if (M < 0 || n < 1 || k < 1 || n_experts < 1 || x_rows < 0 || (!offsets && n_experts != 1))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (order ? !offsets || topk < 1 || !aligned_to(order, 4) : x_rows < M) return LOGRA_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(y_dtype) || n_experts > kMaxExperts || M > kMaxPairs || n > kMaxExpertDim || k > kMaxExpertDim || k % 16)
        return LOGRA_ERR_UNSUPPORTED;
    if (M == 0) return LOGRA_OK;
    if (!aligned_to(offsets, 4) || !w || !aligned16(w) || ldw < k || ldw % 16 || !w_scales || !aligned_to(w_scales, 4) ||
        !y || ldy < n || !aligned_to(y, elem_bytes(y_dtype)))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (x_rows > 0 && (!x || !aligned16(x) || ldx < k || ldx % 16 || !x_scales || !aligned_to(x_scales, 4)))
        return LOGRA_ERR_INVALID_ARGUMENT;
    // rows are read at 32-bit offsets: from a tile's first one, or all of x where the order picks them
    if (ldw > kMaxExpertDim || ldy > (1ll << 40)) return LOGRA_ERR_UNSUPPORTED;
    if (x_rows > 0 && (ldx > kMaxExpertDim || (order && x_rows > ((1ll << 31) - 1) / ldx))) return LOGRA_ERR_UNSUPPORTED;
    if (!fp8_matmul_fits(M, n, offsets ? n_experts : 0)) return LOGRA_ERR_UNSUPPORTED;
    MatmulCall c;
    c.M = M;
    c.N = static_cast<int>(n);
    c.K = static_cast<int>(k);
    c.E = n_experts;
    c.topk = order ? topk : 1;
    c.offsets = offsets;
    c.order = order;
    c.x = static_cast<const uint8_t *>(x);
    c.w = static_cast<const uint8_t *>(w);
    c.ldx = ldx;
    c.x_rows = x_rows;
    c.ldw = ldw;
    c.xs = x_scales;
    c.ws = w_scales;
    c.y = y;
    c.ldy = ldy;
    c.y_bf16 = y_dtype == LOGRA_BF16;
    return from_hip(launch_fp8_matmul(c, static_cast<hipStream_t>(stream)));
}

// ---- AdamW over many tensors ----

namespace {

// The matrix id whose counter stream rounds the 8-bit moments; no sketched
// matrix should have it.
constexpr uint64_t kAdamId = 0xFFFFFFFFFFFFFFFFull;

// The bytes of an array: rows of `width` at a stride, or one run of them (stride 0).
struct AdamSpan {
    uint64_t begin, end, stride, width;
    bool operator<(const AdamSpan &o) const { return begin < o.begin; }
};
constexpr int kAdamLive = 256;      // arrays that may lie between each other's rows

bool adam_array(const void *p, int64_t rows, int64_t cols, int64_t ld, int dtype, AdamSpan *span) {
    const int64_t el = elem_bytes(dtype);
    if (!p || ld < cols || !aligned_to(p, el)) return false;
    span->begin = reinterpret_cast<uint64_t>(p);
    span->end = span->begin + static_cast<uint64_t>(((rows - 1) * ld + cols) * el);
    const bool run = rows == 1 || ld == cols;
    span->stride = run ? 0 : static_cast<uint64_t>(ld * el);
    span->width = run ? span->end - span->begin : static_cast<uint64_t>(cols * el);
    return true;
}

// Whether b, which begins between a's begin and end, has bytes of a. Rows of the
// same stride that start in a gap of a's and end there do so everywhere; of
// different strides they are not told apart.
bool adam_clash(const AdamSpan &a, const AdamSpan &b) {
    if (a.stride == 0 || (b.stride != 0 && b.stride != a.stride)) return true;
    const uint64_t at = (b.begin - a.begin) % a.stride;
    return at < a.width || b.width > a.stride - at;
}

logra_status adam_apart(AdamSpan *span, int64_t n) {
    std::sort(span, span + n);
    const AdamSpan *live[kAdamLive];        // those that have not ended
    int n_live = 0;
    for (int64_t i = 0; i < n; ++i) {
        int kept = 0;
        for (int j = 0; j < n_live; ++j) {
            if (live[j]->end <= span[i].begin) continue;
            if (adam_clash(*live[j], span[i])) return LOGRA_ERR_INVALID_ARGUMENT;
            live[kept++] = live[j];
        }
        n_live = kept;
        if (n_live == kAdamLive) return LOGRA_ERR_UNSUPPORTED;
        live[n_live++] = span + i;
    }
    return LOGRA_OK;
}

}  // namespace

size_t logra_adamw_table_bytes(int64_t n) {
    return n < 0 || n > (1 << 20) ? 0 : static_cast<size_t>(n) * sizeof(AdamEntry);
}

logra_status logra_adamw_list_pack(int64_t n, const logra_adamw_tensor *tensors, void *table_host, size_t table_bytes,
                                   logra_adamw_list *list) {
    if (n < 0 || n > (1 << 20) || !list || (n > 0 && (!tensors || !table_host)) || !aligned_to(table_host, 8))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (table_bytes < logra_adamw_table_bytes(n)) return LOGRA_ERR_WORKSPACE;
    constexpr int64_t kMost = 1ll << 40;
    // the address ranges, in the table's memory before the table takes it
    static_assert(3 * sizeof(AdamSpan) <= sizeof(AdamEntry), "three ranges for an entry");
    AdamSpan *span = static_cast<AdamSpan *>(table_host);
    int64_t n_span = 0;
    for (int64_t i = 0; i < n; ++i) {
        const logra_adamw_tensor &t = tensors[i];
        if (t.rows < 0 || t.cols < 0) return LOGRA_ERR_INVALID_ARGUMENT;
        if (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || !dtype_ok(t.copy_dtype)) return LOGRA_ERR_UNSUPPORTED;
        if (t.rows == 0 || t.cols == 0) continue;
        if (t.rows > kMost || t.cols > kMost || t.rows > kMost / t.cols) return LOGRA_ERR_UNSUPPORTED;
        const struct {
            const void *p;
            int64_t ld;
            int dtype;
        } arrays[] = {{t.param, t.ld_param, t.param_dtype}, {t.grad, t.ld_grad, t.grad_dtype}, {t.copy, t.ld_copy, t.copy_dtype}};
        for (int a = 0; a < 3; ++a) {
            if (a == 2 && !t.copy) continue;
            if (arrays[a].ld > kMost / t.rows) return LOGRA_ERR_UNSUPPORTED;
            if (!adam_array(arrays[a].p, t.rows, t.cols, arrays[a].ld, arrays[a].dtype, span + n_span++))
                return LOGRA_ERR_INVALID_ARGUMENT;
        }
    }
    const logra_status apart = adam_apart(span, n_span);
    if (apart != LOGRA_OK) return apart;
    AdamEntry *table = static_cast<AdamEntry *>(table_host);
    logra_adamw_list out = {};
    for (int64_t i = 0; i < n; ++i) {
        const logra_adamw_tensor &t = tensors[i];
        AdamEntry e;
        e.param = reinterpret_cast<uint64_t>(t.param);
        e.grad = reinterpret_cast<uint64_t>(t.grad);
        e.copy = reinterpret_cast<uint64_t>(t.copy);
        e.rows = t.rows;
        e.cols = t.cols;
        e.ld_param = t.rows == 1 ? t.cols : t.ld_param;
        e.ld_grad = t.rows == 1 ? t.cols : t.ld_grad;
        e.ld_copy = t.rows == 1 ? t.cols : t.ld_copy;
        e.first = out.blocks;
        e.blocks = (t.rows * t.cols + kAdamBlock - 1) / kAdamBlock;
        e.param_bf16 = t.param_dtype == LOGRA_BF16;
        e.grad_bf16 = t.grad_dtype == LOGRA_BF16;
        e.copy_bf16 = t.copy_dtype == LOGRA_BF16;
        out.blocks += e.blocks;
        out.elements += t.rows * t.cols;
        if (out.elements > (kMost << 4)) return LOGRA_ERR_UNSUPPORTED;
        table[i] = e;
    }
    out.n = static_cast<int32_t>(n);
    *list = out;
    return LOGRA_OK;
}

logra_status logra_adamw(const logra_adamw_list *list, int state_bits, void *exp_avg, void *exp_avg_sq, float *scales,
                         double lr, double beta1, double beta2, double eps, double weight_decay, uint64_t step,
                         const float *norm, double max_norm, uint64_t seed, void *stream) {
    if (!list || list->n < 0 || list->blocks < 0 || (list->n > 0 && (!list->table || !aligned16(list->table))))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (state_bits != 8 && state_bits != 32) return LOGRA_ERR_UNSUPPORTED;
    if (!isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
        !isfinite(eps) || (eps > 0.0 && eps < 0x1p-126) || !isfinite(weight_decay) || step < 1 || !aligned_to(norm, 4) || !(max_norm >= 0.0))
        return LOGRA_ERR_INVALID_ARGUMENT;
    if (list->blocks == 0) return LOGRA_OK;
    if (!exp_avg || !aligned16(exp_avg) || !exp_avg_sq || !aligned16(exp_avg_sq) || exp_avg == exp_avg_sq ||
        (state_bits == 8 && (!scales || !aligned_to(scales, 4))))
        return LOGRA_ERR_INVALID_ARGUMENT;
    AdamCall c;
    c.table = static_cast<const AdamEntry *>(list->table);
    c.n = list->n;
    c.blocks = list->blocks;
    c.m = exp_avg;
    c.v = exp_avg_sq;
    c.scales = scales;
    c.norm = norm;
    c.max_norm = max_norm;
    c.beta1 = static_cast<float>(beta1);
    c.rest1 = static_cast<float>(1.0 - beta1);
    c.beta2 = static_cast<float>(beta2);
    c.rest2 = static_cast<float>(1.0 - beta2);
    // 1 - beta^t without the cancellation of a beta near 1 (beta 0: 1)
    const auto past = [&](double beta) { return beta > 0.0 ? -expm1(static_cast<double>(step) * log(beta)) : 1.0; };
    c.decay = static_cast<float>(lr * weight_decay);
    c.rate = static_cast<float>(lr / past(beta1));
    c.root_scale = static_cast<float>(1.0 / sqrt(past(beta2)));
    c.eps = static_cast<float>(eps);
    c.key = stream_key(seed, step, kAdamId);
    return from_hip(launch_adamw(c, state_bits, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
