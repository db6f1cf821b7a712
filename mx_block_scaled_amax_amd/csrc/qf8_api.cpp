// qf8_api.cpp -- the C ABI declared in include/qf8.h: argument validation and kernel dispatch.
// Every check happens on the host before anything is enqueued; nothing here synchronizes.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <limits.h>

#include "../../include/qf8.h"
#include "qf8_internal.h"

namespace {

constexpr int32_t kDelayedMagic = 0x51463844;  // "QF8D"
constexpr int kMaxHistory = 4096;
constexpr int kMaxGuard = 64;
constexpr int64_t kMaxMxDim = 1 << 24;   // keeps every per-wave buffer offset below 2^31
// The columnwise FP8 output of one 256-column tile spans 256 * rows bytes of one buffer
// descriptor; the parking offset 2^31 of idle lanes must stay outside it.
constexpr int64_t kMaxMxColRows = 1 << 23;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool fmt_ok(int fmt) { return fmt == QF8_E4M3 || fmt == QF8_E5M2; }
inline bool dtype_ok(int dt) { return dt == QF8_IN_BF16 || dt == QF8_IN_FP32; }
inline hipStream_t as_stream(void *s) { return (hipStream_t)s; }
// kernel launchers report an int status; the entry points return it as qf8_status
inline qf8_status status_of(int v) { return static_cast<qf8_status>(v); }

// rows, cols >= 0 and rows * cols representable
inline bool dims_ok(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return false;
    if (rows > 0 && cols > INT64_MAX / 16 / rows) return false;
    return true;
}

inline bool kind_ok(int kind) { return kind >= QF8_WEIGHT_NK && kind <= QF8_GROUPS_NK; }
inline bool out_ok(int out) { return out == QF8_OUT_BF16 || out == QF8_OUT_FP32; }
constexpr int64_t kMaxLaunchThreads = (int64_t)1 << 32;      // a launch counts its threads in 32 bits
constexpr int64_t kMaxRouteTokens = kMaxLaunchThreads / 64;  // one token to a wave
constexpr int64_t kMaxMatmulDim = 1 << 22;   // keeps every buffer offset of a tile below 2^31

constexpr int kMatmulFlags = QF8_FLAG_POW2_SCALES | QF8_FLAG_FP32_SUMS;
inline bool fp32_sums(int flags, int out) { return out == QF8_OUT_FP32 || (flags & QF8_FLAG_FP32_SUMS); }

// the sizes a product takes: rows of codes are read as whole dwords
inline bool matmul_dims_ok(int64_t m, int64_t n, int64_t k, int kind) {
    if (m < 0 || n < 0 || k < 0 || m >= (int64_t)1 << 31 || n > kMaxMatmulDim || k > kMaxMatmulDim) return false;
    return k % 4 == 0 && (kind != QF8_WEIGHT_KN || n % 4 == 0);
}

int check_delayed(const qf8_delayed_state *st) {
    if (!st) return QF8_ERR_NULL;
    if (st->magic != kDelayedMagic) return QF8_ERR_STATE;
    if (!st->history || !st->meta || !st->scale) return QF8_ERR_NULL;
    if (st->hist_len < 1 || st->hist_len > kMaxHistory || st->interval < 1 || st->n_guard < 0 ||
        st->n_guard > kMaxGuard || !fmt_ok(st->fmt) || st->step < 0 || st->estimator < 0 ||
        st->estimator > QF8_EST_MEAN || (st->flags & ~QF8_DELAYED_SPLIT_AMAX) != 0)
        return QF8_ERR_STATE;
    return QF8_OK;
}

}  // namespace

extern "C" {

const char *qf8_status_string(qf8_status status) {
    switch (status) {
        case QF8_OK: return "QF8_OK";
        case QF8_ERR_NULL: return "QF8_ERR_NULL: a required pointer is NULL";
        case QF8_ERR_ENUM: return "QF8_ERR_ENUM: format, dtype or rounding mode out of range";
        case QF8_ERR_SHAPE: return "QF8_ERR_SHAPE: size not accepted by this operation";
        case QF8_ERR_ALIGN: return "QF8_ERR_ALIGN: pointer not 16-byte aligned";
        case QF8_ERR_WORKSPACE: return "QF8_ERR_WORKSPACE: workspace missing or too small";
        case QF8_ERR_STATE: return "QF8_ERR_STATE: delayed-scaling state invalid";
        case QF8_ERR_HIP: return "QF8_ERR_HIP: kernel launch failed";
        default: return "unknown qf8 status";
    }
}

size_t qf8_workspace_bytes(int64_t rows, int64_t cols, qf8_dtype dtype) {
    (void)rows; (void)cols; (void)dtype;
    return qf8::kWorkspaceBytes;
}

qf8_status qf8_workspace_init(void *ws, size_t ws_bytes, void *stream) {
    if (!ws) return QF8_ERR_NULL;
    if (ws_bytes < qf8::kWorkspaceBytes) return QF8_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return QF8_ERR_ALIGN;
    return status_of(qf8::launch_fill_u32((uint32_t *)ws, (int64_t)(qf8::kWorkspaceBytes / 4), 0u,
                                          as_stream(stream)));
}

qf8_status qf8_set_onepass_grid(int grid) {
    if (grid < 0 || grid > qf8::kBarMaxGroups) return QF8_ERR_SHAPE;
    return status_of(qf8::set_onepass_grid(grid));
}

qf8_status qf8_cast_scaled(const void *x, qf8_dtype dtype, int64_t n, qf8_fmt fmt, const float *scale, uint8_t *q,
                           void *stream) {
    if (!dtype_ok(dtype) || !fmt_ok(fmt)) return QF8_ERR_ENUM;
    if (n < 0) return QF8_ERR_SHAPE;
    if (n == 0) return QF8_OK;
    if (!x || !scale || !q) return QF8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return QF8_ERR_ALIGN;
    return status_of(qf8::launch_cast_scaled(x, dtype, n, fmt, scale, q, qf8::stream_grid(n, dtype),
                                             as_stream(stream)));
}

qf8_status quantize_per_tensor(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_fmt fmt, uint8_t *q,
                               float *amax, float *scale, int32_t *nonfinite, void *ws, size_t ws_bytes,
                               void *stream) {
    if (!dtype_ok(dtype) || !fmt_ok(fmt)) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols)) return QF8_ERR_SHAPE;
    const int64_t n = rows * cols;
    if ((n > 0 && (!x || !q)) || !amax || !scale) return QF8_ERR_NULL;
    if (!ws || ws_bytes < qf8::kWorkspaceBytes) return QF8_ERR_WORKSPACE;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(amax, 4) || !aligned(scale, 4) || !aligned(ws, 16) ||
        (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    hipStream_t s = as_stream(stream);
    const int g1 = qf8::onepass_grid(n, dtype);
    if (g1 > 0)
        return status_of(qf8::launch_per_tensor_onepass(x, dtype, n, fmt, q, (uint32_t *)ws, amax, scale, nonfinite,
                                                        nullptr, g1, s));
    uint32_t *partials = (uint32_t *)ws + qf8::kPartialsOffsetWords;
    const int agrid = qf8::amax_grid(n, dtype);
    int st = qf8::launch_amax_partials(x, dtype, n, partials, agrid, s);
    if (st != QF8_OK) return status_of(st);
    return status_of(qf8::launch_cast_current(x, dtype, n, fmt, q, partials, agrid, amax, scale, nonfinite,
                                              qf8::stream_grid(n, dtype), s));
}

qf8_status quantize_per_tensor_noalloc(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_fmt fmt,
                                       uint8_t *q, float *amax, float *scale, int32_t *nonfinite, void *stream) {
    // the argument checks of quantize_per_tensor come first, so a bad call touches no device state
    if (!dtype_ok(dtype) || !fmt_ok(fmt)) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols)) return QF8_ERR_SHAPE;
    const int64_t n = rows * cols;
    if ((n > 0 && (!x || !q)) || !amax || !scale) return QF8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(amax, 4) || !aligned(scale, 4) ||
        (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    uint32_t *ws = nullptr;
    size_t ws_bytes = 0;
    const int st = qf8::scratch_workspace(&ws, &ws_bytes);
    if (st != QF8_OK) return status_of(st);
    if (ws_bytes < qf8::kWorkspaceBytes) return QF8_ERR_WORKSPACE;   // fixed size: every shape fits
    return status_of(quantize_per_tensor(x, dtype, rows, cols, fmt, q, amax, scale, nonfinite, ws, ws_bytes, stream));
}

qf8_status qf8_delayed_init_ex(qf8_delayed_state *st, float *history, int32_t *meta, float *scale, int hist_len,
                               int interval, int n_guard, qf8_fmt fmt, qf8_estimator estimator, int flags,
                               void *stream) {
    if (!st || !history || !meta || !scale) return QF8_ERR_NULL;
    if (!fmt_ok(fmt) || estimator < QF8_EST_MAX || estimator > QF8_EST_MEAN || (flags & ~QF8_DELAYED_SPLIT_AMAX))
        return QF8_ERR_ENUM;
    if (hist_len < 1 || hist_len > kMaxHistory || interval < 1 || n_guard < 0 || n_guard > kMaxGuard)
        return QF8_ERR_STATE;
    if (!aligned(history, 4) || !aligned(meta, 4) || !aligned(scale, 4)) return QF8_ERR_ALIGN;
    st->history = history;
    st->meta = meta;
    st->scale = scale;
    st->hist_len = hist_len;
    st->interval = interval;
    st->n_guard = n_guard;
    st->fmt = fmt;
    st->step = 0;
    st->magic = kDelayedMagic;
    st->estimator = estimator;
    st->flags = flags;
    st->reserved = 0;
    return status_of(qf8_delayed_reset(st, stream));
}

qf8_status qf8_delayed_init(qf8_delayed_state *st, float *history, int32_t *meta, float *scale, int hist_len,
                            int interval, int n_guard, qf8_fmt fmt, void *stream) {
    return status_of(qf8_delayed_init_ex(st, history, meta, scale, hist_len, interval, n_guard, fmt, QF8_EST_MAX, 0,
                                         stream));
}

qf8_status qf8_delayed_reset(qf8_delayed_state *st, void *stream) {
    int c = check_delayed(st);
    if (c != QF8_OK) return status_of(c);
    hipStream_t s = as_stream(stream);
    // cleared with a fill kernel rather than a memset, so a captured graph replays it correctly
    int r = qf8::launch_fill_u32((uint32_t *)st->history, st->hist_len, 0u, s);
    if (r == QF8_OK) r = qf8::launch_fill_u32((uint32_t *)st->meta, 4, 0u, s);
    if (r == QF8_OK) r = qf8::launch_fill_u32((uint32_t *)st->scale, 1, 0x3F800000u /* 1.0f */, s);
    if (r == QF8_OK) st->step = 0;
    return status_of(r);
}

qf8_status quantize_delayed(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_fmt fmt,
                            qf8_delayed_state *st, uint8_t *q, float *scale_used, float *amax_out, int32_t *nonfinite,
                            void *ws, size_t ws_bytes, void *stream) {
    int c = check_delayed(st);
    if (c != QF8_OK) return status_of(c);
    if (!dtype_ok(dtype) || !fmt_ok(fmt)) return QF8_ERR_ENUM;
    if (fmt != st->fmt) return QF8_ERR_STATE;     // the state was initialised for another format
    if (!dims_ok(rows, cols)) return QF8_ERR_SHAPE;
    const int64_t n = rows * cols;
    if (n > 0 && (!x || !q)) return QF8_ERR_NULL;
    if (!ws || ws_bytes < qf8::kWorkspaceBytes) return QF8_ERR_WORKSPACE;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(ws, 16) || (scale_used && !aligned(scale_used, 4)) ||
        (amax_out && !aligned(amax_out, 4)) || (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    hipStream_t s = as_stream(stream);
    uint32_t *partials = (uint32_t *)ws + qf8::kPartialsOffsetWords;
    uint32_t *slots = (uint32_t *)ws + qf8::kSlotsOffsetWords;
    const int grid = qf8::stream_grid(n, dtype);
    int r;
    if (st->step == 0) {
        // no history yet: current scaling (Eq.(1)-(2), no margin), then append this amax
        const int g1 = qf8::onepass_grid(n, dtype);
        int nparts = 0;
        if (g1 > 0) {              // the single-pass kernel leaves the amax in slot 0
            r = qf8::launch_per_tensor_onepass(x, dtype, n, st->fmt, q, (uint32_t *)ws, nullptr, scale_used, nullptr,
                                               slots, g1, s);
        } else {
            nparts = qf8::amax_grid(n, dtype);
            r = qf8::launch_amax_partials(x, dtype, n, partials, nparts, s);
            if (r == QF8_OK)
                r = qf8::launch_cast_current(x, dtype, n, st->fmt, q, partials, nparts, nullptr, scale_used, nullptr,
                                             grid, s);
        }
        if (r == QF8_OK)
            r = qf8::launch_delayed_finalize(slots, partials, nparts, st->history, st->meta, st->scale, st->hist_len,
                                             st->n_guard, st->fmt, 1, st->estimator, 0, amax_out, nonfinite, s);
    } else {
        // cast with the scale the history gave, fusing this step's amax into the pass (atomic
        // maxima in the workspace slots); then append the amax on update steps and compute the
        // next scale
        const int update = (st->step % st->interval) == 0;
        const int split = (st->flags & QF8_DELAYED_SPLIT_AMAX) != 0;
        int64_t lo = 0, hi = 0;
        if (split) {
            // piece k = (t - 1) mod I: [floor(k n / I), floor((k+1) n / I)), computed as
            // k (n / I) + k (n % I) / I so that no product exceeds I^2 < 2^62
            const int64_t I = st->interval, k = (st->step - 1) % I, qn = n / I, rn = n % I;
            lo = k * qn + (k * rn) / I;
            hi = (k + 1) * qn + ((k + 1) * rn) / I;
        }
        if (!update && !split && !scale_used && !amax_out && !nonfinite) {
            // a reuse step whose caller wants no diagnostics: the cast alone (its amax would
            // only be reported, and the state does not change)
            r = qf8::launch_cast_scaled(x, dtype, n, st->fmt, st->scale, q, grid, s);
            if (r == QF8_OK) st->step++;
            return status_of(r);
        }
        r = qf8::launch_cast_fused(x, dtype, n, st->fmt, st->scale, q, scale_used, slots, split, lo, hi, grid, s);
        if (r == QF8_OK)
            r = qf8::launch_delayed_finalize(slots, partials, 0, st->history, st->meta, st->scale, st->hist_len,
                                             st->n_guard, st->fmt, update, st->estimator, split, amax_out, nonfinite,
                                             s);
    }
    if (r == QF8_OK) st->step++;
    return status_of(r);
}

qf8_status quantize_block_ex(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, int block_rows,
                             int block_cols, qf8_fmt fmt, int flags, uint8_t *q, float *scales, float *amax,
                             int32_t *nonfinite, void *stream) {
    if (!dtype_ok(dtype) || !fmt_ok(fmt)) return QF8_ERR_ENUM;
    if (flags & ~QF8_FLAG_POW2_SCALES) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols)) return QF8_ERR_SHAPE;
    if (!((block_rows == 1 || block_rows == 128) && block_cols == 128)) return QF8_ERR_SHAPE;
    if (cols % (dtype == QF8_IN_BF16 ? 8 : 4) != 0) return QF8_ERR_SHAPE;
    if (rows > INT32_MAX || cols > INT32_MAX) return QF8_ERR_SHAPE;
    const int64_t ngroups = ((rows + block_rows - 1) / block_rows) * ((cols + 127) / 128);
    if (ngroups > INT32_MAX) return QF8_ERR_SHAPE;
    if (rows * cols == 0) return QF8_OK;
    if (!x || !q || !scales) return QF8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4) || (amax && !aligned(amax, 4)) ||
        (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    return status_of(qf8::launch_block(x, dtype, rows, cols, block_rows, fmt, flags & QF8_FLAG_POW2_SCALES, q, scales,
                                       amax, nonfinite, as_stream(stream)));
}

qf8_status quantize_block(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, int block_rows, int block_cols,
                          qf8_fmt fmt, uint8_t *q, float *scales, float *amax, int32_t *nonfinite, void *stream) {
    return status_of(quantize_block_ex(x, dtype, rows, cols, block_rows, block_cols, fmt, 0, q, scales, amax,
                                       nonfinite, stream));
}

qf8_status requantize_1x128_to_128x1(const uint8_t *q, const float *scales, int64_t rows, int64_t cols,
                                     qf8_fmt fmt_in, qf8_fmt fmt_out, int flags, uint8_t *qT, float *scalesT,
                                     int32_t *nonfinite, void *stream) {
    if (!fmt_ok(fmt_in) || !fmt_ok(fmt_out)) return QF8_ERR_ENUM;
    if (flags & ~QF8_FLAG_POW2_SCALES) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || rows % 16 != 0 || cols % 16 != 0) return QF8_ERR_SHAPE;
    if (rows > INT32_MAX || cols > INT32_MAX || ((rows + 127) / 128) * ((cols + 127) / 128) > INT32_MAX)
        return QF8_ERR_SHAPE;
    if (rows * cols == 0) return QF8_OK;
    if (!q || !scales || !qT || !scalesT) return QF8_ERR_NULL;
    if (!aligned(q, 16) || !aligned(qT, 16) || !aligned(scales, 4) || !aligned(scalesT, 4) ||
        (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    return status_of(qf8::launch_requant_t(q, scales, rows, cols, fmt_in, fmt_out, flags & QF8_FLAG_POW2_SCALES, qT,
                                           scalesT, nonfinite, as_stream(stream)));
}

qf8_status quantize_mx_dual(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_fmt fmt, qf8_mx_round rnd,
                            uint8_t *q_row, uint8_t *s_row, uint8_t *q_colT, uint8_t *s_colT, int32_t *nonfinite,
                            void *stream) {
    if (!dtype_ok(dtype) || !fmt_ok(fmt) || (rnd != QF8_MX_ROUND_DOWN && rnd != QF8_MX_ROUND_UP)) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || rows > kMaxMxDim || cols > kMaxMxDim) return QF8_ERR_SHAPE;
    if (!q_row && !q_colT) return QF8_ERR_NULL;
    if ((q_row && !s_row) || (q_colT && !s_colT)) return QF8_ERR_NULL;
    if (q_row && cols % 32 != 0) return QF8_ERR_SHAPE;
    if (q_colT && (rows % 32 != 0 || rows > kMaxMxColRows)) return QF8_ERR_SHAPE;
    if (cols % (dtype == QF8_IN_BF16 ? 8 : 4) != 0) return QF8_ERR_SHAPE;
    if (rows * cols == 0) return QF8_OK;
    if (!x) return QF8_ERR_NULL;
    if (!aligned(x, 16) || (q_row && !aligned(q_row, 16)) || (q_colT && !aligned(q_colT, 16)) ||
        (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    return status_of(qf8::launch_mx(x, dtype, rows, cols, fmt, rnd, q_row, s_row, q_colT, s_colT, nonfinite,
                                    as_stream(stream)));
}

qf8_status quantize_mxfp4_dual(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_mx_round rnd,
                               uint8_t *q_row, uint8_t *s_row, uint8_t *q_colT, uint8_t *s_colT, int32_t *nonfinite,
                               void *stream) {
    if (!dtype_ok(dtype) || (rnd != QF8_MX_ROUND_DOWN && rnd != QF8_MX_ROUND_UP)) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || rows > kMaxMxDim || cols > kMaxMxDim) return QF8_ERR_SHAPE;
    if (!q_row && !q_colT) return QF8_ERR_NULL;
    if ((q_row && !s_row) || (q_colT && !s_colT)) return QF8_ERR_NULL;
    if (q_row && cols % 32 != 0) return QF8_ERR_SHAPE;
    if (q_colT && rows % 32 != 0) return QF8_ERR_SHAPE;
    if (cols % (dtype == QF8_IN_BF16 ? 8 : 4) != 0) return QF8_ERR_SHAPE;
    if (rows * cols == 0) return QF8_OK;
    if (!x) return QF8_ERR_NULL;
    if (!aligned(x, 16) || (q_row && !aligned(q_row, 16)) || (q_colT && !aligned(q_colT, 16)) ||
        (nonfinite && !aligned(nonfinite, 4)))
        return QF8_ERR_ALIGN;
    return status_of(qf8::launch_mxfp4(x, dtype, rows, cols, rnd, q_row, s_row, q_colT, s_colT, nonfinite,
                                       as_stream(stream)));
}

qf8_status quantize_nvfp4(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, const float *amax_in,
                          uint8_t *q, uint8_t *s_blk, float *tensor_scale, float *amax_out, int32_t *nonfinite,
                          void *ws, size_t ws_bytes, void *stream) {
    if (!dtype_ok(dtype)) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || cols % 16 != 0) return QF8_ERR_SHAPE;
    const int64_t n = rows * cols;
    if ((n > 0 && (!x || !q || !s_blk)) || !tensor_scale) return QF8_ERR_NULL;
    if (!amax_in && (!ws || ws_bytes < qf8::kWorkspaceBytes)) return QF8_ERR_WORKSPACE;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(tensor_scale, 4) || (amax_in && !aligned(amax_in, 4)) ||
        (amax_out && !aligned(amax_out, 4)) || (nonfinite && !aligned(nonfinite, 4)) || (ws && !aligned(ws, 16)))
        return QF8_ERR_ALIGN;
    hipStream_t s = as_stream(stream);
    uint32_t *partials = ws ? (uint32_t *)ws + qf8::kPartialsOffsetWords : nullptr;
    int nparts = 0;
    if (!amax_in && n > 0) {
        // large tensors: amax and cast in one read (the single-pass kernel of per-tensor scaling)
        const int g1 = qf8::onepass_grid(n, dtype);
        if (g1 > 0)
            return status_of(qf8::launch_nvfp4_onepass(x, dtype, n, q, s_blk, (uint32_t *)ws, tensor_scale, amax_out,
                                                       nonfinite, g1, s));
        // otherwise the read-only amax pass first
        nparts = qf8::amax_grid(n, dtype);
        const int r = qf8::launch_amax_partials(x, dtype, n, partials, nparts, s);
        if (r != QF8_OK) return status_of(r);
    }
    return status_of(qf8::launch_nvfp4(x, dtype, n, partials, nparts, amax_in, q, s_blk, tensor_scale, amax_out,
                                       nonfinite, s));
}

qf8_status dequantize_mxfp4(const uint8_t *q, const uint8_t *sb, int64_t rows, int64_t cols, void *out,
                            qf8_out_dtype out_dtype, void *stream) {
    if (out_dtype != QF8_OUT_BF16 && out_dtype != QF8_OUT_FP32) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || cols % 32 != 0 || rows * cols >= ((int64_t)1 << 36)) return QF8_ERR_SHAPE;
    const int64_t n = rows * cols;
    if (n == 0) return QF8_OK;
    if (!q || !sb || !out) return QF8_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16)) return QF8_ERR_ALIGN;
    return status_of(qf8::launch_dequant_fp4(0, q, sb, nullptr, n, out, out_dtype, as_stream(stream)));
}

qf8_status dequantize_nvfp4(const uint8_t *q, const uint8_t *s_blk, const float *tensor_scale, int64_t rows,
                            int64_t cols, void *out, qf8_out_dtype out_dtype, void *stream) {
    if (out_dtype != QF8_OUT_BF16 && out_dtype != QF8_OUT_FP32) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || cols % 16 != 0 || rows * cols >= ((int64_t)1 << 36)) return QF8_ERR_SHAPE;
    const int64_t n = rows * cols;
    if (n == 0) return QF8_OK;
    if (!q || !s_blk || !tensor_scale || !out) return QF8_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(tensor_scale, 4)) return QF8_ERR_ALIGN;
    return status_of(qf8::launch_dequant_fp4(1, q, s_blk, tensor_scale, n, out, out_dtype, as_stream(stream)));
}

}  // extern "C"

// ---- dequantization and error statistics ---------------------------------------------------
namespace {
constexpr int64_t kMaxDequantElems = (int64_t)1 << 33;   // 4-code units stay below 2^31

int check_dequant(const uint8_t *q, int64_t rows, int64_t cols, int fmt, void *out, int out_dtype, const void *x,
                  int x_dtype, qf8_error_stats *stats, void *ws, size_t ws_bytes) {
    if (!fmt_ok(fmt)) return QF8_ERR_ENUM;
    if (out && out_dtype != QF8_OUT_BF16 && out_dtype != QF8_OUT_FP32) return QF8_ERR_ENUM;
    if (stats && !dtype_ok(x_dtype)) return QF8_ERR_ENUM;
    if (!dims_ok(rows, cols) || rows * cols >= kMaxDequantElems) return QF8_ERR_SHAPE;
    if (!out && !stats) return QF8_ERR_NULL;
    const int64_t n = rows * cols;
    if (n > 0 && !q) return QF8_ERR_NULL;
    if (stats && ((n > 0 && !x) || !ws)) return QF8_ERR_NULL;
    if (stats && ws_bytes < qf8::kWorkspaceBytes) return QF8_ERR_WORKSPACE;
    if (!aligned(q, 16) || (out && !aligned(out, 16)) || (x && !aligned(x, 16)) || (stats && !aligned(stats, 8)) ||
        (ws && !aligned(ws, 16)))
        return QF8_ERR_ALIGN;
    return QF8_OK;
}
}  // namespace

extern "C" {

qf8_status dequantize_scaled(const uint8_t *q, int64_t n, qf8_fmt fmt, const float *scale, void *out,
                             qf8_out_dtype out_dtype, const void *x, qf8_dtype x_dtype, qf8_error_stats *stats,
                             void *ws, size_t ws_bytes, void *stream) {
    int c = check_dequant(q, 1, n, fmt, out, out_dtype, x, x_dtype, stats, ws, ws_bytes);
    if (c != QF8_OK) return status_of(c);
    if (!scale) return QF8_ERR_NULL;
    if (!aligned(scale, 4)) return QF8_ERR_ALIGN;
    if (n == 0 && !stats) return QF8_OK;
    return status_of(qf8::launch_dequant(0, fmt, q, 1, n, 1, scale, nullptr, out, out_dtype, x, x_dtype, stats, ws,
                                         as_stream(stream)));
}

qf8_status dequantize_block(const uint8_t *q, int64_t rows, int64_t cols, int block_rows, int block_cols, qf8_fmt fmt,
                            const float *scales, void *out, qf8_out_dtype out_dtype, const void *x, qf8_dtype x_dtype,
                            qf8_error_stats *stats, void *ws, size_t ws_bytes, void *stream) {
    int c = check_dequant(q, rows, cols, fmt, out, out_dtype, x, x_dtype, stats, ws, ws_bytes);
    if (c != QF8_OK) return status_of(c);
    if (!((block_rows == 1 || block_rows == 128) && block_cols == 128)) return QF8_ERR_SHAPE;
    if (cols % 4 != 0) return QF8_ERR_SHAPE;
    if (rows * cols > 0 && !scales) return QF8_ERR_NULL;
    if (scales && !aligned(scales, 4)) return QF8_ERR_ALIGN;
    if (rows * cols == 0 && !stats) return QF8_OK;
    return status_of(qf8::launch_dequant(1, fmt, q, rows, cols, block_rows, scales, nullptr, out, out_dtype, x,
                                         x_dtype, stats, ws, as_stream(stream)));
}

qf8_status dequantize_mx(const uint8_t *q, const uint8_t *s, int64_t rows, int64_t cols, qf8_fmt fmt, void *out,
                         qf8_out_dtype out_dtype, const void *x, qf8_dtype x_dtype, qf8_error_stats *stats, void *ws,
                         size_t ws_bytes, void *stream) {
    int c = check_dequant(q, rows, cols, fmt, out, out_dtype, x, x_dtype, stats, ws, ws_bytes);
    if (c != QF8_OK) return status_of(c);
    if (cols % 32 != 0) return QF8_ERR_SHAPE;
    if (rows * cols > 0 && !s) return QF8_ERR_NULL;
    if (rows * cols == 0 && !stats) return QF8_OK;
    return status_of(qf8::launch_dequant(2, fmt, q, rows, cols, 1, nullptr, s, out, out_dtype, x, x_dtype, stats, ws,
                                         as_stream(stream)));
}

size_t matmul_block_workspace_bytes(int64_t m, int64_t n, int64_t k, qf8_operand kind, qf8_out_dtype out_dtype) {
    if (!kind_ok(kind) || !out_ok(out_dtype) || !matmul_dims_ok(m, n, k, kind)) return 0;
    return qf8::matmul_workspace(m, n, k, kind, out_dtype == QF8_OUT_FP32);
}

qf8_status matmul_block(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int64_t m, int64_t n,
                        int64_t k, qf8_fmt fmt_a, qf8_fmt fmt_b, qf8_operand kind, int flags, void *y,
                        qf8_out_dtype out_dtype, void *ws, size_t ws_bytes, void *stream) {
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b) || !kind_ok(kind) || !out_ok(out_dtype) || (flags & ~kMatmulFlags))
        return QF8_ERR_ENUM;
    if (!matmul_dims_ok(m, n, k, kind)) return QF8_ERR_SHAPE;
    if (m == 0 || n == 0) return QF8_OK;
    if (!y || (k > 0 && (!a || !sa || !b || !sb))) return QF8_ERR_NULL;
    const size_t need = qf8::matmul_workspace(m, n, k, kind, fp32_sums(flags, out_dtype));
    if (need > 0 && (!ws || ws_bytes < need)) return QF8_ERR_WORKSPACE;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(sa, 4) || !aligned(sb, 4) || !aligned(ws, 16))
        return QF8_ERR_ALIGN;
    qf8::MatmulArgs p = {};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.y = y;
    p.m = m; p.n = (int)n; p.k = k; p.a_rows = m;
    p.mode = qf8::kMatmulDense;
    p.out_bf16 = out_dtype == QF8_OUT_BF16;
    p.fp32_sums = fp32_sums(flags, out_dtype);
    return status_of(qf8::launch_matmul(p, fmt_a, fmt_b, kind, flags & QF8_FLAG_POW2_SCALES, (float *)ws, as_stream(stream)));
}

qf8_status matmul_block_experts(const uint8_t *a, const float *sa, int64_t tokens, const uint8_t *b, const float *sb,
                                const int32_t *offsets, int experts, const int32_t *rows, int64_t nrows, int64_t n,
                                int64_t k, qf8_fmt fmt_a, qf8_fmt fmt_b, qf8_operand kind, int flags, void *y,
                                qf8_out_dtype out_dtype, void *stream) {
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b) || (kind != QF8_WEIGHT_NK && kind != QF8_WEIGHT_KN) || !out_ok(out_dtype) ||
        (flags & ~kMatmulFlags))
        return QF8_ERR_ENUM;
    if (!matmul_dims_ok(nrows, n, k, kind) || tokens < 0 || experts < 1 || experts > qf8::kMaxExperts) return QF8_ERR_SHAPE;
    if (rows ? tokens >= (int64_t)1 << 31 || (k > 0 && tokens > 0xFFFFFFFFll / k) : tokens != nrows) return QF8_ERR_SHAPE;
    if (nrows == 0 || n == 0) return QF8_OK;
    if (!y || !offsets || (k > 0 && (!b || !sb)) || (k > 0 && tokens > 0 && (!a || !sa))) return QF8_ERR_NULL;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4))
        return QF8_ERR_ALIGN;
    qf8::MatmulArgs p = {};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.offsets = offsets; p.rows = rows; p.y = y;
    p.m = nrows; p.n = (int)n; p.k = tokens > 0 ? k : 0; p.a_rows = tokens;      // no tokens: every row is zeros
    p.experts = experts;
    p.mode = qf8::kMatmulExperts;
    p.out_bf16 = out_dtype == QF8_OUT_BF16;
    p.fp32_sums = fp32_sums(flags, out_dtype);
    return status_of(qf8::launch_matmul(p, fmt_a, fmt_b, kind, flags & QF8_FLAG_POW2_SCALES, nullptr, as_stream(stream)));
}

qf8_status matmul_block_experts_wgrad(const uint8_t *at, const float *sat, const uint8_t *bt, const float *sbt,
                                      const int32_t *offsets, int experts, int64_t nrows, int64_t m, int64_t n,
                                      qf8_fmt fmt_a, qf8_fmt fmt_b, int flags, void *y, qf8_out_dtype out_dtype,
                                      void *stream) {
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b) || !out_ok(out_dtype) || (flags & ~kMatmulFlags)) return QF8_ERR_ENUM;
    if (!matmul_dims_ok(m, n, nrows, QF8_GROUPS_NK) || experts < 1 || experts > qf8::kMaxExperts) return QF8_ERR_SHAPE;
    if (m == 0 || n == 0) return QF8_OK;
    if (!y || !offsets || (nrows > 0 && (!at || !sat || !bt || !sbt))) return QF8_ERR_NULL;
    if (!aligned(at, 16) || !aligned(bt, 16) || !aligned(y, 16) || !aligned(sat, 4) || !aligned(sbt, 4) ||
        !aligned(offsets, 4))
        return QF8_ERR_ALIGN;
    qf8::MatmulArgs p = {};
    p.a = at; p.sa = sat; p.b = bt; p.sb = sbt; p.offsets = offsets; p.y = y;
    p.m = m; p.n = (int)n; p.k = nrows; p.a_rows = m;
    p.experts = experts;
    p.mode = qf8::kMatmulExpertsK;
    p.out_bf16 = out_dtype == QF8_OUT_BF16;
    p.fp32_sums = fp32_sums(flags, out_dtype);
    return status_of(qf8::launch_matmul(p, fmt_a, fmt_b, QF8_GROUPS_NK, flags & QF8_FLAG_POW2_SCALES, nullptr,
                                        as_stream(stream)));
}

qf8_status route_experts(const void *logits, qf8_dtype dtype, int64_t tokens, int experts, int top_k, qf8_score score,
                         const float *bias, int groups, int top_groups, int renorm, float scale, int32_t *ids,
                         float *weights, void *stream) {
    if (!dtype_ok(dtype) || (score != QF8_SCORE_SOFTMAX && score != QF8_SCORE_SIGMOID)) return QF8_ERR_ENUM;
    if (tokens < 0 || tokens >= kMaxRouteTokens || experts < 1 || experts > qf8::kMaxExperts || groups < 1 ||
        groups > qf8::kMaxExpertGroups || experts % groups != 0 || top_groups < 1 || top_groups > groups || top_k < 1 ||
        top_k > qf8::kMaxTopK || top_k > experts / groups * top_groups)
        return QF8_ERR_SHAPE;
    if (tokens == 0) return QF8_OK;
    if (!logits || !ids || !weights) return QF8_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return QF8_ERR_ALIGN;
    qf8::RouteArgs p = {};
    p.logits = logits; p.bias = bias; p.ids = ids; p.weights = weights;
    p.tokens = tokens; p.experts = experts; p.top_k = top_k; p.score = score;
    p.groups = top_groups == groups ? 1 : groups;      // all groups open: the same as none
    p.top_groups = p.groups == 1 ? 1 : top_groups;
    p.renorm = renorm != 0; p.scale = scale;
    return status_of(qf8::launch_route(p, dtype, 0, as_stream(stream)));
}

qf8_status route_experts_backward(const void *logits, qf8_dtype dtype, int64_t tokens, int experts, const int32_t *ids,
                                  const float *dweights, int top_k, qf8_score score, int renorm, float scale,
                                  void *dlogits, void *stream) {
    if (!dtype_ok(dtype) || (score != QF8_SCORE_SOFTMAX && score != QF8_SCORE_SIGMOID)) return QF8_ERR_ENUM;
    if (tokens < 0 || tokens >= kMaxRouteTokens || experts < 1 || experts > qf8::kMaxExperts || top_k < 1 ||
        top_k > qf8::kMaxTopK || top_k > experts)
        return QF8_ERR_SHAPE;
    if (tokens == 0) return QF8_OK;
    if (!logits || !ids || !dweights || !dlogits) return QF8_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(dweights, 4) || !aligned(dlogits, 4)) return QF8_ERR_ALIGN;
    qf8::RouteArgs p = {};
    p.logits = logits; p.ids = const_cast<int32_t *>(ids); p.dweights = dweights; p.dlogits = dlogits;
    p.tokens = tokens; p.experts = experts; p.top_k = top_k; p.score = score; p.renorm = renorm != 0; p.scale = scale;
    return status_of(qf8::launch_route(p, dtype, 1, as_stream(stream)));
}

int64_t order_experts_rows(int64_t tokens, int top_k, int experts, int align) {
    if (tokens < 0 || tokens >= (int64_t)1 << 31 || top_k < 1 || top_k > qf8::kMaxTopK || experts < 1 ||
        experts > qf8::kMaxExperts || align < 1 || align > 1024)
        return 0;
    const int64_t n = tokens * top_k;
    return (n + (experts < n ? experts : n) * (align - 1) + align - 1) / align * align;
}

size_t order_experts_workspace_bytes(int64_t tokens, int top_k, int experts) {
    return order_experts_rows(tokens, top_k, experts, 1) == 0 ? 0 : qf8::order_workspace(tokens * top_k, experts);
}

qf8_status order_experts(const int32_t *ids, int64_t tokens, int top_k, int experts, int align, int32_t *offsets,
                         int32_t *rows, int64_t nrows, int32_t *slots, void *ws, size_t ws_bytes, void *stream) {
    if (tokens < 0 || tokens >= (int64_t)1 << 31 || top_k < 1 || top_k > qf8::kMaxTopK || experts < 1 ||
        experts > qf8::kMaxExperts || align < 1 || align > 1024)
        return QF8_ERR_SHAPE;
    if (nrows < order_experts_rows(tokens, top_k, experts, align) || nrows >= (int64_t)1 << 31) return QF8_ERR_SHAPE;
    if (!offsets || (tokens > 0 && (!ids || !slots)) || (nrows > 0 && !rows)) return QF8_ERR_NULL;
    const size_t need = qf8::order_workspace(tokens * top_k, experts);
    if (need > 0 && (!ws || ws_bytes < need)) return QF8_ERR_WORKSPACE;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(ws, 16))
        return QF8_ERR_ALIGN;
    qf8::OrderArgs p = {};
    p.ids = ids; p.offsets = offsets; p.rows = rows; p.slots = slots; p.counts = (int32_t *)ws;
    p.n = tokens * top_k; p.nrows = nrows; p.top_k = top_k; p.experts = experts; p.align = align;
    return status_of(qf8::launch_order(p, as_stream(stream)));
}

namespace {
// A workgroup of 256 threads takes one token.
int check_combine(qf8_dtype dtype, int64_t nrows, int64_t dim, int64_t tokens, int top_k) {
    if (!dtype_ok(dtype)) return QF8_ERR_ENUM;
    if (tokens < 0 || tokens >= kMaxLaunchThreads / 256 || nrows < 0 || nrows >= (int64_t)1 << 31 || dim < 0 ||
        dim >= (int64_t)1 << 31 || top_k < 1 || top_k > qf8::kMaxTopK)
        return QF8_ERR_SHAPE;
    return QF8_OK;
}
}  // namespace

qf8_status combine_experts(const void *x, qf8_dtype dtype, int64_t nrows, int64_t dim, const float *weights,
                           const int32_t *slots, int64_t tokens, int top_k, void *y, void *stream) {
    const int c = check_combine(dtype, nrows, dim, tokens, top_k);
    if (c != QF8_OK) return status_of(c);
    if (tokens == 0 || dim == 0) return QF8_OK;
    if ((nrows > 0 && !x) || !weights || !slots || !y) return QF8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weights, 4) || !aligned(slots, 4)) return QF8_ERR_ALIGN;
    qf8::CombineArgs p = {};
    p.x = x; p.weights = weights; p.slots = slots; p.y = y;
    p.tokens = tokens; p.nrows = nrows; p.dim = dim; p.top_k = top_k;
    return status_of(qf8::launch_combine(p, dtype, 0, as_stream(stream)));
}

qf8_status combine_experts_backward(const void *dy, const void *x, qf8_dtype dtype, int64_t nrows, int64_t dim,
                                    const float *weights, const int32_t *slots, const int32_t *rows, int64_t tokens,
                                    int top_k, void *dx, float *dweights, void *stream) {
    const int c = check_combine(dtype, nrows, dim, tokens, top_k);
    if (c != QF8_OK) return status_of(c);
    if (tokens + (nrows + 63) / 64 >= kMaxLaunchThreads / 256) return QF8_ERR_SHAPE;       // and 64 rows for the padding
    if (tokens == 0 && (nrows == 0 || dim == 0)) return QF8_OK;
    if ((tokens > 0 && (!weights || !slots || !dweights || (dim > 0 && !dy))) || (nrows > 0 && (!rows || (dim > 0 && (!x || !dx)))))
        return QF8_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dx, 16) || !aligned(weights, 4) || !aligned(slots, 4) ||
        !aligned(rows, 4) || !aligned(dweights, 4))
        return QF8_ERR_ALIGN;
    qf8::CombineArgs p = {};
    p.x = x; p.dy = dy; p.weights = weights; p.slots = slots; p.rows = rows; p.dx = dx; p.dweights = dweights;
    p.tokens = tokens; p.nrows = nrows; p.dim = dim; p.top_k = top_k;
    return status_of(qf8::launch_combine(p, dtype, 1, as_stream(stream)));
}

}  // extern "C"

// ---- around the expert layer ---------------------------------------------------------------------
namespace {
inline bool act_ok(int act) { return act == QF8_ACT_SILU || act == QF8_ACT_GELU; }

// the sizes of a norm's rows, forward and backward
inline bool norm_dims_ok(int64_t rows, int64_t cols) {
    return dims_ok(rows, cols) && cols % 8 == 0 && cols <= qf8::kMaxNormCols;
}

// gated activation: n columns of results, in one run (forward) or two
int check_gate(const void *dy, const void *x, int dtype, int64_t rows, int64_t cols, int act, int fmt, int flags,
               const uint8_t *q, const float *scales, const void *y, const int32_t *nonfinite, int backward) {
    if (!dtype_ok(dtype) || !act_ok(act) || (q && !fmt_ok(fmt)) || (flags & ~QF8_FLAG_POW2_SCALES)) return QF8_ERR_ENUM;
    if (rows < 0 || cols < 0 || cols % 8 != 0 || cols >= (int64_t)1 << 30 || rows >= (int64_t)1 << 31 ||
        rows * ((cols + 127) / 128) >= kMaxLaunchThreads / 16)     // up to eight threads to a group, in whole workgroups
        return QF8_ERR_SHAPE;
    if (backward && q && cols % 128 != 0) return QF8_ERR_SHAPE;
    if (rows * cols == 0) return QF8_OK;
    if (!x || (backward && !dy) || !q != !scales || (!q && !y)) return QF8_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(q, 16) || !aligned(y, 16) || !aligned(scales, 4) ||
        !aligned(nonfinite, 4))
        return QF8_ERR_ALIGN;
    return QF8_OK;
}

int gate(const void *dy, const void *x, int dtype, int64_t rows, int64_t cols, int act, int fmt, int flags, uint8_t *q,
         float *scales, void *y, int32_t *nonfinite, int backward, void *stream) {
    const int c = check_gate(dy, x, dtype, rows, cols, act, fmt, flags, q, scales, y, nonfinite, backward);
    if (c != QF8_OK || rows * cols == 0) return c;
    qf8::GateArgs p = {};
    p.x = x; p.dy = dy; p.y = y; p.q = q; p.scales = scales; p.nonfinite = nonfinite;
    p.cols = cols;
    p.gcols = (uint32_t)((cols + 127) / 128);
    p.groups = (uint32_t)rows * p.gcols;
    p.fmt = fmt; p.pow2 = flags & QF8_FLAG_POW2_SCALES;
    return qf8::launch_gate(p, dtype, act, backward, as_stream(stream));
}

// Bytes of the sums, and the values of one of them; -1: refused.
int64_t clip_workspace(const qf8_grad *grads, int count, int64_t *chunk) {
    if (count < 0 || count > 1 << 20 || (count > 0 && !grads)) return -1;
    int64_t total = 0, sums = 0;
    for (int i = 0; i < count; ++i) {
        if (grads[i].n < 0 || grads[i].n >= (int64_t)1 << 36) return -1;
        total += grads[i].n;
    }
    *chunk = qf8::clip_chunk(total);
    for (int i = 0; i < count; ++i) sums += (grads[i].n + *chunk - 1) / *chunk;
    return (sums * 8 + 15) / 16 * 16 + 16;
}
}  // namespace

extern "C" {

qf8_status rms_norm_quantize(const void *x, qf8_dtype dtype, const void *residual, qf8_dtype residual_dtype,
                             const void *weight, qf8_dtype weight_dtype, int64_t rows, int64_t cols, float eps, qf8_fmt fmt,
                             int flags, uint8_t *q, float *scales, void *h, void *y, float *rstd, int32_t *nonfinite,
                             void *stream) {
    if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || (residual && !dtype_ok(residual_dtype)) || (q && !fmt_ok(fmt)) ||
        (flags & ~QF8_FLAG_POW2_SCALES))
        return QF8_ERR_ENUM;
    if (!norm_dims_ok(rows, cols) || !(eps >= 1.17549435e-38f) || !(eps <= 3.40282346638528859812e+38f)) return QF8_ERR_SHAPE;
    if (rows * cols == 0) return QF8_OK;
    if (!x || !weight || !q != !scales || (!q && !y) || (residual && !h)) return QF8_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(q, 16) || !aligned(h, 16) ||
        !aligned(y, 16) || !aligned(scales, 4) || !aligned(rstd, 4) || !aligned(nonfinite, 4))
        return QF8_ERR_ALIGN;
    qf8::NormArgs p = {};
    p.x = x; p.residual = residual; p.weight = weight; p.q = q; p.scales = scales; p.h = h; p.y = y; p.rstd = rstd;
    p.nonfinite = nonfinite;
    p.rows = rows; p.cols = cols; p.gcols = (cols + 127) / 128;
    p.eps = eps;
    p.inv_cols = 1.0f / (float)cols;
    p.inv_cols_rest = (float)(1.0 / (double)cols - (double)p.inv_cols);
    p.w_fp32 = weight_dtype == QF8_IN_FP32;
    p.fmt = fmt; p.pow2 = flags & QF8_FLAG_POW2_SCALES;
    return status_of(qf8::launch_norm(p, dtype, residual_dtype, as_stream(stream)));
}

size_t rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    return norm_dims_ok(rows, cols) ? (size_t)(qf8::norm_backward_groups(rows, cols) * cols * 4) : 0;
}

qf8_status rms_norm_backward(const void *dy, qf8_dtype dtype, const void *h, qf8_dtype h_dtype, const float *rstd,
                             const void *weight, qf8_dtype weight_dtype, const void *dres, int64_t rows, int64_t cols,
                             void *dx, float *dweight, void *ws, size_t ws_bytes, void *stream) {
    if (!dtype_ok(dtype) || !dtype_ok(h_dtype) || !dtype_ok(weight_dtype)) return QF8_ERR_ENUM;
    if (!norm_dims_ok(rows, cols)) return QF8_ERR_SHAPE;
    if (cols == 0 || (rows == 0 && !dweight)) return QF8_OK;
    if (rows > 0 && (!dy || !h || !rstd || !weight || !dx)) return QF8_ERR_NULL;
    const size_t need = dweight ? rms_norm_backward_workspace_bytes(rows, cols) : 0;
    if (need > 0 && (!ws || ws_bytes < need)) return QF8_ERR_WORKSPACE;
    if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(dres, 16) || !aligned(dx, 16) ||
        !aligned(ws, 16) || !aligned(rstd, 4) || !aligned(dweight, 4))
        return QF8_ERR_ALIGN;
    qf8::NormArgs p = {};
    p.dy = dy; p.hin = h; p.rstd_in = rstd; p.weight = weight; p.dres = dres; p.dx = dx;
    p.partial = dweight ? (float *)ws : nullptr;
    p.rows = rows; p.cols = cols;
    p.inv_cols = 1.0f / (float)cols;
    p.w_fp32 = weight_dtype == QF8_IN_FP32;
    return status_of(qf8::launch_norm_backward(p, dtype, h_dtype, dweight, as_stream(stream)));
}

qf8_status gated_act_quantize(const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_act act, qf8_fmt fmt, int flags,
                              uint8_t *q, float *scales, void *y, int32_t *nonfinite, void *stream) {
    return status_of(gate(nullptr, x, dtype, rows, cols, act, fmt, flags, q, scales, y, nonfinite, 0, stream));
}

qf8_status gated_act_backward(const void *dy, const void *x, qf8_dtype dtype, int64_t rows, int64_t cols, qf8_act act,
                              qf8_fmt fmt, int flags, uint8_t *q, float *scales, void *dx, int32_t *nonfinite, void *stream) {
    return status_of(gate(dy, x, dtype, rows, cols, act, fmt, flags, q, scales, dx, nonfinite, 1, stream));
}

static bool layer_dims_ok(int64_t tokens, int top_k, int experts, int64_t dim, int64_t hidden) {
    const auto side_ok = [](int64_t n) { return n >= 0 && n % 16 == 0 && n <= qf8::kMaxLayerDim; };
    return tokens >= 0 && tokens <= qf8::kLayerTokens && top_k >= 1 && top_k <= qf8::kMaxTopK &&
           tokens * top_k <= qf8::kLayerChoices && experts >= 1 && experts <= qf8::kMaxExperts && side_ok(dim) && side_ok(hidden);
}

size_t expert_layer_tokens_workspace_bytes(int64_t tokens, int top_k, int experts, int64_t dim, int64_t hidden) {
    return layer_dims_ok(tokens, top_k, experts, dim, hidden) ? qf8::layer_workspace(tokens, top_k, experts, dim, hidden) : 0;
}

qf8_status expert_layer_tokens(const void *x, int64_t tokens, int64_t dim, const uint8_t *w1, const float *s1,
                               const uint8_t *w2, const float *s2, int experts, int64_t hidden, qf8_fmt fmt, qf8_act act,
                               const int32_t *ids, const float *weights, int top_k, void *y, void *ws, size_t ws_bytes,
                               void *stream) {
    if (!fmt_ok(fmt) || !act_ok(act)) return QF8_ERR_ENUM;
    if (!layer_dims_ok(tokens, top_k, experts, dim, hidden)) return QF8_ERR_SHAPE;
    if (tokens == 0 || dim == 0) return QF8_OK;
    if (!x || !ids || !weights || !y || (hidden > 0 && (!w1 || !s1 || !w2 || !s2))) return QF8_ERR_NULL;
    if (!ws || ws_bytes < qf8::layer_workspace(tokens, top_k, experts, dim, hidden)) return QF8_ERR_WORKSPACE;
    if (!aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) || !aligned(y, 16) || !aligned(ws, 16) || !aligned(s1, 4) ||
        !aligned(s2, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return QF8_ERR_ALIGN;
    qf8::LayerArgs p = {};
    p.x = (const uint16_t *)x; p.w1 = w1; p.s1 = s1; p.w2 = w2; p.s2 = s2; p.ids = ids; p.weights = weights;
    p.y = (uint16_t *)y;
    p.tokens = (int)tokens; p.top_k = top_k; p.experts = experts; p.dim = (int)dim; p.hidden = (int)hidden;
    return status_of(qf8::launch_layer(p, fmt, act, ws, as_stream(stream)));
}

size_t clip_grads_workspace_bytes(const qf8_grad *grads, int count) {
    int64_t chunk;
    const int64_t need = clip_workspace(grads, count, &chunk);
    return need < 0 ? 0 : (size_t)need;
}

qf8_status clip_grads(const qf8_grad *grads, int count, double max_norm, float *norm, int32_t *nonfinite, void *ws,
                      size_t ws_bytes, void *stream) {
    if (count > 0 && !grads) return QF8_ERR_NULL;
    int64_t chunk = 0;
    const int64_t need = clip_workspace(grads, count, &chunk);
    if (need < 0 || !(max_norm > 0.0)) return QF8_ERR_SHAPE;
    int written = 0, held = 0;
    for (int i = 0; i < count; ++i) {
        const qf8_grad &g = grads[i];
        if (!dtype_ok(g.dtype)) return QF8_ERR_ENUM;
        if (g.n == 0) continue;
        if (!g.g) return QF8_ERR_NULL;
        const uintptr_t a = g.dtype == QF8_IN_FP32 ? 4 : 2;
        if (!aligned(g.g, a) || !aligned(g.out, a)) return QF8_ERR_ALIGN;
        ++held;
        written += g.out != nullptr;
    }
    if (written != 0 && written != held) return QF8_ERR_NULL;
    if (!norm && written == 0 && !nonfinite) return QF8_OK;
    if (!ws || ws_bytes < (size_t)need) return QF8_ERR_WORKSPACE;
    if (!aligned(ws, 16) || !aligned(norm, 4) || !aligned(nonfinite, 4)) return QF8_ERR_ALIGN;
    return status_of(qf8::launch_clip(grads, count, chunk, max_norm, written > 0, norm, (float *)ws, (double *)((char *)ws + 16),
                                      nonfinite, as_stream(stream)));
}

}  // extern "C"
