// qf8_norm.hip -- root-mean-square norm of a residual stream, its result in FP8 codes with 1x128 scales.
//
//   h = rnd(x + residual)              the stream's type; statistics are those of h as stored
//   R = 1 / sqrt(mean_c h^2 + eps)     fp32 sums in a fixed order
//   y = h R w                          fp32; S = F8max / max|y| over 128 neighbours, q = sat_rne8(fl32(y S))
//
// A row stays in registers from its load to its codes, so each input is read and each output written once:
// HBM is the bound. A group of 128 is sixteen lanes with eight values each, so its maximum is four DPP steps;
// the row's sum takes one more exchange through LDS where several waves share a row.
#include <type_traits>

#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

// Sum over the T threads of a row, the same bits in each of them. red: T / 64 floats that no thread still reads
// from an earlier call.
template <int T>
__device__ __forceinline__ float sum_row(float v, float *red) {
    v = sum_wave(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v += red[w];
    }
    return v;
}

// A row of squares whose fp32 sum overflows: the sum of (h 2^-72)^2, at most 2^14 (2^128 2^-72)^2 = 2^126, and
// the root in fp64. Inf and NaN among the values come through as R = 0 or NaN.
template <int T, int V>
__device__ __forceinline__ float rstd_of_large(const float (&h)[V][8], float *red, int cols, float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = h[v][i] * 0x1p-72f;
            ss = __builtin_fmaf(s, s, ss);
        }
    const double mean = (double)sum_row<T>(ss, red) * 0x1p144 / cols;
    return (float)(1.0 / sqrt(mean + (double)eps));
}

template <typename TW>
__device__ __forceinline__ void weights8(const void *w, int col, float *v) {
    Eight<TW> e;
    e.load((const TW *)w + col);
    e.values(v);
}

// T threads to a row, V pieces of eight columns to a thread: cols <= 8 T V. TR: type of the residual (RES) and of h.
template <typename TX, typename TR, bool RES, int T, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_kernel(NormArgs p) {
    constexpr int R = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T < 256 ? 1 : T / 64];
    const int t = threadIdx.x % T, cols = (int)p.cols;
    for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / T; row < p.rows; row += (int64_t)gridDim.x * R) {
        const int64_t at = row * cols;
        Eight<TX> xe[V];
        Eight<TR> re[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            xe[v].zero();
            if constexpr (RES) re[v].zero();
            if (col < cols) {
                xe[v].stream((const TX *)p.x + at + col);
                if constexpr (RES) re[v].stream((const TR *)p.residual + at + col);
            }
        }
        float h[V][8], ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            xe[v].values(h[v]);
            if constexpr (RES) {
                float r[8];
                re[v].values(r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] += r[i];
                re[v].round(h[v]);
                if (col < cols) re[v].store((TR *)p.h + at + col);
                re[v].values(h[v]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(h[v][i], h[v][i], ss);
        }
        ss = sum_row<T>(ss, red[0]);
        float rstd = 1.0f / sqrtf(ss / (float)cols + p.eps);
        if (!(ss < __builtin_inff())) rstd = rstd_of_large<T, V>(h, red[1], cols, p.eps);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            float w[8], y[8];
            if (col < cols) {
                if (p.w_fp32) weights8<float>(p.weight, col, w);
                else weights8<uint16_t>(p.weight, col, w);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = col < cols ? h[v][i] * rstd * w[i] : 0.0f;
            const uint32_t amax = group_amax(y);
            const bool first = (threadIdx.x & 15) == 0 && col < cols;
            if (p.nonfinite && first && amax >= 0x7F800000u) *p.nonfinite = 1;
            if (p.y && col < cols) {
                Eight<TX> e;
                e.round(y);
                e.store((TX *)p.y + at + col);
            }
            if (p.q) {
                const float s = group_scale(amax, p.fmt, p.pow2);
                const uint2 c = group_codes(y, s, p.fmt);
                if (col < cols) *(uint2 *)(p.q + at + col) = c;
                if (first) p.scales[row * p.gcols + (col >> 7)] = s;
            }
        }
        if constexpr (T > 64) __syncthreads();          // red is written again
    }
}

// ---- gradients ------------------------------------------------------------------------------------
//
// With n = h R and g = dy w:  dh = R (g - n mean_c(g n)) + dres,  dw = sum over the rows of dy n.
// A workgroup takes every gridDim.x-th row and keeps its columns' share of dw in registers; the shares are joined
// in the order of the workgroups by a second kernel, so the same call gives the same bits.
template <typename TX, typename TH, int T, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_backward_kernel(NormArgs p) {
    constexpr int R = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T < 256 ? 1 : T / 64];
    const int t = threadIdx.x % T, cols = (int)p.cols;
    const int64_t group = (int64_t)blockIdx.x * R + threadIdx.x / T;
    float dw[V][8], w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = (v * T + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = w[v][i] = 0.0f;
        if (col < cols) {
            if (p.w_fp32) weights8<float>(p.weight, col, w[v]);
            else weights8<uint16_t>(p.weight, col, w[v]);
        }
    }
    int turn = 0;
    for (int64_t row = group; row < p.rows; row += (int64_t)gridDim.x * R, turn ^= 1) {
        const int64_t at = row * cols;
        Eight<TX> de[V];
        Eight<TH> he[V], se[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            de[v].zero(); he[v].zero(); se[v].zero();
            if (col < cols) {
                de[v].stream((const TX *)p.dy + at + col);
                he[v].stream((const TH *)p.hin + at + col);
                if (p.dres) se[v].stream((const TH *)p.dres + at + col);
            }
        }
        const float rstd = p.rstd_in[row];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float d[8], n[8];
            de[v].values(d);
            he[v].values(n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] *= rstd;
                s = __builtin_fmaf(d[i] * w[v][i], n[i], s);
                dw[v][i] = __builtin_fmaf(d[i], n[i], dw[v][i]);
            }
        }
        const float mean = sum_row<T>(s, red[turn]) / (float)cols;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            float d[8], n[8], o[8];
            de[v].values(d);
            he[v].values(n);
            se[v].values(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += rstd * (d[i] * w[v][i] - n[i] * rstd * mean);
            if (col < cols) {
                Eight<TH> e;
                e.round(o);
                e.store_stream((TH *)p.dx + at + col);
            }
        }
    }
    if (p.partial) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            Eight<float> e;
            e.round(dw[v]);
            if (col < cols) e.store(p.partial + group * cols + col);
        }
    }
}

// dw[c] = sum of parts rows of partial, 64 columns to a workgroup: four runs of rows, joined in their order.
__global__ __launch_bounds__(256) void column_sum_kernel(const float *partial, int64_t parts, int cols, float *dw) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    const int64_t per = (parts + 3) / 4, lo = wave * per, hi = lo + per < parts ? lo + per : parts;
    float s = 0.0f;
    if (col < cols)
        for (int64_t i = lo; i < hi; ++i) s += partial[i * cols + col];
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < cols) dw[col] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

constexpr int64_t kMaxNormGrid = (int64_t)1 << 21;       // threads of a launch are counted in 32 bits

template <typename TX, typename TR, bool RES>
int launch_norm_types(const NormArgs &p, hipStream_t s) {
    const auto go = [&](auto t, auto v) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, R = T < 256 ? 256 / T : 1;
        const int64_t grid = (p.rows + R - 1) / R;
        hipLaunchKernelGGL((rms_norm_kernel<TX, TR, RES, T, V>), dim3((unsigned)(grid < kMaxNormGrid ? grid : kMaxNormGrid)),
                           dim3(T < 256 ? 256 : T), 0, s, p);
        return launched();
    };
    using std::integral_constant;
#define QF8_GO(T, V) return go(integral_constant<int, T>{}, integral_constant<int, V>{})
    if (p.cols <= 512) QF8_GO(64, 1);
    if (p.cols <= 1024) QF8_GO(64, 2);
    if (p.cols <= 2048) QF8_GO(256, 1);
    if (p.cols <= 4096) QF8_GO(256, 2);
    if (p.cols <= 8192) QF8_GO(256, 4);
    QF8_GO(1024, 2);
#undef QF8_GO
}

template <typename TX, typename TH>
int launch_norm_backward_types(const NormArgs &p, hipStream_t s) {
    const auto go = [&](auto t, auto v) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, R = T < 256 ? 256 / T : 1;
        const int64_t grid = norm_backward_groups(p.rows, p.cols) / R;
        hipLaunchKernelGGL((rms_norm_backward_kernel<TX, TH, T, V>), dim3((unsigned)grid), dim3(T < 256 ? 256 : T), 0, s, p);
        return launched();
    };
    using std::integral_constant;
#define QF8_GO(T, V) return go(integral_constant<int, T>{}, integral_constant<int, V>{})
    if (p.cols <= 512) QF8_GO(64, 1);
    if (p.cols <= 1024) QF8_GO(64, 2);
    if (p.cols <= 2048) QF8_GO(256, 1);
    if (p.cols <= 4096) QF8_GO(256, 2);
    if (p.cols <= 8192) QF8_GO(256, 4);
    QF8_GO(1024, 2);
#undef QF8_GO
}

}  // namespace

int64_t norm_backward_groups(int64_t rows, int64_t cols) {
    const int64_t r = cols <= 1024 ? 4 : 1, most = 1024;      // rows that a workgroup takes at once
    const int64_t groups = (rows + r - 1) / r * r;
    return groups < most ? groups : most;
}

int launch_norm(const NormArgs &p, int dtype, int residual_dtype, hipStream_t s) {
    const bool bf = dtype == QF8_IN_BF16;
    if (!p.residual) return bf ? launch_norm_types<uint16_t, uint16_t, false>(p, s) : launch_norm_types<float, float, false>(p, s);
    if (residual_dtype == QF8_IN_BF16)
        return bf ? launch_norm_types<uint16_t, uint16_t, true>(p, s) : launch_norm_types<float, uint16_t, true>(p, s);
    return bf ? launch_norm_types<uint16_t, float, true>(p, s) : launch_norm_types<float, float, true>(p, s);
}

int launch_norm_backward(const NormArgs &p, int dtype, int h_dtype, float *dw, hipStream_t s) {
    const bool bf = dtype == QF8_IN_BF16;
    int r = QF8_OK;
    if (p.rows > 0) {
        if (h_dtype == QF8_IN_BF16)
            r = bf ? launch_norm_backward_types<uint16_t, uint16_t>(p, s) : launch_norm_backward_types<float, uint16_t>(p, s);
        else
            r = bf ? launch_norm_backward_types<uint16_t, float>(p, s) : launch_norm_backward_types<float, float>(p, s);
    }
    if (r != QF8_OK || !dw) return r;
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((p.cols + 63) / 64)), dim3(256), 0, s, p.partial,
                       p.rows > 0 ? norm_backward_groups(p.rows, p.cols) : 0, (int)p.cols, dw);
    return launched();
}

}  // namespace qf8
