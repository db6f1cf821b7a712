// qf8_norm.hip -- root-mean-square norm of a residual stream, its result in FP8 codes with 1x128 scales.
//
//   h = rnd(x + residual)              the stream's type; statistics are those of h as stored
//   R = 1 / sqrt(mean_c h^2 + eps)     fp32 sums in a fixed order
//   y = h R w                          fp32; S = F8max / max|y| over 128 neighbours, q = sat_rne8(fl32(y S))
//
// A row stays in registers from its load to its codes, so each input is read and each output written once:
// HBM is the bound (8192 rows of 7168 BF16 with residual 70 us, 5.9 TB/s; 16384 of 4096 75 us, 6.3; a copy of 2 GiB 4.95).
// Loads are non-temporal, stores are not (70 us; all cached 78, all non-temporal 73). A group of 128 is sixteen lanes with
// eight values each, so its maximum is four DPP steps; the row's sum takes one more exchange through LDS where several waves
// share a row.
#include <type_traits>

#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

// Sum over the T threads of a row and their C shares each, the same bits in each thread. red: C T / 64 floats that no thread
// still reads from an earlier call. T threads with C shares sum as C T threads do: a thread's share c is that of thread c T + t.
template <int T, int C>
__device__ __forceinline__ float sum_row(const float (&v)[C], float *red) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        s = sum_wave(v[c]);
        if (T > 64 && (threadIdx.x & 63) == 0) red[(c * T + (int)threadIdx.x) >> 6] = s;
    }
    if constexpr (T > 64) {
        __syncthreads();
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < C * T / 64; ++w) s += red[w];
    }
    return s;
}

// 1 / sqrt(v), v normal: the hardware's root, an ulp off, and a step r + r (1 - v r^2) / 2 with v r in two parts, which leaves
// half an ulp.
__device__ __forceinline__ float rsqrt_rounded(float v) {
    const float r = __builtin_amdgcn_rsqf(v), t = v * r, rest = __builtin_fmaf(v, r, -t);
    return __builtin_fmaf(0.5f * r, __builtin_fmaf(-rest, r, __builtin_fmaf(-t, r, 1.0f)), r);
}

// A row of squares whose fp32 sum, or mean with eps, overflows: the sum of (h 2^-72)^2, at most 2^14 (2^128 2^-72)^2 = 2^126, and
// the root in fp64. Inf and NaN among the values come through as R = 0 or NaN.
template <int T, int V, int C>
__device__ __forceinline__ float rstd_of_large(const float (&h)[V][8], float *red, int cols, float eps) {
    float ss[C] = {};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = h[v][i] * 0x1p-72f;
            ss[v % C] = __builtin_fmaf(s, s, ss[v % C]);
        }
    const double mean = (double)sum_row<T, C>(ss, red) * 0x1p144 / cols;
    return (float)(1.0 / sqrt(mean + (double)eps));
}

// The workgroup's threads that share a row, and the row, the same for the whole wave.
template <int T>
__device__ __forceinline__ int64_t first_row() {
    constexpr int R = T < 256 ? 256 / T : 1;
    return (int64_t)blockIdx.x * R + (T < 256 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0);
}

// Whether piece v of the whole wave lies behind the columns. Its loads are idle ones all the same (a branch around loads would
// make waits count on the fewest of them), the work on it is left out. us with that work / without it, no residual: 8192 rows of
// 5120 40.8 / 35.6, 16384 of 2056 42.3 / 38.6, 333 of 4104 5.0 / 4.7, whole pieces the same; gradients, 8192 of 4104 59.8 / 53.5.
template <int T>
__device__ __forceinline__ bool behind(int v, int cols) {
    return __builtin_amdgcn_readfirstlane((v * T + (int)(threadIdx.x % T)) * 8) >= cols;
}

// T threads to a row, V pieces of eight columns to a thread: cols <= 8 T V. TR: type of the residual (RES) and of h.
// C: shares of a thread's sum, so that a row's bits do not hang on the number of rows.
template <typename TX, typename TR, bool RES, int T, int V, int C>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_kernel(NormArgs p) {
    constexpr int R = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T < 256 ? 1 : C * T / 64];
    const int t = threadIdx.x % T, cols = (int)p.cols;
    for (int64_t row = first_row<T>(); row < p.rows; row += (int64_t)gridDim.x * R) {
        const auto xr = row_of<TX>(p.x, row, cols);
        Eight<TX> xe[V];
        Eight<TR> re[V];
#pragma unroll
        for (int v = 0; v < V; ++v) xe[v].template from<kNonTemporal>(xr, (v * T + t) * 8);
        if constexpr (RES) {
            const auto rr = row_of<TR>(p.residual, row, cols);
#pragma unroll
            for (int v = 0; v < V; ++v) re[v].template from<kNonTemporal>(rr, (v * T + t) * 8);
        }
        float h[V][8], share[C] = {};
        const auto hr = row_of<TR>(p.h, row, cols);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            xe[v].values(h[v]);
            if (v > 0 && behind<T>(v, cols)) continue;
            if constexpr (RES) {
                float r[8];
                re[v].values(r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] += r[i];
                re[v].round(h[v]);
                re[v].template to<kCached>(hr, (v * T + t) * 8);
                re[v].values(h[v]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) share[v % C] = __builtin_fmaf(h[v][i], h[v][i], share[v % C]);
        }
        const float ss = sum_row<T, C>(share, red[0]);
        // the mean as a product with 1 / cols in two parts, rounded once with eps. us, one part and the hardware's root
        // alone / this, no residual: 1 row of 7168 3.0 / 3.1, 16384 of 2056 37.9 / 38.4 (IEEE divisions and root 39.4)
        const float mean = __builtin_fmaf(ss, p.inv_cols, __builtin_fmaf(ss, p.inv_cols_rest, p.eps));
        float rstd = rsqrt_rounded(mean);
        if (!(mean < __builtin_inff())) rstd = rstd_of_large<T, V, C>(h, red[1], cols, p.eps);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        const auto yr = row_of<TX>(p.y, row, cols, p.y != nullptr);
        const auto qr = row_of<uint8_t>(p.q, row, cols, p.q != nullptr);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (v * T + t) * 8;
            if (v > 0 && behind<T>(v, cols)) break;
            float w[8], y[8];
            if (p.w_fp32) {
                Eight<float> e;
                e.from<kCached>(row_of<float>(p.weight, 0, cols), col);
                e.values(w);
            } else {
                Eight<uint16_t> e;
                e.from<kCached>(row_of<uint16_t>(p.weight, 0, cols), col);
                e.values(w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rstd * w[i];
            const uint32_t amax = group_amax(y, col < cols);       // behind the columns 0 times R, which may be NaN
            const bool first = (threadIdx.x & 15) == 0 && col < cols;
            if (p.nonfinite && first && amax >= (p.y ? kNotFinite<TX> : kNotFinite<float>)) *p.nonfinite = 1;
            if (p.y) {
                Eight<TX> e;
                e.round(y);
                e.template to<kCached>(yr, col);
            }
            if (p.q) {
                const float s = group_scale(amax, p.fmt, p.pow2);
                const uint2 c = group_codes(y, s, p.fmt);
                buf_store8<kCached>(qr, col, 0, c.x, c.y);
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
// in the order of the workgroups by a second kernel, so the same call gives the same bits. HBM is the bound: 8192 rows of
// 4096 BF16 with dres 48.9 us, 5.5 TB/s, 4.4 of them the joining.
// The next row's loads are under way while this one's sum is joined.
template <typename TX, typename TH, int T, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_backward_kernel(NormArgs p) {
    constexpr int R = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T < 256 ? 1 : T / 64];
    const int t = threadIdx.x % T, cols = (int)p.cols;
    const int64_t group = first_row<T>(), stride = (int64_t)gridDim.x * R;
    float dw[V][8], w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
        if (p.w_fp32) {
            Eight<float> e;
            e.from<kCached>(row_of<float>(p.weight, 0, cols), (v * T + t) * 8);
            e.values(w[v]);
        } else {
            Eight<uint16_t> e;
            e.from<kCached>(row_of<uint16_t>(p.weight, 0, cols), (v * T + t) * 8);
            e.values(w[v]);
        }
    }
    Eight<TX> de[V];
    Eight<TH> he[V], se[V];
    float rstd;
    const auto load = [&](int64_t row) {
        const bool there = row < p.rows;
        const auto dr = row_of<TX>(p.dy, row, cols, there);
        const auto hr = row_of<TH>(p.hin, row, cols, there);
        const auto sr = row_of<TH>(p.dres, row, cols, there && p.dres != nullptr);
        const auto rr = make_rsrc(p.rstd_in + row, there ? 4u : 0u);
        rstd = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rr, 0, 0, kCached));
#pragma unroll
        for (int v = 0; v < V; ++v) de[v].template from<kNonTemporal>(dr, (v * T + t) * 8);
#pragma unroll
        for (int v = 0; v < V; ++v) he[v].template from<kNonTemporal>(hr, (v * T + t) * 8);
#pragma unroll
        for (int v = 0; v < V; ++v) se[v].template from<kNonTemporal>(sr, (v * T + t) * 8);
    };
    load(group);
    int turn = 0;
    for (int64_t row = group; row < p.rows; row += stride, turn ^= 1) {
        float s[1] = {0.0f};
        Eight<TX> d0[V];
        Eight<TH> h0[V], s0[V];
        const float r = rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            d0[v] = de[v]; h0[v] = he[v]; s0[v] = se[v];
            if (behind<T>(v, cols)) continue;
            float d[8], n[8];
            d0[v].values(d);
            h0[v].values(n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] *= r;
                s[0] = __builtin_fmaf(d[i] * w[v][i], n[i], s[0]);
                dw[v][i] = __builtin_fmaf(d[i], n[i], dw[v][i]);
            }
        }
        load(row + stride);
        const float mean = sum_row<T, 1>(s, red[turn]) * p.inv_cols;
        const auto out = row_of<TH>(p.dx, row, cols);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (behind<T>(v, cols)) break;
            float d[8], n[8], o[8];
            d0[v].values(d);
            h0[v].values(n);
            s0[v].values(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += r * (d[i] * w[v][i] - n[i] * r * mean);
            Eight<TH> e;
            e.round(o);
            e.template to<kCached>(out, (v * T + t) * 8);
        }
    }
    if constexpr (R > 1) {                            // a wave has a share of its own: joined first, in the order of the waves
        __shared__ __align__(16) float share[R][V * T * 8];
        if (!p.partial) return;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; i += 4)
                *(float4 *)&share[threadIdx.x / T][(v * T + t) * 8 + i] = make_float4(dw[v][i], dw[v][i + 1], dw[v][i + 2], dw[v][i + 3]);
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += 256) {
            float sum = share[0][c];
#pragma unroll
            for (int i = 1; i < R; ++i) sum += share[i][c];
            p.partial[(int64_t)blockIdx.x * cols + c] = sum;
        }
    } else if (p.partial) {
        const auto to = row_of<float>(p.partial, group, cols);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Eight<float> e;
            e.round(dw[v]);
            e.to<kCached>(to, (v * T + t) * 8);
        }
    }
}

// dw[c] = sum of parts rows of partial, 16 columns to a workgroup: 64 runs of rows (a lane's group of four columns
// reads whole 64-byte pieces), joined in their order.
__global__ __launch_bounds__(256) void column_sum_kernel(const float *partial, int64_t parts, int cols, float *dw) {
    __shared__ float red[64][16];
    const int quad = threadIdx.x & 3, run = threadIdx.x >> 2, col = blockIdx.x * 16 + quad * 4;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < cols)
#pragma unroll 8
        for (int64_t i = run; i < parts; i += 64) {
            const float4 v = *(const float4 *)(partial + i * cols + col);
            s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[run][quad * 4 + i] = s[i];
    __syncthreads();
    if (threadIdx.x < 16 && blockIdx.x * 16 + (int)threadIdx.x < cols) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) t += red[i][threadIdx.x];
        dw[blockIdx.x * 16 + threadIdx.x] = t;
    }
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

constexpr int64_t kMaxNormGrid = (int64_t)1 << 21;       // threads of a launch are counted in 32 bits

template <typename TX, typename TR, bool RES>
int launch_norm_types(const NormArgs &p, hipStream_t s) {
    const auto go = [&](auto t, auto v, auto c) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, C = decltype(c)::value, R = T < 256 ? 256 / T : 1;
        const int64_t grid = (p.rows + R - 1) / R;
        hipLaunchKernelGGL((rms_norm_kernel<TX, TR, RES, T, V, C>), dim3((unsigned)(grid < kMaxNormGrid ? grid : kMaxNormGrid)),
                           dim3(T < 256 ? 256 : T), 0, s, p);
        return launched();
    };
    using std::integral_constant;
    // Threads and pieces of a row. us of the kernel, BF16: 7168 columns, 8192 rows 256 x 4 70, 512 x 2 73, 1024 x 1 100;
    // 64 rows 5.7, 4.5, 4.3; 1 row 4.6, 3.5, 3.3. 2048 columns, 16384 rows 256 x 1 41, 64 x 4 42; 64 rows 3.2, 5.2. 16384
    // columns, 2048 rows 512 x 4 47, 1024 x 2 51; 16 rows 5.8, 5.3
    const bool few = p.rows <= 512;
#define QF8_GO(T, V, C) return go(integral_constant<int, T>{}, integral_constant<int, V>{}, integral_constant<int, C>{})
    if (p.cols <= 512) QF8_GO(64, 1, 1);
    if (p.cols <= 1024) QF8_GO(64, 2, 1);
    if (p.cols <= 2048) QF8_GO(256, 1, 1);
    if (p.cols <= 4096) QF8_GO(256, 2, 1);
    if (p.cols <= 8192 && few) QF8_GO(512, 2, 1);
    if (p.cols <= 8192) QF8_GO(256, 4, 2);
    if (few) QF8_GO(1024, 2, 1);
    QF8_GO(512, 4, 2);
#undef QF8_GO
}

template <typename TX, typename TH>
int launch_norm_backward_types(const NormArgs &p, hipStream_t s) {
    const auto go = [&](auto t, auto v) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value;
        const int64_t grid = norm_backward_groups(p.rows, p.cols);
        hipLaunchKernelGGL((rms_norm_backward_kernel<TX, TH, T, V>), dim3((unsigned)grid), dim3(T < 256 ? 256 : T), 0, s, p);
        return launched();
    };
    using std::integral_constant;
    // Few values to a thread, so that the next row's loads find registers. us, 8192 rows of 4096: 512 x 1 44.8, 256 x 2 44.5;
    // 4096 of 16384 512 x 4 94, 1024 x 2 102, of 12296 with h in FP32 (some registers in scratch) 175, 206
#define QF8_GO(T, V) return go(integral_constant<int, T>{}, integral_constant<int, V>{})
    if (p.cols <= 512) QF8_GO(64, 1);
    if (p.cols <= 1024) QF8_GO(64, 2);
    if (p.cols <= 2048) QF8_GO(256, 1);
    if (p.cols <= 4096) QF8_GO(512, 1);
    if (p.cols <= 8192) QF8_GO(1024, 1);
    QF8_GO(512, 4);
#undef QF8_GO
}

}  // namespace

// us with the joining kernel, 8192 rows of 4096: 512 groups 48.9, 768 51.9, 2048 62; without it, 65536 of 512 (four rows at
// once) 512 groups 45.6, 1024 45.3, 2048 48.1, 128 124
int64_t norm_backward_groups(int64_t rows, int64_t cols) {
    const int64_t r = cols <= 1024 ? 4 : 1, most = 512;      // r: rows that a workgroup takes at once
    const int64_t groups = (rows + r - 1) / r;
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
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((p.cols + 15) / 16)), dim3(256), 0, s, p.partial,
                       p.rows > 0 ? norm_backward_groups(p.rows, p.cols) : 0, (int)p.cols, dw);
    return launched();
}

}  // namespace qf8
