// qf8_clip.hip -- the norm over all gradients of a step, and the gradients scaled down to a largest norm.
//
//   N = sqrt(sum g^2),  c = min(1, max_norm / (N + 1e-6)),  out = rnd(g c)
// Squares are summed in fp64: exact for BF16 and FP32 values but for the sums' own 2^-53, so N neither overflows
// nor depends on how the tensors are cut, and the partial sums are joined in a fixed order. The tensors travel in
// the kernels' arguments, kClipTensors to a launch, so a captured call needs no memory of the host later on.
#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipVectors = 8;                  // pieces of eight values in flight to a thread
constexpr int64_t kClipChunk = (int64_t)kClipThreads * kClipVectors * 8;

__device__ __forceinline__ double sum_wave_f64(double v) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
    return v;
}

// Sum over a workgroup of kClipThreads, the same bits in each thread.
__device__ __forceinline__ double sum_block_f64(double v, double *red) {
    v = sum_wave_f64(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// The tensor that chunk `block` of a launch belongs to: the last one whose first chunk is not behind it.
__device__ __forceinline__ int tensor_of(const ClipBatch &b, uint32_t block) {
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.first[mid] <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ double squares(const T *g, int64_t n, int64_t at) {
    Eight<T> e[kClipVectors];
    double s0 = 0.0, s1 = 0.0;
    const int64_t last = n - at;
    if (last >= kClipChunk && ((uintptr_t)g & 15) == 0) {
#pragma unroll
        for (int v = 0; v < kClipVectors; ++v) e[v].load(g + at + ((int64_t)v * kClipThreads + threadIdx.x) * 8);
#pragma unroll
        for (int v = 0; v < kClipVectors; ++v) {
            float x[8];
            e[v].values(x);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                s0 = __builtin_fma((double)x[i], (double)x[i], s0);
                s1 = __builtin_fma((double)x[i + 1], (double)x[i + 1], s1);
            }
        }
    } else {
        const int64_t end = last < kClipChunk ? last : kClipChunk;
        for (int64_t i = threadIdx.x; i < end; i += kClipThreads) {
            const double x = sizeof(T) == 2 ? (double)__uint_as_float((uint32_t)((const uint16_t *)g)[at + i] << 16)
                                            : (double)((const float *)g)[at + i];
            s0 = __builtin_fma(x, x, s0);
        }
    }
    return s0 + s1;
}

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(ClipBatch b, double *partial) {
    __shared__ double red[4];
    const int i = tensor_of(b, blockIdx.x);
    const int64_t at = (int64_t)(blockIdx.x - b.first[i]) * kClipChunk;
    const int64_t n = b.size[i] >> 1;
    double s = (b.size[i] & 1) ? squares((const float *)b.g[i], n, at) : squares((const uint16_t *)b.g[i], n, at);
    s = sum_block_f64(s, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// N and c from the partial sums.
__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(const double *partial, int64_t n, float max_norm, float *norm,
                                                                 float *factor, int32_t *nonfinite) {
    __shared__ double red[4];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kClipThreads) s += partial[i];
    s = sum_block_f64(s, red);
    if (threadIdx.x == 0) {
        const double total = sqrt(s);
        const bool finite = s < __builtin_inf();
        if (norm) *norm = (float)total;
        const double c = (double)max_norm / (total + 1e-6);
        *factor = finite && c < 1.0 ? (float)c : 1.0f;
        if (nonfinite && !finite) *nonfinite = 1;
    }
}

template <typename T>
__device__ __forceinline__ void scale(const T *g, T *out, int64_t n, int64_t at, float c) {
    const int64_t last = n - at;
    if (last >= kClipChunk && (((uintptr_t)g | (uintptr_t)out) & 15) == 0) {
        Eight<T> e[kClipVectors];
#pragma unroll
        for (int v = 0; v < kClipVectors; ++v) e[v].load(g + at + ((int64_t)v * kClipThreads + threadIdx.x) * 8);
#pragma unroll
        for (int v = 0; v < kClipVectors; ++v) {
            float x[8];
            e[v].values(x);
            if (c != 1.0f) {                             // a factor of 1 leaves every bit, NaN's too
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= c;
                e[v].round(x);
            }
            e[v].store(out + at + ((int64_t)v * kClipThreads + threadIdx.x) * 8);
        }
    } else {
        const int64_t end = last < kClipChunk ? last : kClipChunk;
        for (int64_t i = threadIdx.x; i < end; i += kClipThreads) {
            if (c == 1.0f) {
                out[at + i] = g[at + i];
            } else if constexpr (sizeof(T) == 2) {
                out[at + i] = (uint16_t)Eight<uint16_t>::two(__uint_as_float((uint32_t)g[at + i] << 16) * c, 0.0f);
            } else {
                out[at + i] = g[at + i] * c;
            }
        }
    }
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipBatch b, const float *factor) {
    const float c = *factor;
    const int i = tensor_of(b, blockIdx.x);
    if (c == 1.0f && b.out[i] == b.g[i]) return;
    const int64_t at = (int64_t)(blockIdx.x - b.first[i]) * kClipChunk;
    const int64_t n = b.size[i] >> 1;
    if (b.size[i] & 1) scale((const float *)b.g[i], (float *)b.out[i], n, at, c);
    else scale((const uint16_t *)b.g[i], (uint16_t *)b.out[i], n, at, c);
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

// Fills b from grads[at ...] and returns the entry behind the last one taken. chunks: those of the batch.
int next_batch(const qf8_grad *grads, int at, int count, ClipBatch &b, uint32_t &chunks) {
    b.count = 0;
    chunks = 0;
    for (; at < count && b.count < kClipTensors; ++at) {
        if (grads[at].n == 0) continue;
        const int64_t c = (grads[at].n + kClipChunk - 1) / kClipChunk;
        if (b.count > 0 && chunks + c > kMaxClipGrid) break;      // each tensor alone fits
        b.g[b.count] = grads[at].g;
        b.out[b.count] = grads[at].out;
        b.size[b.count] = grads[at].n * 2 + (grads[at].dtype == QF8_IN_FP32);
        b.first[b.count++] = chunks;
        chunks += (uint32_t)c;
    }
    return at;
}

}  // namespace

int64_t clip_chunks(int64_t n) { return (n + kClipChunk - 1) / kClipChunk; }

int launch_clip(const qf8_grad *grads, int count, float max_norm, int write, float *norm, float *factor, double *partial,
                int32_t *nonfinite, hipStream_t s) {
    ClipBatch b;
    uint32_t chunks;
    int64_t total = 0;
    for (int at = 0; at < count;) {
        at = next_batch(grads, at, count, b, chunks);
        if (chunks == 0) continue;
        hipLaunchKernelGGL(clip_squares_kernel, dim3(chunks), dim3(kClipThreads), 0, s, b, partial + total);
        if (launched() != QF8_OK) return QF8_ERR_HIP;
        total += chunks;
    }
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(kClipThreads), 0, s, partial, total, max_norm, norm, factor, nonfinite);
    if (launched() != QF8_OK) return QF8_ERR_HIP;
    for (int at = 0; write && at < count;) {
        at = next_batch(grads, at, count, b, chunks);
        if (chunks == 0) continue;
        hipLaunchKernelGGL(clip_scale_kernel, dim3(chunks), dim3(kClipThreads), 0, s, b, factor);
        if (launched() != QF8_OK) return QF8_ERR_HIP;
    }
    return QF8_OK;
}

}  // namespace qf8
