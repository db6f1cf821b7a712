// qf8_clip.hip -- the norm over all gradients of a step, and the gradients scaled down to a largest norm.
//
//   N = sqrt(sum g^2),  c = min(1, max_norm / (N + 1e-6)),  out = rnd(g c)
// Squares are summed in fp64: exact for BF16 and FP32 values but for the sums' own 2^-53, so N neither overflows
// nor depends on how the tensors are cut, and the partial sums are joined in a fixed order. The tensors travel in
// the kernels' arguments, kClipTensors to a launch, so a captured call needs no memory of the host later on.
// HBM is the bound: 2.1 GB of FP32 in 353 us (6.1 TB/s) and, read again and written, 784 us (5.5 TB/s; a copy of 2 GiB 4.95).
// The squares' loads are cached, so that some of the tensors are still near for the scaling: both without that 316 + 827 us. The
// scaling's are non-temporal (cached loads 812 us). From the last tensor to the first it ran slower: 240 MB 71.6 us for 69.3.
#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipPieces = 8;                   // 16-byte pieces in flight to a thread
constexpr int64_t kClipTrip = (int64_t)kClipThreads * kClipPieces * 8;

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

// len values as a run of whole 16-byte pieces with a few values before and behind it that single threads take.
template <typename T>
struct Run {
    static constexpr int N = 16 / sizeof(T);     // values of a piece
    int64_t head, pieces, tail;
    __device__ __forceinline__ Run(const T *p, int64_t len) {
        head = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / (int64_t)sizeof(T);
        if (head > len) head = len;
        pieces = (len - head) / N;
        tail = len - head - pieces * N;
    }
    // The thread's one value of the two ends, or -1.
    __device__ __forceinline__ int64_t single() const {
        const int64_t t = threadIdx.x;
        return t < head ? t : t < head + tail ? pieces * N + t : -1;
    }
    // Pieces [first, first + a trip) as a buffer: those behind the end read as zeros and are not written, without a branch
    // around them.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t trip(const T *p, int64_t first) const {
        const int64_t left = pieces - first, most = kClipThreads * kClipPieces;
        return make_rsrc(p + head + first * N, (uint32_t)((left < most ? left : most) * 16));
    }
};

template <typename T> __device__ __forceinline__ float value_of(T v);
template <> __device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <> __device__ __forceinline__ float value_of(float v) { return v; }

template <typename T>
__device__ __forceinline__ void values_of(uint4 a, float *v) {
    if constexpr (sizeof(T) == 2) {
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
    } else {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    }
}
template <typename T>
__device__ __forceinline__ uint4 piece_of(const float *v) {
    if constexpr (sizeof(T) == 2) {
        typedef Eight<uint16_t> E;
        return make_uint4(E::two(v[0], v[1]), E::two(v[2], v[3]), E::two(v[4], v[5]), E::two(v[6], v[7]));
    } else {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
}

template <typename T>
__device__ __forceinline__ double squares(const T *g, int64_t len) {
    constexpr int N = Run<T>::N;
    const Run<T> run(g, len);
    double s0 = 0.0, s1 = 0.0;
    for (int64_t first = 0; first < run.pieces; first += kClipThreads * kClipPieces) {
        const auto r = run.trip(g, first);
        uint4 e[kClipPieces];
#pragma unroll
        for (int v = 0; v < kClipPieces; ++v) e[v] = buf_load16<kCached>(r, (v * kClipThreads + threadIdx.x) * 16, 0);
#pragma unroll
        for (int v = 0; v < kClipPieces; ++v) {
            float x[N];
            values_of<T>(e[v], x);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                s0 = __builtin_fma((double)x[i], (double)x[i], s0);
                s1 = __builtin_fma((double)x[i + 1], (double)x[i + 1], s1);
            }
        }
    }
    const int64_t one = run.single();
    if (one >= 0) {
        const double x = (double)value_of(g[one]);
        s0 = __builtin_fma(x, x, s0);
    }
    return s0 + s1;
}

// The values of workgroup `block`: len of tensor i from `at` on.
struct Share {
    int i;
    int64_t at, len;
    bool fp32;
    __device__ __forceinline__ Share(const ClipBatch &b, uint32_t block) {
        i = tensor_of(b, block);
        at = (int64_t)(block - b.first[i]) * b.chunk;
        const int64_t n = b.size[i] >> 1;
        len = n - at < b.chunk ? n - at : b.chunk;
        fp32 = b.size[i] & 1;
    }
};

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(ClipBatch b, double *partial) {
    __shared__ double red[4];
    const Share share(b, blockIdx.x);
    const double s = sum_block_f64(share.fp32 ? squares((const float *)b.g[share.i] + share.at, share.len)
                                              : squares((const uint16_t *)b.g[share.i] + share.at, share.len), red);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// N and c from the partial sums.
__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(const double *partial, int64_t n, double max_norm, float *norm,
                                                                 float *factor, int32_t *nonfinite) {
    __shared__ double red[4];
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += kClipThreads) s += partial[i];
    s = sum_block_f64(s, red);
    if (threadIdx.x == 0) {
        const double total = sqrt(s);                 // beyond fp32 perhaps, beyond fp64 only where a value is
        const bool finite = s < __builtin_inf();
        if (norm) *norm = (float)total;
        const double c = max_norm / (total + 1e-6);
        *factor = finite && c < 1.0 ? (float)c : 1.0f;
        if (nonfinite && !finite) *nonfinite = 1;
    }
}

// A factor of 1 leaves every bit, NaN's too.
template <typename T>
__device__ __forceinline__ T scaled(T v, float c) {
    if (c == 1.0f) return v;
    if constexpr (sizeof(T) == 2) return (T)Eight<uint16_t>::two(value_of(v) * c, 0.0f);
    else return v * c;
}
template <typename T>
__device__ __forceinline__ void scale(const T *g, T *out, int64_t len, float c) {
    if ((((uintptr_t)g ^ (uintptr_t)out) & 15) != 0) {        // no pieces at 16 bytes in both
        for (int64_t i = threadIdx.x; i < len; i += kClipThreads) out[i] = scaled(g[i], c);
        return;
    }
    constexpr int N = Run<T>::N;
    const Run<T> run(g, len);
    for (int64_t first = 0; first < run.pieces; first += kClipThreads * kClipPieces) {
        const auto r = run.trip(g, first), to = run.trip(out, first);
        uint4 e[kClipPieces];
#pragma unroll
        for (int v = 0; v < kClipPieces; ++v) e[v] = buf_load16<kNonTemporal>(r, (v * kClipThreads + threadIdx.x) * 16, 0);
#pragma unroll
        for (int v = 0; v < kClipPieces; ++v) {
            float x[N];
            values_of<T>(e[v], x);
            if (c != 1.0f) {
#pragma unroll
                for (int i = 0; i < N; ++i) x[i] *= c;
                e[v] = piece_of<T>(x);
            }
            buf_store16<kNonTemporal>(to, (v * kClipThreads + threadIdx.x) * 16, 0, e[v]);
        }
    }
    const int64_t one = run.single();
    if (one >= 0) out[one] = scaled(g[one], c);
}

__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipBatch b, const float *factor) {
    const float c = *factor;
    const Share share(b, blockIdx.x);
    const int i = share.i;
    if (c == 1.0f && b.out[i] == b.g[i]) return;
    if (share.fp32) scale((const float *)b.g[i] + share.at, (float *)b.out[i] + share.at, share.len, c);
    else scale((const uint16_t *)b.g[i] + share.at, (uint16_t *)b.out[i] + share.at, share.len, c);
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

// Fills b from grads[at ...] and returns the entry behind the last one taken. chunks: those of the batch.
int next_batch(const qf8_grad *grads, int at, int count, ClipBatch &b, uint32_t &chunks) {
    b.count = 0;
    chunks = 0;
    for (; at < count && b.count < kClipTensors; ++at) {
        if (grads[at].n == 0) continue;
        b.g[b.count] = grads[at].g;
        b.out[b.count] = grads[at].out;
        b.size[b.count] = grads[at].n * 2 + (grads[at].dtype == QF8_IN_FP32);
        b.first[b.count++] = chunks;
        chunks += (uint32_t)((grads[at].n + b.chunk - 1) / b.chunk);
    }
    return at;
}

}  // namespace

int64_t clip_chunk(int64_t total) {
    const int64_t chunk = (total / 4096 + kClipTrip - 1) / kClipTrip * kClipTrip;
    return chunk > kClipTrip ? chunk : kClipTrip;
}

int launch_clip(const qf8_grad *grads, int count, int64_t chunk, double max_norm, int write, float *norm, float *factor, double *partial,
                int32_t *nonfinite, hipStream_t s) {
    ClipBatch b;
    b.chunk = chunk;
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
