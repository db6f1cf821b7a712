// qf8_experts.hip -- the expert layer around its products: the choice of experts for each token, the
// order of the rows by expert, the weighted sum of the experts' rows, and their gradients.
#include "qf8_device.h"
#include "qf8_internal.h"

namespace qf8 {
namespace {

// ---- wave-wide pieces ---------------------------------------------------------------------------
// Reductions by DPP moves, without the LDS round trips of a shuffle. Sums add in a fixed order.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_rows(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// Maximum over the wave, the same in every lane (a scalar): row_shr 1, 2, 4, 8, then the last lane of a
// row to the next row and of the lower half to the upper; lane 63 has seen all.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = umax(v, dpp_rows<0x111, 0xF>(v));
    v = umax(v, dpp_rows<0x112, 0xF>(v));
    v = umax(v, dpp_rows<0x114, 0xF>(v));
    v = umax(v, dpp_rows<0x118, 0xF>(v));
    v = umax(v, dpp_rows<0x142, 0xA>(v));                // row_bcast:15
    v = umax(v, dpp_rows<0x143, 0xC>(v));                // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL>
__device__ __forceinline__ double dpp_double(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = dpp_mov<CTRL>((uint32_t)b), hi = dpp_mov<CTRL>((uint32_t)(b >> 32));
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lane_double(double v, int lane) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// Sum over the first `lanes` lanes (the others hold 0): within rows of 16, then the rows.
__device__ __forceinline__ double wave_sum(double v, int lanes = 64) {
    v += dpp_double<0xB1>(v);
    v += dpp_double<0x4E>(v);
    v += dpp_double<0x141>(v);
    v += dpp_double<0x140>(v);
    double s = lane_double(v, 0);
    if (lanes > 16) s += lane_double(v, 16);
    if (lanes > 32) s += lane_double(v, 32) + lane_double(v, 48);
    return s;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
// LDS written by one lane of a wave and read by another: the wave's LDS accesses run in order.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// Order-preserving integers of floats; 0 is below every value.
__device__ __forceinline__ uint32_t float_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float wave_max(float v) {
    const uint32_t k = wave_max_u32(float_key(v));
    return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k);
}

// Logits as the choice sees them: NaN reads as -Inf, +Inf as the largest finite value of the logits' type
// (with which it ties, in the order and in the weights), and -0 as +0 so that it ties with it.
template <typename T> __device__ __forceinline__ float load_logit(const T *p, int64_t i);
template <> __device__ __forceinline__ float load_logit<uint16_t>(const uint16_t *p, int64_t i) {
    const float v = __uint_as_float((uint32_t)p[i] << 16);
    return v != v ? -INFINITY : fminf(v, __uint_as_float(0x7F7F0000u)) + 0.0f;
}
template <> __device__ __forceinline__ float load_logit<float>(const float *p, int64_t i) {
    const float v = p[i];
    return v != v ? -INFINITY : fminf(v, 3.40282346638528859812e+38f) + 0.0f;
}
__device__ __forceinline__ void store_logit(uint16_t *p, int64_t i, float v) {
    p[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ void store_logit(float *p, int64_t i, float v) { p[i] = v; }

__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// ---- the choice of experts ----------------------------------------------------------------------
//
// One wave per token; lane l holds experts l, l + 64, ... (NE of them). Selection compares either
// the logits themselves (scores rise with them, so without bias and groups the order is exact) or
// the scores plus bias in fp64: fp32 scores would tie or swap experts whose scores differ by less
// than 2^-24, and the chosen indices have to be those of the definition (a masked logit is compared by
// 0 + bias there, like any score). What is read is 2-4 bytes an expert; the time is that of the top_k
// rounds of a wave-wide maximum, so a round's key is as small as it can be: BF16 logits and the index in
// one 32-bit word (no two alike, so the maximum is the choice), FP32 logits in one with ties looked up
// afterwards, scores in two.
constexpr int kRouteWaves = 4;
enum { kByBf16 = 0, kByFp32 = 1, kByScore = 2 };

// The lowest expert e = 64 i + lane whose flag is set (flags: NE per lane); some flag is set.
template <int NE>
__device__ __forceinline__ int first_expert(const bool (&flag)[NE]) {
    int e = 0;
#pragma unroll
    for (int i = NE - 1; i >= 0; --i) {
        const uint64_t m = __ballot(flag[i]);
        e = m ? 64 * i + __ffsll((unsigned long long)m) - 1 : e;
    }
    return __builtin_amdgcn_readfirstlane(e);
}

template <typename T, int NE, int BY>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t route_lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 6) + wave;
    if (tok >= p.tokens) return;                       // whole waves; nothing below synchronizes the workgroup
    const T *row = (const T *)p.logits + tok * p.experts;

    float l[NE];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 64 * i + lane;
        l[i] = e < p.experts ? load_logit(row, e) : -INFINITY;
        top = fmaxf(top, l[i]);
    }
    const bool softmax = p.score == 0;
    double total = 0.0;                                // softmax: sum of exp(l - top)
    if (softmax) {
        top = wave_max(top);
        if (top == -INFINITY) top = 0.0f;              // nothing left by the mask: every score is 0
    }

    uint32_t key[NE], low[NE];                         // low: the other half of a score's key; 0, 0: not to choose
    if constexpr (BY == kByScore) {
        double s[NE];
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = softmax ? exp((double)l[i] - (double)top) : sigmoid64((double)l[i]);
            part += s[i];
        }
        if (softmax) {
            total = wave_sum(part);
#pragma unroll
            for (int i = 0; i < NE; ++i) s[i] = total > 0.0 ? s[i] / total : 0.0;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 64 * i + lane;
            if (e < p.experts && p.bias) s[i] += (double)p.bias[e];
            if (s[i] != s[i]) s[i] = -(double)INFINITY;
        }
        uint64_t open = ~0ull;
        const int size = p.experts / p.groups;
        if (p.groups > 1) {
            // the two best of every group: W lanes scan a group, then join by pairs
            double *sl = (double *)route_lds + (size_t)wave * p.experts;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (64 * i + lane < p.experts) sl[64 * i + lane] = s[i];
            wave_lds_fence();
            int slots = 1;
            while (slots < p.groups) slots <<= 1;
            const int W = 64 / slots, grp = lane / W, sub = lane % W;
            double m1 = -INFINITY, m2 = -INFINITY;
            if (grp < p.groups)
                for (int j = sub; j < size; j += W) {
                    const double v = sl[grp * size + j];
                    m2 = fmax(m2, fmin(m1, v));
                    m1 = fmax(m1, v);
                }
            for (int d = 1; d < W; d <<= 1) {
                const double o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
                m2 = fmax(fmax(m2, o2), fmin(m1, o1));
                m1 = fmax(m1, o1);
            }
            const double two = size > 1 ? m1 + m2 : m1;
            // a group is kept if fewer than top_groups come before it (ties: the lower index first)
            int before = 0;
            for (int o = 0; o < p.groups; ++o) {
                const double v = __shfl(two, o * W);
                before += v > two || (v == two && o < grp);
            }
            const uint64_t kept = __ballot(sub == 0 && grp < p.groups && before < p.top_groups);
            open = 0;
            for (int o = 0; o < p.groups; ++o) open |= ((kept >> (o * W)) & 1ull) << o;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 64 * i + lane;
            const uint64_t k = e < p.experts && ((open >> (e / size)) & 1ull) ? order_key(s[i] + 0.0) : 0ull;
            key[i] = (uint32_t)(k >> 32);
            low[i] = (uint32_t)k;
        }
    } else {
        if (softmax && !p.renorm) {
            double part = 0.0;
#pragma unroll
            for (int i = 0; i < NE; ++i) part += exp((double)l[i] - (double)top);
            total = wave_sum(part);
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 64 * i + lane;
            key[i] = e >= p.experts ? 0u : BY == kByBf16 ? (float_key(l[i]) & 0xFFFF0000u) | (uint32_t)(0xFFFF - e) : float_key(l[i]);
        }
    }

    int mine = 0;                                      // lane j keeps the j-th choice
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) best = umax(best, key[i]);
        best = wave_max_u32(best);
        int e;
        if constexpr (BY == kByBf16) {
            e = 0xFFFF - (int)(best & 0xFFFFu);
        } else {
            bool hit[NE];
#pragma unroll
            for (int i = 0; i < NE; ++i) hit[i] = key[i] == best;
            if constexpr (BY == kByScore) {
                int n = 0;
#pragma unroll
                for (int i = 0; i < NE; ++i) n += __popcll(__ballot(hit[i]));
                if (n > 1) {                           // the same upper half: by the lower one
                    uint32_t second = 0;
#pragma unroll
                    for (int i = 0; i < NE; ++i) second = hit[i] ? umax(second, low[i]) : second;
                    second = wave_max_u32(second);
#pragma unroll
                    for (int i = 0; i < NE; ++i) hit[i] = hit[i] && low[i] == second;
                }
            }
            e = first_expert(hit);
        }
        if (lane == j) mine = e;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (64 * i + lane == e) key[i] = low[i] = 0u;
    }

    // weights of the chosen, in fp64, rounded once
    const bool have = lane < p.top_k && mine < p.experts;
    const float x = have ? load_logit(row, mine) : -INFINITY;
    if (BY == kByScore && softmax && p.renorm) {
        // bias or groups may choose experts far below the largest logit, whose scores are 0 in fp64 but have
        // ratios all the same: relative to the largest chosen logit, as in the gradient
        top = wave_max(x);
        if (top == -INFINITY) top = 0.0f;
    }
    double w = 0.0;
    if (have) {
        if (softmax) {
            w = exp((double)x - (double)top);
            if (!p.renorm) w = total > 0.0 ? w / total : 0.0;
        } else {
            w = sigmoid64((double)x);
        }
    }
    if (p.renorm) {
        const double sum = wave_sum(w, p.top_k);
        w = sum > 0.0 ? w / sum : 0.0;                 // scores that are all 0: weights 0
    }
    if (lane < p.top_k) {
        p.ids[tok * p.top_k + lane] = mine;
        p.weights[tok * p.top_k + lane] = (float)(w * (double)p.scale);
    }
}

// Reductions over a row of 16 lanes; every lane of the row gets the result.
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
    v = umax(v, dpp_mov<0xB1>(v));
    v = umax(v, dpp_mov<0x4E>(v));
    v = umax(v, dpp_mov<0x141>(v));
    return umax(v, dpp_mov<0x140>(v));
}
__device__ __forceinline__ float row_max(float v) {
    const uint32_t k = row_max_u32(float_key(v));
    return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ double row_sum(double v) {
    v += dpp_double<0xB1>(v);
    v += dpp_double<0x4E>(v);
    v += dpp_double<0x141>(v);
    return v + dpp_double<0x140>(v);
}

// The same choice by logits with four tokens to a wave, one to each row of 16 lanes; lane l of a row holds
// experts l, l + 16, ... (NE of them). With many tokens the time is the number of instructions, and a
// round of the maximum costs about as many for four tokens as for one.
template <typename T, int NE, int BY>
__global__ __launch_bounds__(64 * kRouteWaves) void route_rows_kernel(RouteArgs p) {
    const int l16 = threadIdx.x & 15;
    const int64_t tok = (int64_t)blockIdx.x * (4 * kRouteWaves) + (threadIdx.x >> 4);
    if (tok >= p.tokens) return;                       // whole rows; nothing below leaves a row
    const T *row = (const T *)p.logits + tok * p.experts;

    float l[NE];
    uint32_t key[NE];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 16 * i + l16;
        l[i] = e < p.experts ? load_logit(row, e) : -INFINITY;
        top = fmaxf(top, l[i]);
        key[i] = e >= p.experts ? 0u : BY == kByBf16 ? (float_key(l[i]) & 0xFFFF0000u) | (uint32_t)(0xFFFF - e) : float_key(l[i]);
    }
    const bool softmax = p.score == 0;
    double total = 0.0;
    if (softmax) {
        top = row_max(top);
        if (top == -INFINITY) top = 0.0f;
        if (!p.renorm) {
            double part = 0.0;
#pragma unroll
            for (int i = 0; i < NE; ++i) part += exp((double)l[i] - (double)top);
            total = row_sum(part);
        }
    }

    int mine = 0;                                      // lane j of a row keeps the j-th choice
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) best = umax(best, key[i]);
        best = row_max_u32(best);
        int e;
        if constexpr (BY == kByBf16) {
            e = 0xFFFF - (int)(best & 0xFFFFu);
#pragma unroll
            for (int i = 0; i < NE; ++i) key[i] = key[i] == best ? 0u : key[i];       // no two keys are alike
        } else {
            uint32_t low = 0;                          // the lowest index among equal logits
#pragma unroll
            for (int i = 0; i < NE; ++i) low = umax(low, key[i] == best ? (uint32_t)(0xFFFF - 16 * i - l16) : 0u);
            e = 0xFFFF - (int)row_max_u32(low);
#pragma unroll
            for (int i = 0; i < NE; ++i) key[i] = 16 * i + l16 == e ? 0u : key[i];
        }
        mine = l16 == j ? e : mine;
    }

    double w = 0.0;
    if (l16 < p.top_k) {
        const double x = (double)load_logit(row, mine);
        if (softmax) {
            w = exp(x - (double)top);
            if (!p.renorm) w = total > 0.0 ? w / total : 0.0;
        } else {
            w = sigmoid64(x);
        }
    }
    if (p.renorm) {
        const double sum = row_sum(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (l16 < p.top_k) {
        p.ids[tok * p.top_k + l16] = mine;
        p.weights[tok * p.top_k + l16] = (float)(w * (double)p.scale);
    }
}

// Gradient of the logits. With w_j = scale p_j / T (T the sum of the chosen scores, or 1) and
// g_j = scale dw_j:  dL/dp_j = (g_j - sum_i g_i p_i / T) / T, or g_j without renormalisation. Sigmoid:
// dl_j = dL/dp_j p_j (1 - p_j). Softmax: dl_e = p_e (dL/dp_e - sum_j dL/dp_j p_j), where with
// renormalisation the sum is 0 and only ratios of the chosen scores remain.
template <typename T, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_backward_kernel(RouteArgs p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 6) + wave;
    if (tok >= p.tokens) return;
    const T *row = (const T *)p.logits + tok * p.experts;
    T *out = (T *)p.dlogits + tok * p.experts;
    const bool softmax = p.score == 0;
    const bool all = softmax && !p.renorm;             // every expert's score is needed
    const int id = lane < p.top_k ? p.ids[tok * p.top_k + lane] : -1;
    const bool have = id >= 0 && id < p.experts;
    const double x = have ? (double)load_logit(row, id) : 0.0;
    const double g = have ? (double)p.scale * (double)p.dweights[tok * p.top_k + lane] : 0.0;

    float l[NE];
    double total = 1.0, top = 0.0;
    if (all) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 64 * i + lane;
            l[i] = e < p.experts ? load_logit(row, e) : -INFINITY;
            m = fmaxf(m, l[i]);
        }
        m = wave_max(m);
        top = m == -INFINITY ? 0.0 : (double)m;
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i) part += exp((double)l[i] - top);
        total = wave_sum(part);
    } else if (softmax) {
        const float m = wave_max(have ? (float)x : -INFINITY);
        top = m == -INFINITY ? 0.0 : (double)m;
    }
    double s = 0.0;
    if (have) s = softmax ? exp(x - top) : sigmoid64(x);
    if (all) s = total > 0.0 ? s / total : 0.0;
    double d, rest = 0.0;                              // gradients of the chosen logits; rest: -p_e rest for the others
    if (p.renorm) {
        const double sum = wave_sum(s, p.top_k);
        const double w = sum > 0.0 ? s / sum : 0.0;
        const double mean = wave_sum(g * w, p.top_k);
        if (softmax) d = w * (g - mean);
        else d = w * (g - mean) / (1.0 + exp(x));       // p_j / T first: 1 / T alone may leave fp64
    } else if (softmax) {
        rest = wave_sum(g * s, p.top_k);
        d = s * (g - rest);
    } else {
        d = g * (s / (1.0 + exp(x)));
    }
    float v[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i)
        v[i] = all && total > 0.0 ? (float)(-(exp((double)l[i] - top) / total) * rest) : 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        const int e = __builtin_amdgcn_readlane(have ? id : -1, j);
        const float dj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint((float)d), j));
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (64 * i + lane == e) v[i] = dj;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 64 * i + lane;
        if (e < p.experts) store_logit(out, e, v[i]);
    }
}

// The same gradient with four tokens to a wave, one to each row of 16 lanes. A token's chosen entries
// meet the others in LDS: experts are where the lanes of a row are not.
template <typename T, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_backward_rows_kernel(RouteArgs p) {
    __shared__ float grad[4 * kRouteWaves][16 * NE];
    const int l16 = threadIdx.x & 15;
    float *const mine = grad[threadIdx.x >> 4];
    const int64_t tok = (int64_t)blockIdx.x * (4 * kRouteWaves) + (threadIdx.x >> 4);
    if (tok >= p.tokens) return;                       // whole rows; nothing below leaves a row
    const T *row = (const T *)p.logits + tok * p.experts;
    T *out = (T *)p.dlogits + tok * p.experts;
    const bool softmax = p.score == 0;
    const bool all = softmax && !p.renorm;
    const int id = l16 < p.top_k ? p.ids[tok * p.top_k + l16] : -1;
    const bool have = id >= 0 && id < p.experts;
    const double x = have ? (double)load_logit(row, id) : 0.0;
    const double g = have ? (double)p.scale * (double)p.dweights[tok * p.top_k + l16] : 0.0;

    float l[NE];
    double total = 1.0, top = 0.0;
    if (all) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 16 * i + l16;
            l[i] = e < p.experts ? load_logit(row, e) : -INFINITY;
            m = fmaxf(m, l[i]);
        }
        m = row_max(m);
        top = m == -INFINITY ? 0.0 : (double)m;
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i) part += exp((double)l[i] - top);
        total = row_sum(part);
    } else if (softmax) {
        const float m = row_max(have ? (float)x : -INFINITY);
        top = m == -INFINITY ? 0.0 : (double)m;
    }
    double s = 0.0;
    if (have) s = softmax ? exp(x - top) : sigmoid64(x);
    if (all) s = total > 0.0 ? s / total : 0.0;
    double d, rest = 0.0;
    if (p.renorm) {
        const double sum = row_sum(s);
        const double w = sum > 0.0 ? s / sum : 0.0;
        const double mean = row_sum(g * w);
        if (softmax) d = w * (g - mean);
        else d = w * (g - mean) / (1.0 + exp(x));       // p_j / T first: 1 / T alone may leave fp64
    } else if (softmax) {
        rest = row_sum(g * s);
        d = s * (g - rest);
    } else {
        d = g * (s / (1.0 + exp(x)));
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
        mine[16 * i + l16] = all && total > 0.0 ? (float)(-(exp((double)l[i] - top) / total) * rest) : 0.0f;
    wave_lds_fence();
    if (have) mine[id] = (float)d;
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 16 * i + l16;
        if (e < p.experts) store_logit(out, e, mine[e]);
    }
}

// ---- rows by expert -----------------------------------------------------------------------------
//
// A stable counting sort of tokens x top_k choices. Small inputs: one workgroup counts, scans and
// places. Larger ones: order_count_kernel leaves every workgroup's counts, then each workgroup of
// order_place_kernel sums the counts of those before it and places its own choices. The rank of a
// choice among equal ones of its wave is a population count of the lanes that ballots of the
// expert's bits leave; nothing depends on the order of atomics (they only count). Latency bound: 131072
// choices of 128 experts take 2.9 + 7.7 us (1.6 MB in and out), 512 of 256 in one workgroup 4.7 us. Padding
// written by one thread an expert, where 16 do it now, and a 64-bit division for each choice had cost 3.9 us more.
constexpr int kOrderThreads = 1024, kOrderWaves = kOrderThreads / 64;
// Choices up to which one workgroup does all. us, one workgroup / two kernels: 1024 of 64 experts 4.7 / 6.6, 2048 6.4 / 7.1,
// 4096 10.0 / 7.3; of 256 with rows padded to 128: 1024 7.7 / 9.7, 2048 9.7 / 9.1, 4096 13.7 / 8.8.
constexpr int kOrderOne = 2048;
constexpr int kOrderGroups = 256;                      // workgroups at most: each reads the counts of all
inline int64_t order_chunk(int64_t n) {                // choices of a workgroup
    const int64_t c = (n + kOrderGroups - 1) / kOrderGroups;
    return (c + kOrderThreads - 1) / kOrderThreads * kOrderThreads;
}

__global__ __launch_bounds__(kOrderThreads) void order_count_kernel(OrderArgs p) {
    __shared__ int count[kMaxExperts];
    for (int e = threadIdx.x; e < p.experts; e += kOrderThreads) count[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * p.chunk, hi = lo + p.chunk < p.n ? lo + p.chunk : p.n;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kOrderThreads) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.experts) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kOrderThreads) p.counts[(int64_t)blockIdx.x * p.experts + e] = count[e];
}

template <bool ONE>
__global__ __launch_bounds__(kOrderThreads) void order_place_kernel(OrderArgs p) {
    __shared__ int count[kMaxExperts];                 // choices of each expert
    __shared__ int next[kMaxExperts];                  // next free row of each expert, for this workgroup
    __shared__ int scan[kOrderWaves];
    __shared__ int pad[2][kMaxExperts];                // padding rows of each expert
    __shared__ int16_t rank[kOrderWaves * kMaxExperts];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t lo = ONE ? 0 : (int64_t)blockIdx.x * p.chunk;
    const int64_t hi = ONE ? p.n : lo + p.chunk < p.n ? lo + p.chunk : p.n;

    int first_id = -1;                                 // asked for early: used after the counts
    if (lo + t < hi) first_id = p.ids[lo + t];
    // counts of all choices, and of those before this workgroup's
    int before = 0, mine = 0;                          // thread e: expert e
    if (t < p.experts) count[t] = next[t] = 0;
    __syncthreads();
    if constexpr (ONE) {
        for (int64_t i = t; i < p.n; i += kOrderThreads) {
            const int e = p.ids[i];
            if (e >= 0 && e < p.experts) atomicAdd(&count[e], 1);
        }
    } else {
        // 1024 / experts threads share an expert, 8 loads of each in flight
        const int nb = gridDim.x, me = blockIdx.x, parts = kOrderThreads / p.experts;
        const int part = t / p.experts, e = t - part * p.experts;
        if (part < parts) {
            for (int b = part; b < nb; b += 8 * parts) {
                int v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = b + u * parts < nb ? p.counts[(int64_t)(b + u * parts) * p.experts + e] : 0;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    before += b + u * parts < me ? v[u] : 0;
                    mine += v[u];
                }
            }
            atomicAdd(&count[e], mine);
            atomicAdd(&next[e], before);
        }
    }
    __syncthreads();
    if (t < p.experts) {
        mine = count[t];
        before = next[t];
    }
    // first row of every expert: exclusive scan of the counts rounded up to align
    const int padded = t < p.experts ? (mine + p.align - 1) / p.align * p.align : 0;
    int inc = padded;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(inc, d);
        inc += lane >= d ? v : 0;
    }
    if (lane == 63) scan[wave] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wave; ++w) base += scan[w];
    const int first = base + inc - padded;
    if (t < p.experts) {
        next[t] = first + before;
        if (blockIdx.x == 0) {
            p.offsets[t] = first;
            if (t == p.experts - 1) p.offsets[p.experts] = first + padded;
        }
    }
    // rows that hold no choice: the padding of the experts, and what follows the last one
    int end = 0;
    for (int w = 0; w < kOrderWaves; ++w) end += scan[w];
    if (p.align > 1) {
        if (t < p.experts) {
            pad[0][t] = first + mine;
            pad[1][t] = first + padded;
        }
        __syncthreads();
        for (int e = blockIdx.x * (kOrderThreads / 16) + t / 16; e < p.experts; e += gridDim.x * (kOrderThreads / 16))
            for (int r = pad[0][e] + t % 16; r < pad[1][e] && r < p.nrows; r += 16) p.rows[r] = -1;
    }
    for (int64_t r = end + (int64_t)blockIdx.x * kOrderThreads + t; r < p.nrows; r += (int64_t)gridDim.x * kOrderThreads)
        p.rows[r] = -1;

    int bits = 0;
    while ((1 << bits) < p.experts) ++bits;
    for (int64_t c = lo; c < hi; c += kOrderThreads) {
        for (int i = t; i < kOrderWaves * p.experts; i += kOrderThreads) rank[i] = 0;
        __syncthreads();
        const int64_t i = c + t;
        const int e = c == lo ? first_id : i < hi ? p.ids[i] : -1;
        const bool ok = e >= 0 && e < p.experts;
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? m : ~m;
        }
        const int before_in_wave = __popcll(same & ((1ull << lane) - 1ull));
        if (ok && before_in_wave == 0) rank[wave * p.experts + e] = (int16_t)__popcll(same);
        __syncthreads();
        if (t < p.experts) {                           // counts of the waves -> counts before each wave
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kOrderWaves; ++w) {
                const int v = rank[w * p.experts + t];
                rank[w * p.experts + t] = (int16_t)sum;
                sum += v;
            }
            count[t] = sum;
        }
        __syncthreads();
        if (i < hi) {
            int slot = -1;
            if (ok) {
                slot = next[e] + rank[wave * p.experts + e] + before_in_wave;
                if (slot < p.nrows) p.rows[slot] = (int)((uint32_t)i / (uint32_t)p.top_k);   // fewer than 2^31 choices
                else slot = -1;
            }
            p.slots[i] = slot;
        }
        __syncthreads();
        if (t < p.experts) next[t] += count[t];
    }
}

// ---- the weighted sum ---------------------------------------------------------------------------
//
// y[t] = sum_j weights[t][j] x[slots[t][j]], in fp32, in the order of j, rounded once. Bound by the
// rows of x: every thread keeps the 16-byte pieces of all its top_k rows in flight. 8192 x 8 rows of 4096
// BF16: 125 us, 4.8 TB/s (a copy of 2 GiB 4.9); the gradients below 278 us, 4.4 TB/s.
template <typename T> struct Piece;                    // 16 bytes as fp32 values
template <> struct Piece<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint16_t *p, bool vec, int left, float *v) {
        if (vec) {
            const uint4 w = ld_stream((const uint4 *)p);
            v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
            v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < left ? __uint_as_float((uint32_t)p[i] << 16) : 0.0f;
        }
    }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        v2bf16 v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ void store(uint16_t *p, bool vec, int left, const float *v) {
        if (vec) {
            st_stream((uint4 *)p, make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7])));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) p[i] = (uint16_t)two(v[i], 0.0f);
        }
    }
};
template <> struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, bool vec, int left, float *v) {
        if (vec) {
            const uint4 w = ld_stream((const uint4 *)p);
            v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i < left ? p[i] : 0.0f;
        }
    }
    static __device__ __forceinline__ void store(float *p, bool vec, int left, const float *v) {
        if (vec) {
            st_stream((uint4 *)p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) p[i] = v[i];
        }
    }
};

constexpr int kCombineThreads = 256;
constexpr int kRowsAtOnce = 8;

template <typename T>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineArgs p) {
    constexpr int N = Piece<T>::N;
    const int64_t tok = blockIdx.x;
    const T *x = (const T *)p.x;
    T *y = (T *)p.y + tok * p.dim;
    for (int64_t c = ((int64_t)blockIdx.y * kCombineThreads + threadIdx.x) * N; c < p.dim;
         c += (int64_t)gridDim.y * kCombineThreads * N) {
        const int left = p.dim - c < N ? (int)(p.dim - c) : N;
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < p.top_k; j0 += kRowsAtOnce) {
            float v[kRowsAtOnce][N], w[kRowsAtOnce];
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j) {
                const bool on = j0 + j < p.top_k;
                const int64_t slot = on ? p.slots[tok * p.top_k + j0 + j] : -1;
                const bool ok = slot >= 0 && slot < p.nrows;
                w[j] = ok ? p.weights[tok * p.top_k + j0 + j] : 0.0f;
                if (ok) {
                    Piece<T>::load(x + slot * p.dim + c, p.vec, left, v[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[j][i] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(w[j], v[j][i], acc[i]);
        }
        Piece<T>::store(y + c, p.vec, left, acc);
    }
}

// dx[slots[t][j]] = weights[t][j] dy[t], dweights[t][j] = dy[t] . x[slots[t][j]]; rows without a token
// are zeros. One workgroup per token reads dy[t] once per 8 rows; the dot products are summed in fp32
// in a fixed order. The workgroups after the tokens' clear the rows that hold no token.
template <typename T>
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(CombineArgs p) {
    constexpr int N = Piece<T>::N, W = kCombineThreads / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T *dx = (T *)p.dx;
    if ((int64_t)blockIdx.x >= p.tokens) {
        const int64_t r0 = ((int64_t)blockIdx.x - p.tokens) * 64;
        const int64_t r = r0 + lane;
        const bool empty = r < p.nrows && (p.rows[r] < 0 || p.rows[r] >= p.tokens);
        uint64_t todo = __ballot(empty);
        const float zero[N] = {};
        while (todo) {
            const int at = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            for (int64_t c = (int64_t)threadIdx.x * N; c < p.dim; c += kCombineThreads * N)
                Piece<T>::store(dx + (r0 + at) * p.dim + c, p.vec, p.dim - c < N ? (int)(p.dim - c) : N, zero);
        }
        return;
    }
    __shared__ float red[W][kRowsAtOnce];
    const int64_t tok = blockIdx.x;
    const T *x = (const T *)p.x, *dy = (const T *)p.dy + tok * p.dim;
    for (int j0 = 0; j0 < p.top_k; j0 += kRowsAtOnce) {
        int64_t slot[kRowsAtOnce];
        float w[kRowsAtOnce], dot[kRowsAtOnce];
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j) {
            const bool on = j0 + j < p.top_k;
            const int64_t s = on ? p.slots[tok * p.top_k + j0 + j] : -1;
            slot[j] = s >= 0 && s < p.nrows ? s : -1;
            w[j] = slot[j] >= 0 ? p.weights[tok * p.top_k + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int64_t c = (int64_t)threadIdx.x * N; c < p.dim; c += kCombineThreads * N) {
            const int left = p.dim - c < N ? (int)(p.dim - c) : N;
            float d[N], v[kRowsAtOnce][N];
            Piece<T>::load(dy + c, p.vec, left, d);
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j)
                if (slot[j] >= 0) Piece<T>::load(x + slot[j] * p.dim + c, p.vec, left, v[j]);
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j) {
                if (slot[j] < 0) continue;
                float o[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot[j] = __builtin_fmaf(d[i], v[j][i], dot[j]);
                    o[i] = w[j] * d[i];
                }
                Piece<T>::store(dx + slot[j] * p.dim + c, p.vec, left, o);
            }
        }
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j) {
            const float s = wave_sum(dot[j]);
            if (lane == 0) red[wave][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < kRowsAtOnce && j0 + (int)threadIdx.x < p.top_k) {
            float s = 0.0f;
#pragma unroll
            for (int u = 0; u < W; ++u) s += red[u][threadIdx.x];
            p.dweights[tok * p.top_k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

// Whether four tokens share a wave. us a call, one token to a wave / four, top_k 8, BF16 logits:
//   forward   4096 x 128  4.4 / 4.4   8192 x 128  5.7 / 4.6   16384 x 128  8.9 / 5.6
//             4096 x 256  5.0 / 6.1   8192 x 256  6.7 / 6.4   16384 x 256  10.8 / 8.1 (FP32 7.5 / 8.1 at 8192)
//   backward  1024 x 128  3.4 / 3.3   2048 x 256  3.7 / 3.9    4096 x 128  4.3 / 3.5    16384 x 128  8.9 / 4.4
inline bool route_by_rows(const RouteArgs &p, bool backward) {
    if (p.top_k > 16 || p.experts > 256) return false;
    if (backward) return p.tokens > 2048;
    return !p.bias && p.groups == 1 && p.tokens > (p.experts <= 128 ? 4096 : 8192);
}

template <typename T, int NE>
int launch_route_ne(const RouteArgs &p, bool backward, hipStream_t s) {
    // few tokens: one wave per workgroup, so that they spread over the CUs. us, 1 wave / 4: 64 x 128 BF16 3.1 / 3.4,
    // 1024 3.4 / 3.5, 2048 3.8 / 3.5; 64 x 256 with bias and groups 7.3 / 7.7, 1024 7.7 / 7.7, 4096 11.2 / 10.9;
    // backward 64 x 128 3.1 / 3.3, 1024 3.3 / 3.4, 2048 3.7 / 3.4
    const int waves = p.tokens <= 1024 ? 1 : kRouteWaves;
    const dim3 grid((unsigned)((p.tokens + waves - 1) / waves)), block(64 * waves);
    if (backward) {
        hipLaunchKernelGGL((route_backward_kernel<T, NE>), grid, block, 0, s, p);
    } else if (p.bias || p.groups > 1) {
        const size_t lds = p.groups > 1 ? (size_t)waves * p.experts * sizeof(double) : 0;
        hipLaunchKernelGGL((route_kernel<T, NE, kByScore>), grid, block, lds, s, p);
    } else {
        hipLaunchKernelGGL((route_kernel<T, NE, sizeof(T) == 2 ? kByBf16 : kByFp32>), grid, block, 0, s, p);
    }
    return launched();
}
// NE: 16 experts each.
template <typename T, int NE>
int launch_route_rows(const RouteArgs &p, bool backward, hipStream_t s) {
    const int per = 4 * kRouteWaves;
    const dim3 grid((unsigned)((p.tokens + per - 1) / per)), block(64 * kRouteWaves);
    if (backward) hipLaunchKernelGGL((route_backward_rows_kernel<T, NE>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((route_rows_kernel<T, NE, sizeof(T) == 2 ? kByBf16 : kByFp32>), grid, block, 0, s, p);
    return launched();
}
template <typename T>
int launch_route_type(const RouteArgs &p, bool backward, hipStream_t s) {
    if (route_by_rows(p, backward)) {
        if (p.experts <= 64) return launch_route_rows<T, 4>(p, backward, s);
        if (p.experts <= 128) return launch_route_rows<T, 8>(p, backward, s);
        return launch_route_rows<T, 16>(p, backward, s);
    }
    if (p.experts <= 64) return launch_route_ne<T, 1>(p, backward, s);
    if (p.experts <= 128) return launch_route_ne<T, 2>(p, backward, s);
    if (p.experts <= 256) return launch_route_ne<T, 4>(p, backward, s);
    if (p.experts <= 512) return launch_route_ne<T, 8>(p, backward, s);
    return launch_route_ne<T, 16>(p, backward, s);
}

}  // namespace

int launch_route(const RouteArgs &p, int dtype, int backward, hipStream_t s) {
    if (p.tokens == 0) return QF8_OK;
    return dtype == QF8_IN_BF16 ? launch_route_type<uint16_t>(p, backward != 0, s)
                                : launch_route_type<float>(p, backward != 0, s);
}

size_t order_workspace(int64_t n, int experts) {
    if (n <= kOrderOne) return 0;
    const int64_t chunk = order_chunk(n);
    return (size_t)((n + chunk - 1) / chunk) * experts * sizeof(int32_t);
}

int launch_order(const OrderArgs &args, hipStream_t s) {
    OrderArgs p = args;
    p.chunk = order_chunk(p.n);
    if (p.n <= kOrderOne) {
        hipLaunchKernelGGL((order_place_kernel<true>), dim3(1), dim3(kOrderThreads), 0, s, p);
        return launched();
    }
    const dim3 grid((unsigned)((p.n + p.chunk - 1) / p.chunk));
    hipLaunchKernelGGL(order_count_kernel, grid, dim3(kOrderThreads), 0, s, p);
    if (launched() != QF8_OK) return QF8_ERR_HIP;
    hipLaunchKernelGGL((order_place_kernel<false>), grid, dim3(kOrderThreads), 0, s, p);
    return launched();
}

int launch_combine(const CombineArgs &args, int dtype, int backward, hipStream_t s) {
    CombineArgs p = args;
    const int N = dtype == QF8_IN_BF16 ? 8 : 4;
    p.vec = p.dim % N == 0;
    if (backward) {
        const int64_t groups = p.tokens + (p.nrows + 63) / 64;
        if (groups == 0) return QF8_OK;
        if (dtype == QF8_IN_BF16)
            hipLaunchKernelGGL((combine_backward_kernel<uint16_t>), dim3((unsigned)groups), dim3(kCombineThreads), 0, s, p);
        else
            hipLaunchKernelGGL((combine_backward_kernel<float>), dim3((unsigned)groups), dim3(kCombineThreads), 0, s, p);
        return launched();
    }
    if (p.tokens == 0) return QF8_OK;
    // A row's pieces spread over several workgroups, but for many tokens of few rows. us, several / one, BF16: 64 x 8
    // rows of 7168 6.3 / 15.6, 1024 x 8 31.5 / 34.2, 4096 x 8 113 / 127, 8192 x 8 of 4096 124 / 130, 16384 x 4 of 2880
    // 116 / 116; 16384 x 2 of 7168 169 / 161, 65536 x 2 of 2100 583 / 558, 32768 x 1 of 4096 137 / 126
    const int64_t per = (p.dim + (int64_t)kCombineThreads * N - 1) / ((int64_t)kCombineThreads * N);
    const unsigned gy = (unsigned)(p.tokens >= 2048 && p.top_k <= 2 ? 1 : per < 64 ? per : 64);
    const dim3 grid((unsigned)p.tokens, gy);
    if (dtype == QF8_IN_BF16) hipLaunchKernelGGL((combine_kernel<uint16_t>), grid, dim3(kCombineThreads), 0, s, p);
    else hipLaunchKernelGGL((combine_kernel<float>), grid, dim3(kCombineThreads), 0, s, p);
    return launched();
}

}  // namespace qf8
