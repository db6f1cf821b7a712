// qf8_layer.hip -- a whole expert layer with gated activation for a few tokens, in two kernels.
//
//   a[t][e] = rnd_bf16(act(A_e x[t]) * (B_e x[t])),  W1[e] = [A_e; B_e]      the first kernel
//   y[t]    = rnd_bf16(sum_e wt[t][e] W2[e] a[t][e])                          the second
//
// Each chosen expert's weights are read once, which is the bound: a weight's byte takes part in as many products as
// its expert has tokens, about eight, where the matrix cores would need hundreds. Codes are exact in BF16, so they
// are converted beside the loads and multiplied with BF16 activations (16x16x32 products: sixteen rows of a weight
// times up to sixteen tokens); a 128x128 block's sums meet 1/S in fp32. The activations are not quantized.
//
// Every workgroup of the first kernel sorts the choices by expert on its own (in LDS, at most 1024 of them); the first
// one leaves the list, cut into jobs of up to 16 NT tokens of an expert, in the workspace for the second kernel.
#include <type_traits>

#include "qf8_act.h"
#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef float v4f32 __attribute__((ext_vector_type(4)));

// ---- jobs ---------------------------------------------------------------------------------------
// A job in 32 bits: expert (10), first entry (11), entries - 1 (6). An entry: choice t * top_k + j (16) and token.
constexpr int kMaxJobs = kLayerChoices;              // a job has an entry at least
__device__ __forceinline__ uint32_t pack_job(int e, int start, int n) { return (uint32_t)(e | start << 10 | (n - 1) << 21); }
__device__ __forceinline__ int job_expert(uint32_t j) { return (int)(j & 1023); }
__device__ __forceinline__ int job_start(uint32_t j) { return (int)(j >> 10 & 2047); }
__device__ __forceinline__ int job_count(uint32_t j) { return (int)(j >> 21) + 1; }

struct Jobs {
    uint32_t job[kMaxJobs];          // one for each chosen expert, with all its entries
    uint32_t entry[kLayerChoices];
    int start[kMaxExperts];          // counts, then the next free entry of each expert
    int16_t id[kLayerChoices];
    int total, entries;
};

// All threads of the workgroup; ends with a barrier. The order of an expert's entries is this workgroup's own: what
// leaves it (activations) is placed by choice. A token that names an expert twice has one entry, at its first choice.
// cut: the jobs of up to per_job entries go to p.jobs, their number to p.job_count.
template <int THREADS>
__device__ void find_jobs(const LayerArgs &p, bool cut, int per_job, Jobs &s) {
    const int n = p.tokens * p.top_k;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int e = p.ids[i];
        s.id[i] = (int16_t)((uint32_t)e < (uint32_t)p.experts ? e : -1);
    }
    for (int i = threadIdx.x; i < p.experts; i += THREADS) s.start[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int e = s.id[i], t0 = i / p.top_k * p.top_k;
        bool first = e >= 0;
        for (int j = t0; j < i; ++j) first = first && s.id[j] != e;
        if (first) atomicAdd(&s.start[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < 64) {                           // counts -> first entries, and the jobs in the order of the experts
        int entries = 0, jobs = 0, pieces = 0;
        for (int base = 0; base < p.experts; base += 64) {
            const int e = base + (int)threadIdx.x;
            const int c = e < p.experts ? s.start[e] : 0, q = (c + per_job - 1) / per_job;
            int before = c, qbefore = q;              // inclusive sums over the lanes
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int a = __shfl_up(before, off), b = __shfl_up(qbefore, off);
                if ((int)threadIdx.x >= off) { before += a; qbefore += b; }
            }
            const uint64_t chosen = __ballot(c > 0);
            const int at = entries + before - c;
            if (e < p.experts) s.start[e] = at;
            if (c > 0) s.job[jobs + __popcll(chosen & ((1ull << threadIdx.x) - 1))] = pack_job(e, at, c);
            for (int k = 0; cut && k < q; ++k)
                p.jobs[pieces + qbefore - q + k] = pack_job(e, at + k * per_job, c - k * per_job < per_job ? c - k * per_job : per_job);
            entries += __shfl(before, 63);
            pieces += __shfl(qbefore, 63);
            jobs += __popcll(chosen);
        }
        if (threadIdx.x == 0) {
            s.total = jobs;
            s.entries = entries;
            if (cut) *p.job_count = pieces;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int e = s.id[i], t = i / p.top_k, t0 = t * p.top_k;
        bool first = e >= 0;
        for (int j = t0; j < i; ++j) first = first && s.id[j] != e;
        if (first) s.entry[atomicAdd(&s.start[e], 1)] = (uint32_t)(i | t << 16);
    }
    __syncthreads();
}

// ---- products -----------------------------------------------------------------------------------

// Sixteen codes of a row (k ascending) -> two operands of eight BF16 values, exactly.
template <int FMT>
__device__ __forceinline__ v8bf16 operand(uint32_t lo, uint32_t hi) {
    v2bf16 p[4];
    if constexpr (FMT == kE4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
    }
    return v8bf16{p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
}

// 128 values of k for RT tiles of sixteen rows of a weight and NT of sixteen tokens. Lane (r, g) = (lane % 16,
// lane / 16) holds k = 64 h + 16 g .. + 15 of row (token) r, h = 0, 1: two 16-byte loads of codes, four of BF16. The
// products' own order of k is another one, the same for both operands.
template <int RT, int NT>
struct Step {
    uint4 w[RT][2];
    uint4 x[NT][4];
};

template <int FMT, int RT, int NT>
__device__ __forceinline__ void multiply(const Step<RT, NT> &s, const float (&inv)[RT], bool second, v4f32 (&acc)[RT][NT]) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        v8bf16 w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[2 * h] = operand<FMT>(s.w[r][h].x, s.w[r][h].y);
            w[2 * h + 1] = operand<FMT>(s.w[r][h].z, s.w[r][h].w);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n > 0 && !second) continue;           // the same for the whole wave
            v4f32 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[k], __builtin_bit_cast(v8bf16, s.x[n][k]), sum, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][n][i] = __builtin_fmaf(sum[i], inv[r], acc[r][n][i]);
        }
    }
}

constexpr int kUpThreads = 256, kUpWaves = kUpThreads / 64;

// A workgroup takes sixteen hidden units of a job, 16 rows of A_e and 16 of B_e; its waves share k, wave w the blocks
// of 128 with index w mod 4, and their sums are joined in LDS in the order of the waves.
template <int FMT, int ACT, int NT>
__global__ __launch_bounds__(kUpThreads, 4) void layer_up_kernel(LayerArgs p) {
    __shared__ Jobs jobs;
    __shared__ float part[kUpWaves][2][NT][256];
    find_jobs<kUpThreads>(p, blockIdx.x == 0, 16 * NT, jobs);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < jobs.entries; i += kUpThreads) {
            const int c = (int)(jobs.entry[i] & 0xFFFF), t0 = (int)(jobs.entry[i] >> 16) * p.top_k;
            float w = p.weights[c];
            for (int j = c + 1; j < t0 + p.top_k; ++j)
                if (jobs.id[j] == jobs.id[c]) w += p.weights[j];
            p.entries[i] = jobs.entry[i];
            p.entry_weights[i] = w;
        }
    }
    const int dim = p.dim, blocks = p.hidden / 16, gk = (dim + 127) / 128;
    const int gn = (2 * p.hidden + 127) / 128;
    const uint32_t items = (uint32_t)jobs.total * (uint32_t)blocks;
    const auto xr = make_rsrc(p.x, (uint32_t)p.tokens * (uint32_t)dim * 2u);
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t job = jobs.job[item / (uint32_t)blocks];
        const int j0 = (int)(item % (uint32_t)blocks) * 16;
        const int e = job_expert(job);
        const auto wr = make_rsrc(p.w1 + (int64_t)e * 2 * p.hidden * dim, 2u * (uint32_t)p.hidden * (uint32_t)dim);
        uint32_t wrow[2];
        wrow[0] = (uint32_t)(j0 + r) * (uint32_t)dim + 16 * g;
        wrow[1] = wrow[0] + (uint32_t)p.hidden * (uint32_t)dim;
        // 1 / S of this wave's i-th block in lane i
        float inv[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int b = wave + lane * kUpWaves;
            inv[q] = b < gk ? 1.0f / p.s1[((int64_t)e * gn + (q * p.hidden + j0) / 128) * gk + b] : 0.0f;
        }
        for (int c0 = 0; c0 < job_count(job); c0 += 16 * NT) {
            const int start = job_start(job) + c0, count = job_count(job) - c0;
            uint32_t xrow[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int i = n * 16 + r;
                xrow[n] = i < count ? (jobs.entry[start + i] >> 16) * (uint32_t)dim * 2u + 32 * g : kOutOfRange;
            }
            v4f32 acc[2][NT];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[q][n] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
            Step<2, NT> step[2];
            const auto load = [&](Step<2, NT> &s, int i) {
                const int k0 = (wave + i * kUpWaves) * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = k0 + 64 * h + 16 * g < dim;
#pragma unroll
                    for (int q = 0; q < 2; ++q) s.w[q][h] = buf_load16<kNonTemporal>(wr, in ? wrow[q] + k0 + 64 * h : kOutOfRange, 0);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t at = in && xrow[n] != kOutOfRange ? xrow[n] + 2 * (k0 + 64 * h) : kOutOfRange;
                        s.x[n][2 * h] = buf_load16(xr, at, 0);
                        s.x[n][2 * h + 1] = buf_load16(xr, at == kOutOfRange ? at : at + 16, 0);
                    }
                }
            };
            const auto use = [&](const Step<2, NT> &s, int i) {
                const float f[2] = {__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv[0]), i)),
                                    __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv[1]), i))};
                multiply<FMT, 2, NT>(s, f, count > 16, acc);
            };
            const int steps = (gk - wave + kUpWaves - 1) / kUpWaves;      // at most 64
            load(step[0], 0);
            for (int i = 0; i < steps; i += 2) {
                load(step[1], i + 1);
                use(step[0], i);
                load(step[0], i + 2);
                if (i + 1 < steps) use(step[1], i + 1);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int n = 0; n < NT; ++n) *(v4f32 *)&part[wave][q][n][r * 16 + 4 * g] = acc[q][n];
            __syncthreads();
            // one hidden unit of one token to a thread
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int i = n * 16 + (int)(threadIdx.x >> 4);
                if (i < count) {
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kUpWaves; ++w) {
                        sum[0] += part[w][0][n][threadIdx.x];
                        sum[1] += part[w][1][n][threadIdx.x];
                    }
                    const float a = act<ACT, false>(sum[0]) * sum[1];
                    const int c = (int)(jobs.entry[start + i] & 0xFFFF);
                    p.a[(int64_t)c * p.hidden + j0 + (threadIdx.x & 15)] = (uint16_t)Eight<uint16_t>::two(a, 0.0f);
                }
            }
            __syncthreads();
        }
    }
}

constexpr int kDownWaves = 8, kDownThreads = 64 * kDownWaves;

// A workgroup owns sixteen columns of y. The blocks of 128 hidden units of all jobs form one run of steps, cut into
// eight equal parts; each wave goes through its part and adds every job's products, weighted, to its own sums of all
// tokens in LDS, and the eight are joined in the order of the waves: nothing is exchanged between workgroups.
template <int FMT, int NT>
__global__ __launch_bounds__(kDownThreads, 4) void layer_down_kernel(LayerArgs p) {
    extern __shared__ float sums[];                   // [waves][tokens][16], then the list
    const int n = p.tokens * p.top_k, total = *p.job_count;
    uint32_t *entry = (uint32_t *)(sums + kDownWaves * p.tokens * 16);
    float *weight = (float *)(entry + n);
    uint32_t *job_list = (uint32_t *)(weight + n);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    float *mine = sums + wave * p.tokens * 16;
    for (int i = lane; i < p.tokens * 16; i += 64) mine[i] = 0.0f;
    for (int i = threadIdx.x; i < n; i += kDownThreads) {       // what is behind the list's end is not used
        entry[i] = p.entries[i];
        weight[i] = p.entry_weights[i];
        job_list[i] = p.jobs[i];
    }
    __syncthreads();
    const int hidden = p.hidden, gk = (hidden + 127) / 128, gn = (p.dim + 127) / 128, d0 = (int)blockIdx.x * 16;
    const int64_t units = (int64_t)total * gk;
    const int lo = (int)(units * wave / kDownWaves), hi = (int)(units * (wave + 1) / kDownWaves);
    const auto ar = make_rsrc(p.a, (uint32_t)n * (uint32_t)hidden * 2u);
    const uint32_t wrow = (uint32_t)(d0 + r) * (uint32_t)hidden + 16 * g;
    v4f32 acc[1][NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[0][i] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};

    // the loads run ahead of the products, so each side keeps its own place in the run
    int ljob = gk > 0 ? lo / gk : 0, lblock = lo - ljob * gk, ujob = ljob, ublock = lblock;
    uint32_t arow[NT];
    __amdgpu_buffer_rsrc_t wr;
    const float *scale;
    const auto place = [&](int j) {
        const uint32_t job = (uint32_t)__builtin_amdgcn_readfirstlane((int)job_list[j < total ? j : 0]);
        const int e = job_expert(job);
        wr = make_rsrc(p.w2 + (int64_t)e * p.dim * hidden, (uint32_t)p.dim * (uint32_t)hidden);
        scale = p.s2 + ((int64_t)e * gn + d0 / 128) * gk;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int at = i * 16 + r;
            arow[i] = at < job_count(job) ? (entry[job_start(job) + at] & 0xFFFF) * (uint32_t)hidden * 2u + 32 * g : kOutOfRange;
        }
    };
    Step<1, NT> step[2];
    float inv[2];
    const auto load = [&](Step<1, NT> &s, float &f, int unit) {
        const int k0 = lblock * 128;
        const bool on = unit < hi;
        f = scale[lblock];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = on && k0 + 64 * h + 16 * g < hidden;
            s.w[0][h] = buf_load16<kNonTemporal>(wr, in ? wrow + k0 + 64 * h : kOutOfRange, 0);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint32_t at = in && arow[i] != kOutOfRange ? arow[i] + 2 * (k0 + 64 * h) : kOutOfRange;
                s.x[i][2 * h] = buf_load16(ar, at, 0);
                s.x[i][2 * h + 1] = buf_load16(ar, at == kOutOfRange ? at : at + 16, 0);
            }
        }
        if (++lblock == gk) {
            lblock = 0;
            place(++ljob);
        }
    };
    const auto use = [&](const Step<1, NT> &s, float f, int unit) {
        const uint32_t job = (uint32_t)__builtin_amdgcn_readfirstlane((int)job_list[ujob]);
        const float one[1] = {1.0f / f};
        multiply<FMT, 1, NT>(s, one, job_count(job) > 16, acc);
        if (++ublock == gk || unit + 1 == hi) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int at = i * 16 + r;
                if (at < job_count(job)) {
                    const int k = job_start(job) + at;
                    v4f32 *to = (v4f32 *)(mine + (entry[k] >> 16) * 16 + 4 * g);
                    v4f32 v = *to;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(weight[k], acc[0][i][q], v[q]);
                    *to = v;
                }
                acc[0][i] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
            }
            ublock = 0;
            ++ujob;
        }
    };
    if (lo < hi) {
        place(ljob);
        load(step[0], inv[0], lo);
        for (int u = lo; u < hi; u += 2) {
            load(step[1], inv[1], u + 1);
            use(step[0], inv[0], u);
            load(step[0], inv[0], u + 2);
            if (u + 1 < hi) use(step[1], inv[1], u + 1);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.tokens * 16; i += kDownThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) s += sums[w * p.tokens * 16 + i];
        p.y[(int64_t)(i >> 4) * p.dim + d0 + (i & 15)] = (uint16_t)Eight<uint16_t>::two(s, 0.0f);
    }
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

template <int FMT, int ACT, int NT>
int launch_layer_kernels(const LayerArgs &p, hipStream_t s) {
    const int n = p.tokens * p.top_k;
    const int64_t jobs = n < p.experts ? n : p.experts, most = 256 * 4;      // four workgroups to a CU
    const int64_t items = p.hidden > 0 ? jobs * (p.hidden / 16) : 1;
    hipLaunchKernelGGL((layer_up_kernel<FMT, ACT, NT>), dim3((unsigned)(items < most ? items : most)), dim3(kUpThreads), 0, s, p);
    if (launched() != QF8_OK) return QF8_ERR_HIP;
    const size_t lds = (size_t)kDownWaves * p.tokens * 64 + (size_t)n * 12;
    hipLaunchKernelGGL((layer_down_kernel<FMT, NT>), dim3((unsigned)(p.dim / 16)), dim3(kDownThreads), lds, s, p);
    return launched();
}
template <int FMT, int ACT>
int launch_layer_tokens(const LayerArgs &p, hipStream_t s) {
    return p.tokens <= 16 ? launch_layer_kernels<FMT, ACT, 1>(p, s) : launch_layer_kernels<FMT, ACT, 2>(p, s);
}

}  // namespace

size_t layer_workspace(int64_t tokens, int top_k, int64_t hidden) {
    const size_t n = (size_t)tokens * top_k;
    return up16(n * hidden * 2) + up16(kMaxJobs * 4) + 2 * up16(n * 4) + 16;
}

int launch_layer(const LayerArgs &args, int fmt, int act, void *ws, hipStream_t s) {
    LayerArgs p = args;
    const size_t n = (size_t)p.tokens * p.top_k;
    char *at = (char *)ws;
    p.a = (uint16_t *)at;
    at += up16(n * p.hidden * 2);
    p.jobs = (uint32_t *)at;
    at += up16(kMaxJobs * 4);
    p.entries = (uint32_t *)at;
    at += up16(n * 4);
    p.entry_weights = (float *)at;
    at += up16(n * 4);
    p.job_count = (int *)at;
    if (fmt == QF8_E4M3)
        return act == QF8_ACT_SILU ? launch_layer_tokens<kE4M3, QF8_ACT_SILU>(p, s) : launch_layer_tokens<kE4M3, QF8_ACT_GELU>(p, s);
    return act == QF8_ACT_SILU ? launch_layer_tokens<kE5M2, QF8_ACT_SILU>(p, s) : launch_layer_tokens<kE5M2, QF8_ACT_GELU>(p, s);
}

}  // namespace qf8
