// qf8_layer.hip -- a whole expert layer with gated activation for a few tokens, in two kernels.
//
//   a[t][e] = act(A_e x[t]) * (B_e x[t]),  W1[e] = [A_e; B_e]                the first kernel
//   y[t]    = rnd_bf16(sum_e wt[t][e] W2[e] a[t][e])                          the second
//
// Each chosen expert's weights are read once, which is the bound: a weight's byte takes part in as many products as
// its expert has tokens, about eight, where the matrix cores would need hundreds. Codes are exact in BF16 and in FP16, so they
// are converted beside the loads and multiplied with 16-bit activations (16x16x32 products: sixteen rows of a weight
// times up to sixteen tokens); a 128x128 block's sums meet 1/S in fp32. The activations are not quantized: x is BF16, and those
// between the products are FP16 times a power of two for sixteen neighbours, 2^-11 off, an eighth of what rounding y is (BF16 has
// them off by as much as y, for 4% less time with 64 tokens of 7168, 8 of 64 experts; two BF16 pieces take 8% more).
// us of the two kernels: 64 tokens of 7168, 8 of 64 experts, hidden 2048 312 + 174 (6.1 and 5.4 TB/s; a loop of loads alone
// reaches 7.1), 1 token of 4096 29 + 16, of which a launch and the list of jobs take 5 each.
//
// Every workgroup of the first kernel sorts the choices by expert on its own (in LDS, at most 1024 of them); the first
// one leaves the list, cut into pieces of up to 32 tokens of an expert, those of experts with more than sixteen first, in the
// workspace for the second kernel.
#include <type_traits>

#include "qf8_act.h"
#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef _Float16 v2f16 __attribute__((ext_vector_type(2)));
typedef _Float16 v8f16 __attribute__((ext_vector_type(8)));
typedef float v4f32 __attribute__((ext_vector_type(4)));

// ---- jobs ---------------------------------------------------------------------------------------
// A job in 32 bits: expert (10), first entry (10), entries - 1 (6). A piece of one, up to 32 entries, has its number
// in the job and the number of the job's pieces - 1 too (2 each). An entry: choice t * top_k + j (16) and token.
constexpr int kMaxJobs = kLayerChoices;              // a job, and a piece, has an entry at least
__device__ __forceinline__ uint32_t pack_job(int e, int start, int n) { return (uint32_t)(e | start << 10 | (n - 1) << 20); }
__device__ __forceinline__ int job_expert(uint32_t j) { return (int)(j & 1023); }
__device__ __forceinline__ int job_start(uint32_t j) { return (int)(j >> 10 & 1023); }
__device__ __forceinline__ int job_count(uint32_t j) { return (int)(j >> 20 & 63) + 1; }
__device__ __forceinline__ int piece_number(uint32_t j) { return (int)(j >> 26 & 3); }
__device__ __forceinline__ int piece_total(uint32_t j) { return (int)(j >> 28 & 3) + 1; }

struct Jobs {
    uint32_t job[kMaxJobs];          // one for each chosen expert, with all its entries
    uint32_t entry[kLayerChoices];
    int start[kMaxExperts];          // counts, then the next free entry of each expert
    int16_t id[kLayerChoices];
    int total, entries;
};

// All threads of the workgroup; ends with a barrier. The order of an expert's entries is this workgroup's and this run's
// own: activations are placed by choice, and each is a result of its own. A token that names an expert twice has one entry, at its first choice.
// cut: the pieces go to p.jobs, their number and that of the first kind to p.job_count.
template <int THREADS>
__device__ void find_jobs(const LayerArgs &p, bool cut, Jobs &s) {
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
        int entries = 0, jobs = 0, large = 0, small = 0;       // pieces of experts with more than sixteen entries, and of the others
        for (int base = 0; cut && base < p.experts; base += 64) {
            const int c = base + (int)threadIdx.x < p.experts ? s.start[base + threadIdx.x] : 0;
            small += __popcll(__ballot(c > 16)) + __popcll(__ballot(c > 32));       // where the others begin
        }
        if (cut && threadIdx.x == 0) p.job_count[1] = small;
        for (int base = 0; base < p.experts; base += 64) {
            const int e = base + (int)threadIdx.x;
            const int c = e < p.experts ? s.start[e] : 0;
            int before = c;                           // inclusive sum over the lanes
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int a = __shfl_up(before, off);
                if ((int)threadIdx.x >= off) before += a;
            }
            const uint64_t chosen = __ballot(c > 0), first = __ballot(c > 16), second = __ballot(c > 32);
            const uint64_t below = (1ull << threadIdx.x) - 1;
            const int at = entries + before - c;
            if (e < p.experts) s.start[e] = at;
            if (c > 0) s.job[jobs + __popcll(chosen & below)] = pack_job(e, at, c);
            if (cut && c > 16) {
                const int to = large + __popcll(first & below) + __popcll(second & below);
                const uint32_t pieces = c > 32 ? 1u << 28 : 0u;
                p.jobs[to] = pack_job(e, at, c > 32 ? 32 : c) | pieces;
                if (c > 32) p.jobs[to + 1] = pack_job(e, at + 32, c - 32) | pieces | 1u << 26;
            } else if (cut && c > 0) {
                p.jobs[small + __popcll(chosen & ~first & below)] = pack_job(e, at, c);
            }
            large += __popcll(first) + __popcll(second);
            small += __popcll(chosen & ~first);
            entries += __shfl(before, 63);
            jobs += __popcll(chosen);
        }
        if (threadIdx.x == 0) {
            s.total = jobs;
            s.entries = entries;
            if (cut) p.job_count[0] = small;
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

// Eight codes of a row (k ascending) -> an operand of eight values, exactly, and products of operands. Bf16: of x. Fp16: of the
// activations between the products.
struct Bf16 {
    typedef v8bf16 Operand;
    template <int FMT> static __device__ __forceinline__ Operand of(uint32_t lo, uint32_t hi) {
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
        return Operand{p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
    }
    static __device__ __forceinline__ v4f32 product(Operand a, Operand b, v4f32 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
struct Fp16 {
    typedef v8f16 Operand;
    template <int FMT> static __device__ __forceinline__ Operand of(uint32_t lo, uint32_t hi) {
        v2f16 p[4];
        if constexpr (FMT == kE4M3) {
            p[0] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
            p[1] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
            p[2] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
            p[3] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
        } else {
            p[0] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(lo, 1.0f, false));
            p[1] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(lo, 1.0f, true));
            p[2] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(hi, 1.0f, false));
            p[3] = __builtin_bit_cast(v2f16, __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(hi, 1.0f, true));
        }
        return Operand{p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
    }
    static __device__ __forceinline__ v4f32 product(Operand a, Operand b, v4f32 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

// An activation between the products is v 2^(E - kScaleBias), v FP16 and E a byte for sixteen neighbours: the exponent field of
// their largest magnitude, which v holds in [2^14, 2^15), or kLeastScale (2^-126) if that is more.
constexpr uint32_t kScaleBias = 127 + 14, kLeastScale = 15;
__device__ __forceinline__ float scale_value(uint32_t e) { return __uint_as_float((umax(e, kLeastScale) + 127 - kScaleBias) << 23); }

// 128 values of k for RT tiles of sixteen rows of a weight and up to sixteen tokens. Both are loaded in whole lines, a
// weight eight rows to an instruction (lane l: chunk l % 8 of row l / 8), the tokens four (chunk l % 16 of token l / 16, as
// many instructions as there are tokens for), and turned in LDS, 4 KB of a wave's own, into the products' layout: lane
// (r, g) = (lane % 16, lane / 16) holds k = 64 h + 16 g .. + 15 of row (token) r, h = 0, 1. The products' own order of k
// is another one, the same for both. Weights loaded straight into that layout, half a line of a row each, came at 5.7 TB/s
// (6.3 cached) against 7.1 in a loop of loads alone (64 weights of 4096x7168); tokens loaded so took four
// instructions where eight tokens need two, and the vector memory units were the bound of the second kernel.
// Chunk c of row r, rows of 128 and of 256 bytes: sixteen lanes that read one chunk of sixteen rows, or that write whole
// rows, meet no bank twice.
__device__ __forceinline__ int chunk128(int r, int c) { return r * 128 + ((c ^ (r >> 1)) & 7) * 16; }
__device__ __forceinline__ int chunk256(int r, int c) { return r * 256 + ((c ^ r) & 15) * 16; }

// The lane, computed where it is used: addresses that hang on it stay out of the registers of the loops around (the first
// kernel, whose three workgroups to a CU leave 168 to a thread; the second has registers for them).
__device__ __forceinline__ int lane_here() {
    int lane = (int)(threadIdx.x & 63);
    asm volatile("" : "+v"(lane));
    return lane;
}

// Loaded rows into the products' layout, over the same LDS one after the other (a wave's LDS operations keep their
// order); the registers they come from can be loaded again then.
template <int RT>
__device__ __forceinline__ void turn_weights(const uint4 (&w)[RT][2], char *tile, uint4 (&o)[RT][2], int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int q = 0; q < 2; ++q) *(uint4 *)(tile + t * 2048 + chunk128(8 * q + (lane >> 3), lane & 7)) = w[t][q];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) o[t][h] = *(const uint4 *)(tile + t * 2048 + chunk128(r, g + 4 * h));
}
__device__ __forceinline__ void place_tokens(const uint4 (&x)[4], int instructions, char *tile, int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (q < instructions) *(uint4 *)(tile + chunk256(4 * q + g, r)) = x[q];
}

// The scales of 128 activations of a token, a byte for each sixteen: the values move to the largest of them (what falls below
// FP16 there is below 2^-39 of the largest value). by[h]: the factor of the lane's k in half h; returns the token's scale.
__device__ __forceinline__ float find_scales(uint2 e, int g, _Float16 (&by)[2]) {
    const v2u16 a = __builtin_bit_cast(v2u16, e.x & 0x00FF00FFu), b = __builtin_bit_cast(v2u16, (e.x >> 8) & 0x00FF00FFu);
    const v2u16 c = __builtin_bit_cast(v2u16, e.y & 0x00FF00FFu), d = __builtin_bit_cast(v2u16, (e.y >> 8) & 0x00FF00FFu);
    const v2u16 m = __builtin_elementwise_max(__builtin_elementwise_max(a, b), __builtin_elementwise_max(c, d));
    const uint32_t most = umax(m.x, m.y);
    by[0] = __builtin_ldexpf16((_Float16)1.0f, (int)(e.x >> 8 * g & 255) - (int)most);
    by[1] = __builtin_ldexpf16((_Float16)1.0f, (int)(e.y >> 8 * g & 255) - (int)most);
    return scale_value(most);
}

// Products of turned weights with placed tokens, one half of the 128 values of k after the other (the fence keeps the
// second half's operands out of the registers meanwhile). Tokens behind the last one are what LDS held: their columns are
// not used. f: the factor of each tile's sums, for this lane's token; by: factors of the token's values (Fp16).
template <typename T, int FMT, int RT>
__device__ __forceinline__ void multiply(const uint4 (&w)[RT][2], const char *tile, const float (&f)[RT], v4f32 (&acc)[RT], int lane, const _Float16 (&by)[2] = {}) {
    const int r = lane & 15, g = lane >> 4;
    v4f32 sum[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) sum[t] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        typename T::Operand x0 = *(const typename T::Operand *)(tile + chunk256(r, 8 * h + 2 * g));
        typename T::Operand x1 = *(const typename T::Operand *)(tile + chunk256(r, 8 * h + 2 * g + 1));
        if constexpr (std::is_same<T, Fp16>::value) {
            x0 *= by[h];
            x1 *= by[h];
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            sum[t] = T::product(T::template of<FMT>(w[t][h].x, w[t][h].y), x0, sum[t]);
            sum[t] = T::product(T::template of<FMT>(w[t][h].z, w[t][h].w), x1, sum[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(sum[t][i], f[t], acc[t][i]);
}

// Weights are read past the caches where rows are whole lines; where they are not, neighbouring rows share lines, and cached
// loads take them once: 13 tokens x 6 of 40 experts, 2064, hidden 720 46.3 -> 44.1 us, 64 x 4 of 16, 4112, hidden 2000 156 -> 144.
constexpr int kUpThreads = 256, kUpWaves = kUpThreads / 64, kUpGroups = 3;      // workgroups to a CU

// A workgroup takes sixteen hidden units of a job, 16 rows of A_e and 16 of B_e; its waves share k, wave w the blocks
// of 128 with index w mod 4, and their sums are joined in LDS in the order of the waves. More than 32 tokens take another
// pass over the rows.
template <int FMT, int ACT, int CP>
__global__ __launch_bounds__(kUpThreads, kUpGroups) void layer_up_kernel(LayerArgs p) {
    __shared__ Jobs jobs;
    __shared__ __align__(16) char tile[kUpWaves][4096];          // at the end the sums of each wave, [2][2][256]
    float(*part)[1024] = (float(*)[1024])tile;
    find_jobs<kUpThreads>(p, blockIdx.x == 0, jobs);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (blockIdx.x == 0) {
        if (p.parts > 1)
            for (int i = threadIdx.x; i < p.columns; i += kUpThreads) p.arrivals[i] = 0;
        // the entries of an expert in the order of the choices, so that the second kernel's sums have one order too
        for (int i = threadIdx.x; i < jobs.entries; i += kUpThreads) {
            const int c = (int)(jobs.entry[i] & 0xFFFF), t0 = (int)(jobs.entry[i] >> 16) * p.top_k, e = jobs.id[c];
            int k = jobs.start[e], before = 0;        // the end of the expert's entries
            for (; k > 0 && jobs.id[jobs.entry[k - 1] & 0xFFFF] == e; --k) before += (int)(jobs.entry[k - 1] & 0xFFFF) < c;
            float w = p.weights[c];
            for (int j = c + 1; j < t0 + p.top_k; ++j)
                if (jobs.id[j] == e) w += p.weights[j];
            p.entries[k + before] = jobs.entry[i];
            p.entry_weights[k + before] = w;
        }
    }
    const int dim = p.dim, blocks = p.hidden / 16, gk = (dim + 127) / 128;
    const int gn = (2 * p.hidden + 127) / 128;
    const int steps = (gk - wave + kUpWaves - 1) / kUpWaves;      // at most 64, an even number or one more taken
    const uint32_t items = (uint32_t)jobs.total * (uint32_t)blocks;
    const auto xr = make_rsrc(p.x, (uint32_t)p.tokens * (uint32_t)dim * 2u);
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t job = jobs.job[item / (uint32_t)blocks];
        const int j0 = (int)(item % (uint32_t)blocks) * 16;
        const int e = __builtin_amdgcn_readfirstlane(job_expert(job));
        const auto wr = make_rsrc(p.w1 + (int64_t)e * 2 * p.hidden * dim, 2u * (uint32_t)p.hidden * (uint32_t)dim);
        uint32_t wrow[2];
        wrow[0] = (uint32_t)(j0 + (lane >> 3)) * (uint32_t)dim + 16 * (lane & 7);
        wrow[1] = wrow[0] + (uint32_t)p.hidden * (uint32_t)dim;
        // 1 / S of this wave's i-th block in lane i
        float inv[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int b = wave + lane * kUpWaves;
            inv[q] = b < gk ? 1.0f / p.s1[((int64_t)e * gn + (q * p.hidden + j0) / 128) * gk + b] : 0.0f;
        }
        const int all = __builtin_amdgcn_readfirstlane(job_count(job));
        for (int c0 = 0; c0 < all; c0 += 32) {
            const int start = job_start(job) + c0, count = all - c0 < 32 ? all - c0 : 32;
            // NX: instructions that load sixteen tokens, NC: sixteens of tokens
            const auto run = [&](auto nx, auto nc) {
                constexpr int NX = decltype(nx)::value, NC = decltype(nc)::value;
                uint32_t xrow[NC][NX];
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int q = 0; q < NX; ++q) {
                        const int at = 16 * c + 4 * q + g;
                        xrow[c][q] = at < count ? (jobs.entry[start + at] >> 16) * (uint32_t)dim * 2u + 16 * r : kOutOfRange;
                    }
                v4f32 acc[NC][2];
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[c][0] = acc[c][1] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
                uint4 w[2][2][2], x[2][4];
                const auto load_w = [&](uint4 (&to)[2][2], int i) {
                    const int k0 = (wave + i * kUpWaves) * 128;
                    const bool in = k0 + 16 * (lane & 7) < dim;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            to[q][h] = buf_load16<CP>(wr, in ? wrow[q] : kOutOfRange, (uint32_t)(k0 + 8 * h * dim));
                };
                const auto load_x = [&](uint4 (&to)[4], int i, int c) {
                    const int k0 = (wave + i * kUpWaves) * 128;
                    const bool in = k0 + 8 * r < dim;
#pragma unroll
                    for (int q = 0; q < NX; ++q) to[q] = buf_load16(xr, in ? xrow[c][q] : kOutOfRange, (uint32_t)(2 * k0));
                };
                // one sixteen of tokens: its x of two steps; two: those of the next step
                const auto step = [&](uint4 (&from)[2][2], int s, int i) {
                    uint4 wo[2][2];
                    turn_weights<2>(from, tile[wave], wo, lane_here());
                    const float f[2] = {__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv[0]), i)),
                                        __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv[1]), i))};
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        uint4(&xfrom)[4] = x[NC > 1 ? c : s];
                        place_tokens(xfrom, NX, tile[wave], lane_here());
                        load_x(xfrom, NC > 1 ? i + 1 : i + 2, c);
                        if (c + 1 == NC) load_w(from, i + 2);        // last: loads come back in their order
                        multiply<Bf16, FMT, 2>(wo, tile[wave], f, acc[c], lane_here());
                    }
                };
                load_x(x[0], 0, 0);
                if (NC > 1) load_x(x[1], 0, NC - 1);
                load_w(w[0], 0);
                if (NC == 1) load_x(x[1], 1, 0);
                load_w(w[1], 1);
                // both steps always: a step behind the last one multiplies zeros. A branch around loads would make every wait
                // count on the fewest of them
                for (int i = 0; i < steps; i += 2) {
                    step(w[0], 0, i);
                    step(w[1], 1, i + 1);
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) *(v4f32 *)&part[wave][(2 * c + q) * 256 + r * 16 + 4 * g] = acc[c][q];
                }
            };
            using std::integral_constant;
            const integral_constant<int, 1> one;
            const integral_constant<int, 2> two;
            const integral_constant<int, 4> four;
            if (count <= 4) run(one, one);
            else if (count <= 8) run(two, one);
            else if (count <= 16) run(four, one);
            else run(four, two);
            __syncthreads();
            // one hidden unit of one token to a thread
            for (int c = 0; c * 16 < count; ++c) {
                const int i = c * 16 + (int)(threadIdx.x >> 4);
                if (i < count) {
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kUpWaves; ++w) {
                        sum[0] += part[w][c * 512 + threadIdx.x];
                        sum[1] += part[w][c * 512 + 256 + threadIdx.x];
                    }
                    const float a = act<ACT, false>(sum[0]) * sum[1];
                    const int to = (int)(jobs.entry[start + i] & 0xFFFF);
                    const uint32_t scale = umax(max_row16(__float_as_uint(a) & 0x7FFFFFFFu) >> 23, kLeastScale);
                    const float down = __uint_as_float((127 + kScaleBias - scale) << 23);
                    p.a[(int64_t)to * p.hidden + j0 + (threadIdx.x & 15)] = __builtin_bit_cast(uint16_t, (_Float16)(a * down));
                    // the last sixteen also write the zeros that fill the row to whole 128s
                    const int u = (int)(threadIdx.x & 15), at = j0 / 16 + u, bytes = (p.hidden + 127) / 128 * 8;
                    if (u == 0 || (j0 + 16 == p.hidden && at < bytes)) p.a_scales[(int64_t)to * bytes + at] = u == 0 ? (uint8_t)scale : 0;
                }
            }
            __syncthreads();
        }
    }
}

// A workgroup owns 32 columns of y and one of p.parts equal shares of the products: the blocks of 128 hidden units of all
// pieces form one run of steps, cut into 8 p.parts parts. Each wave goes through its part and adds every expert's products,
// weighted, to its own sums of all tokens in LDS; the eight are joined in the order of the waves. With several shares the
// workgroup that comes last joins those of its columns, in their order. The pieces of an expert take turns at each block,
// so its weights are in the L2 for all but the first. One workgroup fills a CU.
constexpr int kDownWaves = 8, kDownThreads = 64 * kDownWaves, kDownTiles = 2, kDownCols = 16 * kDownTiles;

template <int FMT, int CP>
__global__ __launch_bounds__(kDownThreads, 2) void layer_down_kernel(LayerArgs p) {
    constexpr int W = kDownWaves, RT = kDownTiles, COLS = kDownCols;
    extern __shared__ __align__(16) float sums[];     // [waves][tokens][COLS], then the list
    __shared__ __align__(16) char tile[W][4096];
    __shared__ int arrived;
    const int n = p.tokens * p.top_k, total = p.job_count[0], large = p.job_count[1];
    uint32_t *entry = (uint32_t *)(sums + W * p.tokens * COLS);
    float *weight = (float *)(entry + n);
    uint32_t *piece_list = (uint32_t *)(weight + n);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    float *mine = sums + wave * p.tokens * COLS;
    for (int i = lane; i < p.tokens * COLS; i += 64) mine[i] = 0.0f;
    for (int i = threadIdx.x; i < n; i += kDownThreads) {       // what is behind the list's end is not used
        entry[i] = p.entries[i];
        weight[i] = p.entry_weights[i];
        piece_list[i] = p.jobs[i];
    }
    __syncthreads();
    const int hidden = p.hidden, gk = (hidden + 127) / 128, gn = (p.dim + 127) / 128;
    const int column = (int)blockIdx.x / p.parts, share = (int)blockIdx.x % p.parts, d0 = column * COLS;
    // Equal parts in time: a step of up to 32 tokens counts as two of sixteen. us of both kernels, as one and a half / two: 64
    // tokens of 7168, 8 of 64 experts 489 / 488, 40 tokens 445 / 441, 64 of 4096, 4 of 16 experts 118 / 116.5.
    const auto bound = [&](int part) {
        const int64_t first = (int64_t)large * gk, at = (first * 2 + ((int64_t)total * gk - first)) * part / (p.parts * W);
        return (int)(at < first * 2 ? at / 2 : at - first);
    };
    const int lo = bound(share * W + wave), hi = bound(share * W + wave + 1);
    const auto ar = make_rsrc(p.a, (uint32_t)n * (uint32_t)hidden * 2u);
    const auto er = make_rsrc(p.a_scales, (uint32_t)n * (uint32_t)gk * 8u);
    uint32_t wrow[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)                      // columns behind the last one: no loads
        wrow[t] = d0 + 16 * t < p.dim ? (uint32_t)(d0 + 16 * t + (lane >> 3)) * (uint32_t)hidden + 16 * (lane & 7) : kOutOfRange;
    const auto piece_at = [&](int j) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)piece_list[j < total ? j : total - 1]); };

    // Where a step is in the run: the expert's first piece and their number, the block, the piece.
    struct Place {
        int base, pieces, block, piece;
    };
    const auto next = [&](Place &at) {                // whether the expert is another one now
        if (++at.piece < at.pieces) return false;
        at.piece = 0;
        if (++at.block < gk) return false;
        at.block = 0;
        at.base += at.pieces;
        at.pieces = piece_total(piece_at(at.base));
        return true;
    };
    // NX: instructions that load sixteen tokens, NC: sixteens of tokens, enough for each piece of this wave. Loads run ahead of
    // the products, weights two steps and tokens two (NC 2: one), each side with a place of its own, and each step issues the same
    // ones (behind the end: none from memory), so a wait counts on all of them. They come back in their order: tokens loaded later
    // than the next weights would hold those up.
    const auto run = [&](auto instructions, auto sixteens) {
        constexpr int NX = decltype(instructions)::value, NC = decltype(sixteens)::value;
        const uint32_t first = piece_at(lo / gk);
        Place pw;
        pw.base = lo / gk - piece_number(first);
        pw.pieces = piece_total(first);
        pw.block = (lo - pw.base * gk) / pw.pieces;
        pw.piece = (lo - pw.base * gk) % pw.pieces;
        Place px = pw, pu = pw;
        __amdgpu_buffer_rsrc_t wr, sr;
        const auto place_w = [&]() {
            const int e = job_expert(piece_at(pw.base));
            wr = make_rsrc(p.w2 + (int64_t)e * p.dim * hidden, (uint32_t)p.dim * (uint32_t)hidden);
            sr = make_rsrc(p.s2 + ((int64_t)e * gn + d0 / 128) * gk, (uint32_t)gk * 4u);
        };
        uint32_t arow[NC][NX], erow[NC];
        const auto place_x = [&]() {
            const uint32_t piece = piece_at(px.base + px.piece);
            const auto row_at = [&](int at, uint32_t bytes, uint32_t more) {
                const uint32_t row = entry[job_start(piece) + (at < job_count(piece) ? at : 0)] & 0xFFFF;
                return at < job_count(piece) ? row * bytes + more : kOutOfRange;
            };
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                erow[c] = row_at(16 * c + r, (uint32_t)gk * 8u, 0);
#pragma unroll
                for (int q = 0; q < NX; ++q) arow[c][q] = row_at(16 * c + 4 * q + g, (uint32_t)hidden * 2u, 16 * r);
            }
        };
        uint4 w[2][RT][2], x[2][4];
        uint2 ex[2];
        float scale_of[2];
        v4f32 acc[NC][RT];
        const auto clear = [&]() {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int t = 0; t < RT; ++t) acc[c][t] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
        };
        clear();
        const auto load_w = [&](uint4 (&to)[RT][2], float &f, int unit) {
            const int k0 = pw.block * 128;
            const bool in = unit < hi && k0 + 16 * (lane & 7) < hidden;
            // 32 columns lie in one block of 128. A vector load: a scalar one would have every wait for LDS wait for it too
            f = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sr, 0, pw.block * 4, kCached));
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    to[t][h] = buf_load16<CP>(wr, in ? wrow[t] : kOutOfRange, (uint32_t)(k0 + 8 * h * hidden));
            if (next(pw)) place_w();
        };
        const auto load_x = [&](int s, int unit, int c) {
            const int k0 = px.block * 128;
            const bool in = unit < hi && k0 + 8 * r < hidden;
#pragma unroll
            for (int q = 0; q < NX; ++q) x[s][q] = buf_load16(ar, in ? arow[c][q] : kOutOfRange, (uint32_t)(2 * k0));
            const v2u32 e = __builtin_amdgcn_raw_buffer_load_b64(er, (int)(unit < hi ? erow[c] : kOutOfRange), k0 >> 4, kCached);
            ex[s] = make_uint2(e.x, e.y);
            if (c + 1 == NC && (next(px) || px.pieces > 1)) place_x();
        };
        const auto step = [&](int s, int unit) {
            uint4 wo[RT][2];
            turn_weights<RT>(w[s], tile[wave], wo, lane);
            float inv[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) inv[t] = unit < hi ? 1.0f / scale_of[s] : 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int from = NC > 1 ? c : s;
                place_tokens(x[from], NX, tile[wave], lane);
                const uint2 e = ex[from];
                load_x(from, NC > 1 ? unit + 1 : unit + 2, c);
                if (c + 1 == NC) load_w(w[s], scale_of[s], unit + 2);
                _Float16 by[2];
                const float scale = find_scales(e, g, by);
                float f[RT];
#pragma unroll
                // The largest value for Inf (a sum of 0 stays 0), NaN stays. Below 2^-126 it has fewer bits, nine where the largest
                // product of the 128, 2^23 times it, is 2^-117: BF16's own are next to their end there.
                for (int t = 0; t < RT; ++t) {
                    f[t] = inv[t] * scale;
                    f[t] = f[t] > 3.40282346638528859812e+38f ? 3.40282346638528859812e+38f : f[t];
                }
                multiply<Fp16, FMT, RT>(wo, tile[wave], f, acc[c], lane, by);
            }
            if (unit < hi && (pu.pieces > 1 || pu.block + 1 == gk || unit + 1 == hi)) {
                const uint32_t piece = piece_at(pu.base + pu.piece);
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (16 * c + r < job_count(piece)) {
                        const int k = job_start(piece) + 16 * c + r;
                        const float f = weight[k];
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            v4f32 *to = (v4f32 *)(mine + (entry[k] >> 16) * COLS + 16 * t + 4 * g);
                            v4f32 v = *to;
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(f, acc[c][t][q], v[q]);
                            *to = v;
                        }
                    }
                clear();
            }
            next(pu);
        };
        place_w();
        place_x();
        load_x(0, lo, 0);
        if (NC > 1) load_x(1, lo, NC - 1);
        load_w(w[0], scale_of[0], lo);
        if (NC == 1) load_x(1, lo + 1, 0);
        load_w(w[1], scale_of[1], lo + 1);
        for (int u = lo; u < hi; u += 2) {
            step(0, u);
            step(1, u + 1);
        }
    };
    if (lo < hi) {
        int most = 0;
        for (int j = lo / gk; j <= (hi - 1) / gk; ++j) {       // an expert's second piece may have few where its first has 32
            const uint32_t piece = piece_at(j);
            const int count = piece_total(piece) > 1 ? 32 : job_count(piece);
            most = most > count ? most : count;
            if (most > 16) break;
        }
        using std::integral_constant;
        const integral_constant<int, 1> one;
        const integral_constant<int, 2> two;
        const integral_constant<int, 4> four;
        if (most <= 4) run(one, one);
        else if (most <= 8) run(two, one);
        else if (most <= 16) run(four, one);
        else run(four, two);
    }
    __syncthreads();
    const int values = p.tokens * COLS;
    float *part = p.partial + (int64_t)blockIdx.x * values;
    for (int i = threadIdx.x; i < values; i += kDownThreads) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < W; ++v) s += sums[v * values + i];
        const int col = d0 + i % COLS;
        if (p.parts > 1) __hip_atomic_store(&part[i], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        else if (col < p.dim) p.y[(int64_t)(i / COLS) * p.dim + col] = (uint16_t)Eight<uint16_t>::two(s, 0.0f);
    }
    if (p.parts == 1) return;
    // The shares are written, then counted; whoever counts the last one reads them all. (The first kernel cleared the counts.)
    // Every access to a share is one of the device's scope, which passes the XCDs' L2; a fence would write back and
    // invalidate a whole L2 for each workgroup (15 to 25 us).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) arrived = __hip_atomic_fetch_add(&p.arrivals[column], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != p.parts - 1) return;
    for (int i = threadIdx.x; i < values; i += kDownThreads) {
        float s = 0.0f;
        for (int v = 0; v < p.parts; ++v)
            s += __hip_atomic_load(&p.partial[(int64_t)(column * p.parts + v) * values + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int col = d0 + i % COLS;
        if (col < p.dim) p.y[(int64_t)(i / COLS) * p.dim + col] = (uint16_t)Eight<uint16_t>::two(s, 0.0f);
    }
}

int launched() { return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP; }

// Shares of the second kernel's columns: the fewest that fill three quarters of the CUs in every round of workgroups (or the
// most of them), with two steps at least for each wave that may have some. us of the second kernel, one share / this: 13 tokens x 6
// of 40 experts, 2048, hidden 768 27.1 / 15.4 (4 shares), 64 x 4 of 16, 4096, hidden 2048 61 / 41 (2), 4112, hidden 2000 74.5 / 67 (3).
int down_parts(int64_t tokens, int top_k, int experts, int64_t dim, int64_t hidden) {
    const int64_t columns = (dim + kDownCols - 1) / kDownCols, n = tokens * top_k;
    const int64_t steps = (n < experts ? n : experts) * ((hidden + 127) / 128), most = steps / (2 * kDownWaves);
    int best = 1;
    int64_t filled = 0;                               // of 1024
    for (int p = 1; p <= 16 && p <= most; ++p) {
        const int64_t groups = columns * p, f = groups * 1024 / ((groups + 255) / 256 * 256);
        if (f > filled) {
            best = p;
            filled = f;
        }
        if (f >= 768) break;
    }
    return best;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

template <int FMT, int ACT>
int launch_layer_kernels(const LayerArgs &p, hipStream_t s) {
    const int n = p.tokens * p.top_k;
    const int64_t jobs = n < p.experts ? n : p.experts, most = 256 * kUpGroups;
    const int64_t items = p.hidden > 0 ? jobs * (p.hidden / 16) : 1;
    const dim3 grid((unsigned)(items < most ? items : most));
    if (p.dim % 128 == 0) hipLaunchKernelGGL((layer_up_kernel<FMT, ACT, kNonTemporal>), grid, dim3(kUpThreads), 0, s, p);
    else hipLaunchKernelGGL((layer_up_kernel<FMT, ACT, kCached>), grid, dim3(kUpThreads), 0, s, p);
    if (launched() != QF8_OK) return QF8_ERR_HIP;
    const size_t lds = (size_t)kDownWaves * p.tokens * kDownCols * 4 + (size_t)n * 12;
    const dim3 columns((unsigned)(p.columns * p.parts));
    if (p.hidden % 128 == 0) hipLaunchKernelGGL((layer_down_kernel<FMT, kNonTemporal>), columns, dim3(kDownThreads), lds, s, p);
    else hipLaunchKernelGGL((layer_down_kernel<FMT, kCached>), columns, dim3(kDownThreads), lds, s, p);
    return launched();
}

}  // namespace

size_t layer_workspace(int64_t tokens, int top_k, int experts, int64_t dim, int64_t hidden) {
    const size_t n = (size_t)tokens * top_k, columns = ((size_t)dim + kDownCols - 1) / kDownCols;
    const size_t parts = down_parts(tokens, top_k, experts, dim, hidden);
    return up16(n * hidden * 2) + up16(n * ((hidden + 127) / 128 * 8)) + up16(kMaxJobs * 4) + 2 * up16(n * 4) + 16 +
           (parts > 1 ? up16(columns * 4) + columns * parts * tokens * kDownCols * 4 : 0);
}

int launch_layer(const LayerArgs &args, int fmt, int act, void *ws, hipStream_t s) {
    LayerArgs p = args;
    const size_t n = (size_t)p.tokens * p.top_k;
    char *at = (char *)ws;
    p.a = (uint16_t *)at;
    at += up16(n * p.hidden * 2);
    p.a_scales = (uint8_t *)at;
    at += up16(n * ((p.hidden + 127) / 128 * 8));
    p.jobs = (uint32_t *)at;
    at += up16(kMaxJobs * 4);
    p.entries = (uint32_t *)at;
    at += up16(n * 4);
    p.entry_weights = (float *)at;
    at += up16(n * 4);
    p.job_count = (int *)at;
    at += 16;
    p.arrivals = (int *)at;
    p.columns = (p.dim + kDownCols - 1) / kDownCols;
    at += up16((size_t)p.columns * 4);
    p.partial = (float *)at;
    p.parts = down_parts(p.tokens, p.top_k, p.experts, p.dim, p.hidden);
    if (fmt == QF8_E4M3)
        return act == QF8_ACT_SILU ? launch_layer_kernels<kE4M3, QF8_ACT_SILU>(p, s) : launch_layer_kernels<kE4M3, QF8_ACT_GELU>(p, s);
    return act == QF8_ACT_SILU ? launch_layer_kernels<kE5M2, QF8_ACT_SILU>(p, s) : launch_layer_kernels<kE5M2, QF8_ACT_GELU>(p, s);
}

}  // namespace qf8
