// qf8_matmul.hip -- host side of the matrix products: tile size, split of k, launch; and the sum of
// the parts of a split k.
#include "qf8_matmul.h"

namespace qf8 {

// instantiated in qf8_matmul_<a>_<b>.hip
extern template int launch_matmul_formats<kE4M3, kE4M3>(const MatmulArgs &, int, int, int, int64_t, hipStream_t);
extern template int launch_matmul_formats<kE4M3, kE5M2>(const MatmulArgs &, int, int, int, int64_t, hipStream_t);
extern template int launch_matmul_formats<kE5M2, kE4M3>(const MatmulArgs &, int, int, int, int64_t, hipStream_t);
extern template int launch_matmul_formats<kE5M2, kE5M2>(const MatmulArgs &, int, int, int, int64_t, hipStream_t);

namespace {

constexpr int kCUs = 256;

struct Plan { int size, splits; int64_t split_k; };

// Tile size and split of k from a model of the time: workgroups run in rounds of CUs x (workgroups
// that fit on one), a round costs its steps of k.
Plan plan_matmul(int64_t m, int64_t n, int64_t k, int parts, bool may_split, bool exact) {
    // cycles of one step of k of a full CU: FP8, BF16 products
    constexpr double kStep[2][kTileCount] = {{4300.0, 2900.0, 2250.0, 1900.0},
                                             {1e9, 4600.0, 3900.0, 3400.0}};
    const TileSize *sizes = kTileSizes;
    const int64_t steps = (k + kBK - 1) / kBK;
    Plan best = {2, 1, steps * kBK};
    double best_t = 1e300;
    for (int size = 0; size < kTileCount; ++size) {
        const int64_t tiles = ((m + sizes[size].bm - 1) / sizes[size].bm) *
                              ((n + sizes[size].bn - 1) / sizes[size].bn) * parts;
        for (int splits = 1; splits <= (may_split ? 16 : 1); splits *= 2) {
            const int64_t per = (steps + splits - 1) / splits;
            if (splits > 1 && (per < 4 || (int64_t)splits * m * n * 4 > (int64_t)256 << 20)) break;
            const int64_t slots = (int64_t)kCUs * sizes[size].fit;
            const int64_t rounds = (tiles * splits + slots - 1) / slots;
            double t = (double)rounds * (double)(per + 3) * kStep[exact][size];
            if (splits > 1) t += 6000.0 + (double)splits * (double)m * (double)n * 8.0 / 2000.0;
            if (t < best_t) {
                best_t = t;
                best.size = size;
                best.splits = splits;
                best.split_k = per * kBK;
            }
        }
    }
    best.splits = best.splits > 1 ? (int)((steps * kBK + best.split_k - 1) / best.split_k) : 1;
    return best;
}

// y = sum over the parts in their order, rounded once.
template <typename T>
__global__ __launch_bounds__(256) void matmul_join_kernel(const float *parts, int splits, int64_t count, T *y) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i + 4 <= count && (count & 3) == 0) {
        float4 s = *(const float4 *)(parts + i);
        for (int p = 1; p < splits; ++p) {
            const float4 v = *(const float4 *)(parts + p * count + i);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        if constexpr (sizeof(T) == 2) *(uint2 *)(y + i) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
        else *(float4 *)(y + i) = s;
    } else {
        for (int64_t j = i; j < i + 4 && j < count; ++j) {
            float s = parts[j];
            for (int p = 1; p < splits; ++p) s += parts[p * count + j];
            if constexpr (sizeof(T) == 2) y[j] = (T)pack_bf16(s, 0.0f);
            else y[j] = s;
        }
    }
}

int launch_by_format(const MatmulArgs &p, int fa, int fb, int kind, int math, int size, int64_t groups, hipStream_t s) {
    if (fa == kE4M3)
        return fb == kE4M3 ? launch_matmul_formats<kE4M3, kE4M3>(p, kind, math, size, groups, s)
                           : launch_matmul_formats<kE4M3, kE5M2>(p, kind, math, size, groups, s);
    return fb == kE4M3 ? launch_matmul_formats<kE5M2, kE4M3>(p, kind, math, size, groups, s)
                       : launch_matmul_formats<kE5M2, kE5M2>(p, kind, math, size, groups, s);
}

}  // namespace

size_t matmul_workspace(int64_t m, int64_t n, int64_t k, int kind, int out_bf16) {
    (void)kind;
    if (m == 0 || n == 0 || k == 0) return 0;
    const Plan pl = plan_matmul(m, n, k, 1, true, !out_bf16);
    return pl.splits > 1 ? (size_t)pl.splits * m * n * sizeof(float) : 0;
}

int launch_matmul(const MatmulArgs &args, int fmt_a, int fmt_b, int kind, int pow2, float *ws, hipStream_t s) {
    MatmulArgs p = args;
    if (p.m == 0 || p.n == 0) return QF8_OK;
    p.splits = 1;
    p.split_k = p.k;
    const bool exact = !args.out_bf16;
    const int math = exact ? (pow2 ? kMathExactPow2 : kMathExact) : pow2 ? kMathE8m0 : kMathFp8;
    const TileSize *sizes = kTileSizes;
    if (p.mode == kMatmulDense) {
        const Plan pl = plan_matmul(p.m, p.n, p.k, 1, true, exact);
        const int64_t tiles = ((p.m + sizes[pl.size].bm - 1) / sizes[pl.size].bm) *
                              ((p.n + sizes[pl.size].bn - 1) / sizes[pl.size].bn);
        if (pl.splits == 1) return launch_by_format(p, fmt_a, fmt_b, kind, math, pl.size, tiles, s);
        p.splits = pl.splits;
        p.split_k = pl.split_k;
        p.y = ws;
        p.out_bf16 = 0;
        const int st = launch_by_format(p, fmt_a, fmt_b, kind, math, pl.size, tiles * pl.splits, s);
        if (st != QF8_OK) return st;
        const int64_t count = p.m * p.n;
        const dim3 grid((unsigned)((count + 1023) / 1024));
        if (args.out_bf16)
            hipLaunchKernelGGL((matmul_join_kernel<uint16_t>), grid, dim3(256), 0, s, ws, pl.splits, count, (uint16_t *)args.y);
        else
            hipLaunchKernelGGL((matmul_join_kernel<float>), grid, dim3(256), 0, s, ws, pl.splits, count, (float *)args.y);
        return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP;
    }
    if (p.mode == kMatmulExpertsK) {
        const int64_t mean = p.k / (p.experts > 0 ? p.experts : 1) + 1;
        const Plan pl = plan_matmul(p.m, p.n, mean, p.experts, false, exact);
        const int64_t tiles = ((p.m + sizes[pl.size].bm - 1) / sizes[pl.size].bm) *
                              ((p.n + sizes[pl.size].bn - 1) / sizes[pl.size].bn);
        return launch_by_format(p, fmt_a, fmt_b, kind, math, pl.size, tiles * p.experts, s);
    }
    const int64_t mean = p.m / (p.experts > 0 ? p.experts : 1) + 1;
    const Plan pl = plan_matmul(mean, p.n, p.k, p.experts, false, exact);
    const int64_t tm = p.m / sizes[pl.size].bm + p.experts + 1, tn = (p.n + sizes[pl.size].bn - 1) / sizes[pl.size].bn;
    return launch_by_format(p, fmt_a, fmt_b, kind, math, pl.size, tm * tn, s);
}

}  // namespace qf8
