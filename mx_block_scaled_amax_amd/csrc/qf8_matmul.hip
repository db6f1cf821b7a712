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

// Tile size and split of k by a model of the time, in us, fitted to sweeps over m 1-8192, n 512-7168,
// k 512-16384 (its choice is within 10% of the best of all sizes and splits in most of them, 25% in
// the worst). A workgroup takes a fixed time and one per step of k, longer where two share a CU;
// workgroups run in rounds of what the CUs hold; parts of a split k are joined by a second kernel.
// tiles: number of output tiles of a size, which for experts is an estimate.
// Two operands in 1x128 groups with FP8 sums take the 256 x 256 tile in its plain form, 1.7-2.1 us a step, and the
// same times in the plan. Measured, us, 256 x 256 / 128 x 128 (the plan takes the lower one): 2048 x 2048 x 4096 65 / 39,
// 3000 x 3000 x 4096 68 / 75, 7168 x 4096 x 8192 252 / 306; power-of-two scales 57 / 39, 58 / 73, 223 / 283. A step of
// 2.05 us in the plan gave the same choices, but no split of 2048 x 2048 x 16384 in that tile: 98 -> 122 us.
template <typename Tiles>
Plan plan_matmul(int64_t k, double outputs, bool may_split, bool exact, Tiles tiles) {
    struct Step { double alone, shared; };                  // us per step of k
    constexpr Step kStep[2][kTileCount] = {{{1.50, 1.90}, {0.78, 1.30}, {0.47, 0.83}, {0.39, 0.63}},
                                           {{1e9, 1e9}, {1.40, 2.40}, {1.04, 1.60}, {0.78, 1.09}}};
    const int64_t steps = (k + kBK - 1) / kBK;
    Plan best = {2, 1, steps * kBK};
    double best_t = 1e300;
    for (int size = 0; size < kTileCount; ++size) {
        const double count = tiles(kTileSizes[size]);
        const Step c = kStep[exact][size];
        for (int splits = 1; splits <= (may_split ? 16 : 1); splits *= 2) {
            const int64_t per = (steps + splits - 1) / splits;
            const double bytes = (double)splits * outputs * 4.0;
            if (splits > 1 && (per < 2 || bytes > (double)((int64_t)256 << 20))) break;
            const double groups = count * splits, slots = (double)kCUs * kTileSizes[size].fit;
            const double full = groups > slots ? (double)(int64_t)((groups - 1.0) / slots) : 0.0;   // rounds before the last
            const double last = groups - full * slots;
            double t = 5.0 + (double)(per + 1) * (full * c.shared + (last > (size == 0 ? 0.75 * kCUs : kCUs) ? c.shared : c.alone));
            if (splits > 1) t += 2.5 + 0.1 * splits + 2.0 * bytes / 4e6;
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

Plan plan_dense(int64_t m, int64_t n, int64_t k, bool exact) {
    return plan_matmul(k, (double)m * (double)n, true, exact, [=](const TileSize &t) {
        return (double)((m + t.bm - 1) / t.bm) * (double)((n + t.bn - 1) / t.bn);
    });
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
    if (groups * (size == 0 ? 512 : 256) > 0xFFFFFFFFll) return QF8_ERR_SHAPE;       // a launch counts threads in 32 bits
    if (fa == kE4M3)
        return fb == kE4M3 ? launch_matmul_formats<kE4M3, kE4M3>(p, kind, math, size, groups, s)
                           : launch_matmul_formats<kE4M3, kE5M2>(p, kind, math, size, groups, s);
    return fb == kE4M3 ? launch_matmul_formats<kE5M2, kE4M3>(p, kind, math, size, groups, s)
                       : launch_matmul_formats<kE5M2, kE5M2>(p, kind, math, size, groups, s);
}

}  // namespace

size_t matmul_workspace(int64_t m, int64_t n, int64_t k, int kind, int fp32_sums) {
    (void)kind;
    if (m == 0 || n == 0 || k == 0) return 0;
    const Plan pl = plan_dense(m, n, k, fp32_sums != 0);
    return pl.splits > 1 ? (size_t)pl.splits * m * n * sizeof(float) : 0;
}

int launch_matmul(const MatmulArgs &args, int fmt_a, int fmt_b, int kind, int pow2, float *ws, hipStream_t s) {
    MatmulArgs p = args;
    if (p.m == 0 || p.n == 0) return QF8_OK;
    p.splits = 1;
    p.split_k = p.k;
    const bool exact = args.fp32_sums != 0;
    const int math = exact ? (pow2 ? kMathExactPow2 : kMathExact) : pow2 ? kMathE8m0 : kMathFp8;
    const TileSize *sizes = kTileSizes;
    if (p.mode == kMatmulDense) {
        const Plan pl = plan_dense(p.m, p.n, p.k, exact);
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
        const int64_t mean = p.k / p.experts + 1;
        const Plan pl = plan_matmul(mean, 0.0, false, exact, [&](const TileSize &t) {
            return (double)((p.m + t.bm - 1) / t.bm) * (double)((p.n + t.bn - 1) / t.bn) * p.experts;
        });
        const int64_t tiles = ((p.m + sizes[pl.size].bm - 1) / sizes[pl.size].bm) *
                              ((p.n + sizes[pl.size].bn - 1) / sizes[pl.size].bn);
        return launch_by_format(p, fmt_a, fmt_b, kind, math, pl.size, (tiles + 7) / 8 * 8 * p.experts, s);
    }
    // the rows of an expert end inside a tile: half a tile more for each that has rows
    const double used = (double)(p.m < p.experts ? p.m : p.experts);
    const Plan pl = plan_matmul(p.k, 0.0, false, exact, [&](const TileSize &t) {
        const double rows = (double)p.m / t.bm + 0.5 * used;
        return (rows > used ? rows : used) * (double)((p.n + t.bn - 1) / t.bn);
    });
    // the experts and the rows before and after them: each stretch may end inside a tile
    const int64_t tm = p.m / sizes[pl.size].bm + p.experts + 2, tn = (p.n + sizes[pl.size].bn - 1) / sizes[pl.size].bn;
    return launch_by_format(p, fmt_a, fmt_b, kind, math, pl.size, tm * tn, s);
}

}  // namespace qf8
