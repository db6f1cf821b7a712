// qf8_matmul.h -- matrix products of FP8 codes under fp32 group scales on the gfx950 matrix cores.
//
//   y[i][j] = sum over groups g of 128 along k of  (sum_{k in g} a[i][k] * b[j][k]) / (Sa[i][g] * Sb(j, g))
//
// where a, b are the values of the codes and a group scale S holds fl(x * S) in its codes. Three ways
// to form it (kMath*):
//   kMathFp8    one 16x16x128 FP8 MFMA covers exactly one group of k; its result is the group's
//               partial sum, and what is left per group and element is one fp32 FMA with the
//               quotient of the scales (1/Sa * 1/Sb, each reciprocal one IEEE division, staged once
//               per workgroup and group).
//   kMathE8m0   the same with power-of-two scales: the matrix core applies the exponents itself and
//               accumulates in place, without VALU work.
//   kMathExact  the codes become BF16 (exactly) and go through 32x32x16 BF16 MFMAs, the group's sum
//               then scaled by an FMA.
// Why two precisions: the FP8 MFMAs of gfx950 align the products of each 8 neighbours along k to the
// largest of them and keep 14 bits (measured: beside a product of 2^16 one of 2^3 counts and one of
// 2^2 is lost; 1.4e-5 relative error on normal data, for the 16x16x32 form too), while the BF16
// MFMA keeps fp32's 24 bits. A BF16 result is rounded to 8 bits, a hundred times that error, so it
// takes the FP8 instructions (4.4-4.8 PFLOP/s alone); an FP32 result is asked for where sums count
// (weight gradients) and takes the BF16 ones (1.7 PFLOP/s alone), whose sums are true fp32 sums.
//
// Orientation: b's rows are the MFMA's first operand, so a lane of the result holds one row i of y
// and neighbouring j: 1/Sa is one register per fragment and Sb's block is uniform.
#pragma once
#include "qf8_device.h"
#include "qf8_internal.h"

namespace qf8 {

typedef int v8i32 __attribute__((ext_vector_type(8)));
typedef int v4i32 __attribute__((ext_vector_type(4)));
typedef int v2i32 __attribute__((ext_vector_type(2)));
typedef float v4f32 __attribute__((ext_vector_type(4)));

typedef float v16f32 __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));

enum { kNK = 0, kKN = 1, kGroups = 2 };
enum { kMathFp8 = 0, kMathE8m0 = 1, kMathExact = 2 };
constexpr int kBK = 128;                                  // bytes of k per step: one scale group

// ---- pieces ------------------------------------------------------------------------------------

// A buffer descriptor whose base moves along k: `left` is the number of bytes from the base to the
// end of the tensor, so every lane past it reads zeros.
struct MovingBuffer {
    uint64_t base;
    uint32_t left;
    __device__ __forceinline__ v4i32 rsrc() const {
        v4i32 r;
        r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
        r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xFFFF);
        r.z = __builtin_amdgcn_readfirstlane((int)left);
        r.w = 0x00020000;
        return r;
    }
    __device__ __forceinline__ void advance(uint32_t bytes) {
        base += bytes;
        left = left > bytes ? left - bytes : 0u;
    }
};
__device__ __forceinline__ uint32_t cap31(int64_t bytes) {
    return bytes > 0x7FFFFFFFll ? 0x7FFFFFFFu : bytes < 0 ? 0u : (uint32_t)bytes;
}
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32) |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}

// 16 bytes per lane from buffer offset voff to LDS at lds (wave-uniform byte address) + 16 * lane.
// Written in assembly because the compiler waits for every such load before any later LDS read;
// here the wait is explicit, once per step. It writes no register.
__device__ __forceinline__ void lds_dma16(v4i32 rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(voff), "s"(rsrc) : "memory");
}
__device__ __forceinline__ void wait_vmem() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(lds_u8 *)p;
}

// The transposing read: every 16 lanes read 8 rows of 16 bytes (two lanes a row) and lane i gets byte
// i of each row.
__device__ __forceinline__ v2i32 read_transposed(const uint8_t *p) {
    typedef __attribute__((address_space(3))) v2i32 lds_v2;
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2 *)p);
}

// 1/S, or for power-of-two scales the E8M0 byte of 1/S from S's exponent field.
template <bool POW2>
__device__ __forceinline__ float inverse_scale(float s) {
    if constexpr (POW2) return __uint_as_float(umax(254u - umin((__float_as_uint(s) >> 23) & 0xFFu, 254u), 0u));
    else return 1.0f / s;
}

template <int FA, int FB>
__device__ __forceinline__ v4f32 mfma_raw(v8i32 b, v8i32 a, v4f32 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FB, FA, 0, 0, 0, 0);
}
template <int FA, int FB>
__device__ __forceinline__ v4f32 mfma_e8m0(v8i32 b, v8i32 a, v4f32 c, int eb, int ea) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FB, FA, 0, eb, 0, ea);
}

__device__ __forceinline__ v8i32 join16(uint4 lo, uint4 hi) {
    v8i32 r = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return r;
}

// 8 codes -> 8 BF16 values (exact for both formats).
template <int F>
__device__ __forceinline__ v8bf16 codes_to_bf16(uint32_t lo, uint32_t hi) {
    v2bf16 p[4];
    if constexpr (F == kE4M3) {
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

// Where LDS row rho of a wave's TN rows of b lies among its TN columns of y. The result of an MFMA
// gives a lane rows 4 q + i of every 16 (FP8) or 8 q + 4 h + i of every 32 (BF16); with this order
// they are TN/4 (TN/2) neighbouring columns, stored 16 bytes at a time.
template <int TN, bool EXACT>
__device__ __forceinline__ int column_of(int rho) {
    if constexpr (EXACT) return ((rho >> 2) & 1) * (TN / 2) + 16 * (rho >> 5) + 4 * ((rho >> 3) & 3) + (rho & 3);
    else return ((rho >> 2) & 3) * (TN / 4) + 4 * (rho >> 4) + (rho & 3);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    v2bf16 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Bytes [0, keep) of a 16-byte chunk, the others cleared.
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int keep) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = keep - 4 * i;
        w[i] = n >= 4 ? w[i] : n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- where a tile lies --------------------------------------------------------------------------

struct TilePlace {
    int64_t row0;        // first output row of the tile
    int rows;            // rows of the tile that exist (<= 0: nothing to do)
    int n0;              // first output column
    int expert;          // -1: rows that belong to no expert (zeros)
    int64_t k0, k1;      // range of k
    int split;
};

// Contiguous ranges of tiles for each of the 8 XCDs (workgroups are dealt to them in turn), so that
// tiles that share operands share an L2.
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
    const int64_t x = id & 7, i = id >> 3, q = total >> 3, r = total & 7;
    if (i >= q + (x < r ? 1 : 0)) return -1;
    return x * q + (x < r ? x : r) + i;
}

// Tile number t of tm x tn tiles, in panels of 8 tile rows: neighbours share both operands.
__device__ __forceinline__ void panel_order(int64_t t, int tm, int tn, int &im, int &in) {
    constexpr int kPanel = 8;
    const int64_t per = (int64_t)kPanel * tn;
    const int p = (int)(t / per), r = (int)(t - p * per);
    const int h = tm - p * kPanel < kPanel ? tm - p * kPanel : kPanel;
    im = p * kPanel + r % h;
    in = r / h;
}

// Row tiles of every expert, found by each wave from the offsets: expert e owns rows
// [offsets[e], offsets[e+1]) and ceil(rows / bm) tiles; the rows after the last expert are one more
// stretch, of zeros. Returns the number of row tiles; with want >= 0 also the place of that one.
__device__ __forceinline__ int find_row_tile(const int32_t *offsets, int experts, int64_t nrows, int bm, int want,
                                             TilePlace &pl) {
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int e0 = 0; e0 <= experts; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e < experts) {
            lo = offsets[e];
            hi = offsets[e + 1];
        } else if (e == experts) {
            lo = offsets[experts];
            hi = nrows;
        }
        lo = lo < 0 ? 0 : lo > nrows ? nrows : lo;
        hi = hi < lo ? lo : hi > nrows ? nrows : hi;
        const int c = (int)((hi - lo + bm - 1) / bm);
        int inc = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(inc, d);
            inc += lane >= d ? v : 0;
        }
        const int first = total + inc - c;
        const uint64_t hit = __ballot(want >= first && want < first + c);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int64_t r0 = lo + (int64_t)(want - first) * bm;
            const int64_t left = hi - r0;
            pl.row0 = (int64_t)uniform64((uint64_t)__shfl((long long)r0, src));
            pl.rows = __builtin_amdgcn_readfirstlane(__shfl((int)(left < bm ? left : bm), src));
            pl.expert = e0 + src < experts ? e0 + src : -1;
        }
        total += __builtin_amdgcn_readlane(inc, 63);
    }
    return total;
}

// RUN neighbouring columns of one row, rounded once to BF16 or stored as FP32.
template <int RUN>
__device__ __forceinline__ void store_run(const MatmulArgs &p, const TilePlace &pl, int64_t row, int n, const float *v) {
    const int64_t plane = p.mode == kMatmulExpertsK ? pl.expert : pl.split;
    const int64_t at = (plane * p.m + row) * p.n + n;
    if (p.out_bf16) {
        uint16_t *y = (uint16_t *)p.y + at;
        if (p.vec && n + RUN <= p.n) {
            if constexpr (RUN % 8 == 0) {
#pragma unroll
                for (int e = 0; e < RUN; e += 8)
                    *(uint4 *)(y + e) = make_uint4(pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]),
                                                   pack_bf16(v[e + 4], v[e + 5]), pack_bf16(v[e + 6], v[e + 7]));
            } else {
                *(uint2 *)y = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (n + e < p.n) y[e] = (uint16_t)pack_bf16(v[e], 0.0f);
        }
    } else {
        float *y = (float *)p.y + at;
        if (p.vec && n + RUN <= p.n) {
#pragma unroll
            for (int e = 0; e < RUN; e += 4) *(float4 *)(y + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (n + e < p.n) y[e] = v[e];
        }
    }
}

// ---- the tiled kernel ---------------------------------------------------------------------------

// BM x BN outputs per workgroup, WM x WN waves. Operand tiles of 128 bytes of k go straight from
// memory to LDS, double-buffered: the loads of step s+1 run under the products of step s, with one
// barrier a step.
//
// LDS tiles of rows along k (a, and b unless KN): 128-byte rows of eight 16-byte chunks, chunk c of
// row r at position c ^ (r & 7), so the rows of a fragment read spread over all banks. The lanes of
// the load fetch the permuted chunk, which stays inside the same 128 bytes of memory.
// KN: b's tile keeps k as rows of BN bytes (chunk c of row k at c ^ (k & 7)) and the transposing
// LDS read hands each lane 8 codes along k of one column.
template <int FA, int FB, int KIND, int MATH, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void matmul_tile_kernel(MatmulArgs p) {
    constexpr int NT = 64 * WM * WN, TM = BM / WM, TN = BN / WN;
    constexpr bool POW2 = MATH == kMathE8m0, EXACT = MATH == kMathExact;
    constexpr int FR = EXACT ? 32 : 16, FM = TM / FR, FN = TN / FR;      // fragments
    constexpr int kA = BM * kBK, kB = BN * kBK, kStage = kA + kB;
    constexpr int LA = kA / 16 / NT, LB = kB / 16 / NT;   // loads per thread and step
    constexpr int SB = KIND == kGroups ? BN : (BN + 127) / 128;
    static_assert(LA * NT * 16 == kA && LB * NT * 16 == kB, "tile and workgroup do not match");
    static_assert(BM + SB <= NT * 2, "scales");
    __shared__ __attribute__((aligned(1024))) uint8_t tiles[2][kStage];
    __shared__ float scales[2][BM + SB];

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, g = lane >> 4;

    // ---- the tile of this workgroup
    TilePlace pl;
    pl.split = 0;
    pl.expert = 0;
    const int tn = (p.n + BN - 1) / BN;
    if (p.mode == kMatmulExperts) {
        pl.rows = 0;
        const int tiles_m = find_row_tile(p.offsets, p.experts, p.m, BM, -1, pl);
        const int64_t id = xcd_order(blockIdx.x, (int64_t)tiles_m * tn);
        if (id < 0) return;
        // all columns of up to 4 row tiles, then the next ones: the row tiles of one expert run together
        int im, in;
        constexpr int kPanel = 4;
        const int64_t per = (int64_t)kPanel * tn;
        const int pn = (int)(id / per), rr = (int)(id - pn * per);
        const int h = tiles_m - pn * kPanel < kPanel ? tiles_m - pn * kPanel : kPanel;
        im = pn * kPanel + rr % h;
        in = rr / h;
        find_row_tile(p.offsets, p.experts, p.m, BM, im, pl);
        pl.n0 = in * BN;
        pl.k0 = 0;
        pl.k1 = p.k;
    } else {
        const int tm = (int)((p.m + BM - 1) / BM);
        const int64_t per = (int64_t)tm * tn;
        const int64_t total = per * (p.mode == kMatmulExpertsK ? p.experts : p.splits);
        const int64_t id = xcd_order(blockIdx.x, total);
        if (id < 0) return;
        const int part = (int)(id / per);
        int im, in;
        panel_order(id - part * per, tm, tn, im, in);
        pl.row0 = (int64_t)im * BM;
        pl.rows = (int)(p.m - pl.row0 < BM ? p.m - pl.row0 : BM);
        pl.n0 = in * BN;
        if (p.mode == kMatmulExpertsK) {
            pl.expert = part;
            int64_t lo = p.offsets[part], hi = p.offsets[part + 1];
            lo = lo < 0 ? 0 : lo > p.k ? p.k : lo & ~(int64_t)(kBK - 1);
            hi = hi < lo ? lo : hi > p.k ? p.k : hi;
            pl.k0 = lo;
            pl.k1 = hi;
        } else {
            pl.split = part;
            pl.k0 = (int64_t)part * p.split_k;
            pl.k1 = pl.k0 + p.split_k < p.k ? pl.k0 + p.split_k : p.k;
        }
    }
    const int steps = pl.expert < 0 || pl.k1 <= pl.k0 ? 0 : (int)((pl.k1 - pl.k0 + kBK - 1) / kBK);
    const int kend = (int)(pl.k1 - pl.k0);
    const int gk = (int)((p.k + kBK - 1) / kBK), g0 = (int)(pl.k0 / kBK);
    const bool gather = p.rows != nullptr;

    // ---- operand addresses
    MovingBuffer ba, bb;
    uint32_t va[LA], vb[LB];
    if (gather) {
        ba.base = uniform64((uint64_t)(uintptr_t)p.a);
        ba.left = (uint32_t)(p.a_rows * p.k);
    } else {
        ba.base = uniform64((uint64_t)(uintptr_t)p.a + (uint64_t)(pl.row0 * p.k + pl.k0));
        ba.left = cap31((p.m - pl.row0) * p.k - pl.k0);
    }
    ba.left = __builtin_amdgcn_readfirstlane((int)ba.left);
    auto a_row = [&](int r) -> int64_t {               // row of a for tile row r; rows past the end repeat the last
        r = r < pl.rows ? r : pl.rows - 1;
        if (!gather) return r;
        const int64_t v = p.rows[pl.row0 + r];
        return v < 0 || v >= p.a_rows ? 0 : v;         // no such row: any values, the result is not stored
    };
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int id = i * NT + t, row = id >> 3, ch = (id & 7) ^ (row & 7);
        va[i] = steps ? (uint32_t)(a_row(row) * p.k) + 16u * ch : 0u;
    }
    const uint64_t bmat = (uint64_t)(p.mode == kMatmulExperts && pl.expert > 0 ? pl.expert : 0) * (uint64_t)p.n * (uint64_t)p.k;
    if constexpr (KIND == kKN) {
        bb.base = uniform64((uint64_t)(uintptr_t)p.b + bmat + (uint64_t)(pl.k0 * p.n + pl.n0));
        bb.left = cap31((p.k - pl.k0) * p.n - pl.n0);
        constexpr int C = BN / 16;
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            const int id = i * NT + t, kr = id / C, ch = (id % C) ^ (kr & 7);
            vb[i] = (uint32_t)kr * (uint32_t)p.n + 16u * ch;
        }
    } else {
        bb.base = uniform64((uint64_t)(uintptr_t)p.b + bmat + (uint64_t)((int64_t)pl.n0 * p.k + pl.k0));
        bb.left = cap31((int64_t)(p.n - pl.n0) * p.k - pl.k0);
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            const int id = i * NT + t, row = id >> 3, ch = (id & 7) ^ (row & 7);
            int n = (row / TN) * TN + column_of<TN, EXACT>(row % TN);
            n = n < p.n - pl.n0 ? n : p.n - pl.n0 - 1;
            vb[i] = (uint32_t)n * (uint32_t)p.k + 16u * ch;
        }
    }
    bb.left = __builtin_amdgcn_readfirstlane((int)bb.left);
    const uint32_t stepb = KIND == kKN ? (uint32_t)kBK * (uint32_t)p.n : (uint32_t)kBK;

    // ---- scale addresses: thread u < BM loads a row's scale, BM <= u < BM + SB one of b
    constexpr int LS = (BM + SB + NT - 1) / NT;
    const float *sp[LS];
#pragma unroll
    for (int i = 0; i < LS; ++i) {
        const int u = i * NT + t;
        if (u < BM) {
            const int64_t r = gather ? a_row(u) : pl.row0 + a_row(u);
            sp[i] = p.sa + (steps ? r : 0) * gk + g0;
        } else if (u < BM + SB) {
            const int v = u - BM;
            if constexpr (KIND == kGroups) {
                int n = pl.n0 + (v / TN) * TN + column_of<TN, EXACT>(v % TN);
                n = n < p.n ? n : p.n - 1;
                sp[i] = p.sb + (int64_t)n * gk + g0;
            } else if constexpr (KIND == kNK) {
                const int gn = (p.n + 127) / 128;
                int nb = pl.n0 / 128 + v;
                nb = nb < gn ? nb : gn - 1;
                sp[i] = p.sb + ((int64_t)(pl.expert > 0 ? pl.expert : 0) * gn + nb) * gk + g0;
            } else {                                    // scales [k/128][n/128]: one row of them per step
                const int gn = (p.n + 127) / 128;
                int nb = pl.n0 / 128 + v;
                nb = nb < gn ? nb : gn - 1;
                sp[i] = p.sb + ((int64_t)(pl.expert > 0 ? pl.expert : 0) * gk + g0) * gn + nb;
            }
        } else {
            sp[i] = nullptr;
        }
    }
    const int sstep_b = KIND == kKN ? (p.n + 127) / 128 : 1;

    constexpr int FV = FR * FR / 64;                     // values of a fragment in a lane
    float acc[FM][FN][FV];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < FV; ++e) acc[i][j][e] = 0.0f;

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((int)lds_address(&tiles[0][0])) + (uint32_t)wave * 1024u;
    float sreg[LS];
    auto load_step = [&](int s) {
        const uint32_t at = lds0 + (uint32_t)(s & 1) * kStage;
        const v4i32 ra = ba.rsrc(), rb = bb.rsrc();
#pragma unroll
        for (int i = 0; i < LA; ++i) lds_dma16(ra, va[i], at + (uint32_t)i * NT * 16);
#pragma unroll
        for (int i = 0; i < LB; ++i) lds_dma16(rb, vb[i], at + kA + (uint32_t)i * NT * 16);
        ba.advance(kBK);
        bb.advance(stepb);
#pragma unroll
        for (int i = 0; i < LS; ++i) {
            if (sp[i]) {
                sreg[i] = *sp[i];
                sp[i] += i * NT + t < BM ? 1 : sstep_b;
            }
        }
    };

    if (steps) load_step(0);
    for (int s = 0; s < steps; ++s) {
        wait_vmem();
        float *sc = scales[s & 1];
#pragma unroll
        for (int i = 0; i < LS; ++i)
            if (i * NT + t < BM + SB) sc[i * NT + t] = inverse_scale<POW2>(sreg[i]);
        __syncthreads();
        uint8_t *const ta = tiles[s & 1], *const tb = ta + kA;
        const int krem = kend - s * kBK;
        if (krem < kBK) {                               // the last step of a k that is no multiple of 128
#pragma unroll
            for (int i = 0; i < LA; ++i) {
                const int id = i * NT + t, row = id >> 3, ch = (id & 7) ^ (row & 7);
                uint4 *at = (uint4 *)(ta + 16 * id);
                if (16 * ch + 16 > krem) *at = keep_bytes(*at, krem - 16 * ch);
            }
#pragma unroll
            for (int i = 0; i < LB; ++i) {
                const int id = i * NT + t;
                uint4 *at = (uint4 *)(tb + 16 * id);
                if constexpr (KIND == kKN) {
                    if (id / (BN / 16) >= krem) *at = make_uint4(0, 0, 0, 0);
                } else {
                    const int row = id >> 3, ch = (id & 7) ^ (row & 7);
                    if (16 * ch + 16 > krem) *at = keep_bytes(*at, krem - 16 * ch);
                }
            }
            __syncthreads();
        }
        if (s + 1 < steps) load_step(s + 1);

        if constexpr (EXACT) {
            // lane (r32, h): row r32 of a fragment; slice u of 16 k holds, for half h, the 8 codes at
            // k = 16 (2 (u / 2) + h) + 8 (u % 2)
            const int r32 = lane & 31, h = lane >> 5;
            v8bf16 fb[FN][8];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (KIND == kKN) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int kr = 16 * (2 * (u >> 1) + h) + 8 * (u & 1) + (r16 >> 1);
                        const int ch = (wn * TN + 32 * j) / 16 + ((lane >> 4) & 1);
                        const v2i32 q = read_transposed(tb + kr * BN + ((ch ^ (kr & 7)) << 4) + 8 * (r16 & 1));
                        fb[j][u] = codes_to_bf16<FB>((uint32_t)q.x, (uint32_t)q.y);
                    }
                } else {
                    const int row = wn * TN + 32 * j + r32;
#pragma unroll
                    for (int u = 0; u < 8; u += 2) {
                        const uint4 q = *(const uint4 *)(tb + row * kBK + (((u + h) ^ (row & 7)) << 4));
                        fb[j][u] = codes_to_bf16<FB>(q.x, q.y);
                        fb[j][u + 1] = codes_to_bf16<FB>(q.z, q.w);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int row = wm * TM + 32 * i + r32;
                v16f32 part[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) part[j][e] = 0.0f;
#pragma unroll
                for (int u = 0; u < 8; u += 2) {
                    const uint4 q = *(const uint4 *)(ta + row * kBK + (((u + h) ^ (row & 7)) << 4));
                    const v8bf16 f0 = codes_to_bf16<FA>(q.x, q.y), f1 = codes_to_bf16<FA>(q.z, q.w);
#pragma unroll
                    for (int j = 0; j < FN; ++j) part[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j][u], f0, part[j], 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < FN; ++j) part[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j][u + 1], f1, part[j], 0, 0, 0);
                }
                const float sa = sc[row];
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (KIND == kGroups) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const v4f32 sb = *(const v4f32 *)(sc + BM + wn * TN + 32 * j + 8 * q + 4 * h);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[i][j][4 * q + e] = __builtin_fmaf(part[j][4 * q + e] * sa, sb[e], acc[i][j][4 * q + e]);
                        }
                    } else {
                        const float f = sa * sc[BM + wn * TN / 128];
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[i][j][e] = __builtin_fmaf(part[j][e], f, acc[i][j][e]);
                    }
                }
            }
        } else {
            // fragments of b: lane (r16, g) holds row r16 and k = 16 g + [0, 16) and 64 + 16 g + [0, 16)
            v8i32 fb[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (KIND == kKN) {
                    v2i32 q[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        // 16 lanes read 8 rows of k x 16 columns; two neighbouring lanes cover a row
                        const int kr = (h >> 1) * 64 + 16 * g + 8 * (h & 1) + (r16 >> 1);
                        const int ch = (wn * TN + 16 * j) / 16;
                        const uint8_t *src = tb + kr * BN + ((ch ^ (kr & 7)) << 4) + 8 * (r16 & 1);
                            q[h] = read_transposed(src);
                    }
                    fb[j] = v8i32{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
                } else {
                    const int row = wn * TN + 16 * j + r16;
                    const uint8_t *src = tb + row * kBK;
                    fb[j] = join16(*(const uint4 *)(src + ((g ^ (row & 7)) << 4)),
                                   *(const uint4 *)(src + (((g + 4) ^ (row & 7)) << 4)));
                }
            }
            float sbu = 0.0f;
            v4f32 sbg[FN];
            int ebg[FN];
            if constexpr (KIND == kGroups) {
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (POW2) ebg[j] = __float_as_int(sc[BM + wn * TN + 16 * j + r16]);
                    else sbg[j] = *(const v4f32 *)(sc + BM + wn * TN + 16 * j + 4 * g);
                }
            } else {
                sbu = sc[BM + wn * TN / 128];
#pragma unroll
                for (int j = 0; j < FN; ++j) ebg[j] = __float_as_int(sbu);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int row = wm * TM + 16 * i + r16;
                const uint8_t *src = ta + row * kBK;
                const v8i32 fa = join16(*(const uint4 *)(src + ((g ^ (row & 7)) << 4)),
                                        *(const uint4 *)(src + (((g + 4) ^ (row & 7)) << 4)));
                const float sa = sc[row];
                if constexpr (POW2) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const v4f32 c = mfma_e8m0<FA, FB>(fb[j], fa, v4f32{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]},
                                                          ebg[j], __float_as_int(sa));
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] = c[e];
                    }
                } else {
                    v4f32 part[FN];
#pragma unroll
                    for (int j = 0; j < FN; ++j) part[j] = mfma_raw<FA, FB>(fb[j], fa, v4f32{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        if constexpr (KIND == kGroups) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[j][e] * sa, sbg[j][e], acc[i][j][e]);
                        } else {
                            const float f = sa * sbu;
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[j][e], f, acc[i][j][e]);
                        }
                    }
                }
            }
        }
    }

    // ---- store
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = wm * TM + FR * i + (EXACT ? lane & 31 : r16);
        if (r >= pl.rows) continue;
        const int64_t row = pl.row0 + r;
        bool zero = false;
        if (gather) {
            const int64_t src = p.rows[row];
            zero = src < 0 || src >= p.a_rows;
        }
        // runs of neighbouring columns: all a lane holds, or 4 with KN, whose columns keep their order
        constexpr int PER = TN * FR / 64, RUN = KIND == kKN ? 4 : PER;
        const int q = lane / FR;
#pragma unroll
        for (int u = 0; u < PER / RUN; ++u) {
            int n = pl.n0 + wn * TN;
            if constexpr (KIND != kKN) n += q * PER;
            else if constexpr (EXACT) n += 32 * (u >> 2) + 8 * (u & 3) + 4 * q;
            else n += 16 * u + 4 * q;
            float v[RUN];
#pragma unroll
            for (int e = 0; e < RUN; ++e) {
                const int at = u * RUN + e;
                v[e] = zero ? 0.0f : acc[i][at / FV][at % FV];
            }
            store_run<RUN>(p, pl, row, n, v);
        }
    }
}

// ---- launch ----------------------------------------------------------------------------------------

struct TileSize { int bm, bn; };
constexpr TileSize kTileSizes[2][3] = {{{256, 256}, {128, 128}, {64, 128}},      // FP8 MFMAs
                                       {{256, 128}, {128, 128}, {64, 128}}};     // BF16 MFMAs

template <int FA, int FB, int KIND, int MATH>
int launch_matmul_tile(const MatmulArgs &p, int size, int64_t groups, hipStream_t s) {
    const dim3 grid((unsigned)groups);
    if (size == 0) {
        if constexpr (MATH == kMathExact) hipLaunchKernelGGL((matmul_tile_kernel<FA, FB, KIND, MATH, 256, 128, 4, 2>), grid, dim3(512), 0, s, p);
        else hipLaunchKernelGGL((matmul_tile_kernel<FA, FB, KIND, MATH, 256, 256, 2, 4>), grid, dim3(512), 0, s, p);
    } else if (size == 1) {
        hipLaunchKernelGGL((matmul_tile_kernel<FA, FB, KIND, MATH, 128, 128, 2, 2>), grid, dim3(256), 0, s, p);
    } else {
        hipLaunchKernelGGL((matmul_tile_kernel<FA, FB, KIND, MATH, 64, 128, 1, 4>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP;
}

template <int FA, int FB, int KIND>
int launch_matmul_kind(const MatmulArgs &p, int math, int size, int64_t groups, hipStream_t s) {
    if (math == kMathFp8) return launch_matmul_tile<FA, FB, KIND, kMathFp8>(p, size, groups, s);
    if (math == kMathE8m0) return launch_matmul_tile<FA, FB, KIND, kMathE8m0>(p, size, groups, s);
    return launch_matmul_tile<FA, FB, KIND, kMathExact>(p, size, groups, s);
}

template <int FA, int FB>
int launch_matmul_formats(const MatmulArgs &p, int kind, int math, int size, int64_t groups, hipStream_t s) {
    if (kind == kNK) return launch_matmul_kind<FA, FB, kNK>(p, math, size, groups, s);
    if (kind == kKN) return launch_matmul_kind<FA, FB, kKN>(p, math, size, groups, s);
    return launch_matmul_kind<FA, FB, kGroups>(p, math, size, groups, s);
}

}  // namespace qf8
