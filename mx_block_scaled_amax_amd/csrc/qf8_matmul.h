// qf8_matmul.h -- matrix products of FP8 codes under fp32 group scales on the gfx950 matrix cores.
//
//   y[i][j] = sum over groups g of 128 along k of  (sum_{k in g} a[i][k] * b[j][k]) / (Sa[i][g] * Sb(j, g))
//
// where a, b are the values of the codes and a group scale S holds fl(x * S) in its codes. Four ways
// to form it (kMath*):
//   kMathFp8    one 16x16x128 FP8 MFMA covers exactly one group of k; its result is the group's
//               partial sum, and what is left per group and element is one fp32 FMA with the
//               quotient of the scales (1/Sa * 1/Sb, each reciprocal one IEEE division, staged once
//               per workgroup and group).
//   kMathE8m0   the same with power-of-two scales: the matrix core applies the exponents itself and
//               accumulates in place, without VALU work.
//   kMathExact  the codes become BF16 (exactly) and go through 32x32x16 BF16 MFMAs, the group's sum
//               then scaled by an FMA.
//   kMathExactPow2  the same with power-of-two scales: the conversion to BF16 multiplies by 1/S,
//               which is exact for 1/S of 2^-64 to 2^64, and the sums need no scaling. A tile that meets
//               another scale is done again as by kMathExact.
// Why two precisions: the FP8 MFMAs of gfx950 align the products of each 8 neighbours along k to the
// largest of them and keep 14 bits (measured: beside a product of 2^16 one of 2^3 counts and one of
// 2^2 is lost; 1.4e-5 relative error on normal data, for the 16x16x32 form too), while the BF16
// MFMA keeps fp32's 24 bits. A BF16 result is rounded to 8 bits, a hundred times that error, so it
// takes the FP8 instructions (4.4-4.8 PFLOP/s alone); an FP32 result is asked for where sums count
// (weight gradients) and takes the BF16 ones (1.7 PFLOP/s alone), whose sums are true fp32 sums, as does a
// BF16 result on request.
//
// Orientation: b's rows are the MFMA's first operand, so a lane of the result holds one row i of y
// and neighbouring j: 1/Sa is one register per fragment and Sb's block is uniform.
#pragma once
#include <type_traits>
#include "qf8_device.h"
#include "qf8_internal.h"

// Lambdas called from two loops: outlined, their variables would live in memory and no longer be uniform.
#define QF8_INLINE __attribute__((always_inline))

namespace qf8 {

typedef int v8i32 __attribute__((ext_vector_type(8)));
typedef int v4i32 __attribute__((ext_vector_type(4)));
typedef int v2i32 __attribute__((ext_vector_type(2)));
typedef float v4f32 __attribute__((ext_vector_type(4)));

typedef float v16f32 __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));

enum { kNK = 0, kKN = 1, kGroups = 2 };
enum { kMathFp8 = 0, kMathE8m0 = 1, kMathExact = 2, kMathExactPow2 = 3 };
constexpr int kBK = 128;                                  // bytes of k per step: one scale group

// ---- pieces ------------------------------------------------------------------------------------

// Position of chunk 0 of a 128-byte row in LDS. A 16-byte read serves 16 lanes a cycle (0-3, 12-15,
// 20-23 and 24-27 of each half wave): two rows fill the 64 banks, so the 8 even and the 8 odd rows
// among those lanes need 8 positions each, for fragments of 16 rows x 4 chunks and of 32 rows x 2
// alike. Measured 233 bytes a cycle; with r & 7 the 32-row form took twice as long.
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

// A buffer descriptor whose base moves along k: `left` is the number of bytes from the base to the
// end of the tensor, so every lane past it reads zeros. LONG: the base may move over 4 GiB and more
// (whole rows of k), where a count capped at its start would run out before the tensor does.
template <bool LONG>
struct MovingBufferOf {
    typedef typename std::conditional<LONG, uint64_t, uint32_t>::type Count;
    uint64_t base;
    Count left;
    __device__ __forceinline__ v4i32 rsrc() const {
        v4i32 r;
        r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
        r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xFFFF);
        r.z = __builtin_amdgcn_readfirstlane((int)(uint32_t)(LONG && left > 0xFFFFFFFFu ? 0xFFFFFFFFu : left));
        r.w = 0x00020000;
        return r;
    }
    __device__ __forceinline__ void advance(uint32_t bytes) {
        base += bytes;
        left = left > bytes ? left - bytes : 0u;
    }
};
typedef MovingBufferOf<false> MovingBuffer;
__device__ __forceinline__ uint32_t cap31(int64_t bytes) {
    return bytes > 0x7FFFFFFFll ? 0x7FFFFFFFu : bytes < 0 ? 0u : (uint32_t)bytes;
}
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32) |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}

// 16 bytes per lane from buffer offset voff to LDS at lds (wave-uniform byte address) + 16 * lane.
// Written in assembly because the compiler waits for every such load before any later LDS read;
// here the wait is explicit, once per step. It writes no register but M0, which is reserved: the compiler
// keeps no value there and sets it before each use of its own.
__device__ __forceinline__ void lds_dma16(v4i32 rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(voff), "s"(rsrc) : "memory");
}
__device__ __forceinline__ void lds_dma4(v4i32 rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(voff), "s"(rsrc) : "memory");
}
template <int N> __device__ __forceinline__ void wait_vmem_but() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory"); }
// End of a phase: this wave's LDS traffic is done; then the workgroup meets.
__device__ __forceinline__ void phase_end() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
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
template <int MATH>
__device__ __forceinline__ float inverse_scale(float s) {
    if constexpr (MATH == kMathE8m0) return __uint_as_float(umax(254u - umin((__float_as_uint(s) >> 23) & 0xFFu, 254u), 0u));
    else return 1.0f / s;
}

// 2^-64 <= f <= 2^64: BF16 holds any code (2^-16 to 2^16) times f in full.
__device__ __forceinline__ bool near_one(float f) {
    return __float_as_uint(f) - 0x1F800000u <= 0x5F800000u - 0x1F800000u;
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

// 8 codes times a power of two -> 8 BF16 values (exact for both formats, down to BF16's subnormals).
template <int F>
__device__ __forceinline__ v8bf16 codes_to_bf16(uint32_t lo, uint32_t hi, float f = 1.0f) {
    v2bf16 p[4];
    if constexpr (F == kE4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, f, true);
    }
    return v8bf16{p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
}

// Where LDS row rho of a wave's TN rows of b lies among its TN columns of y. An FP8 MFMA's result
// gives a lane rows 4 q + i of every 16; in this order two fragments make 8 neighbouring columns, so
// a lane stores 16 bytes at a time and four lanes 64. (BF16 MFMAs run with a first: a lane has one
// column, and the natural order stores whole lines.)
template <bool EXACT>
__device__ __forceinline__ int column_of(int rho) {
    if constexpr (EXACT) return rho;
    else return (rho & ~31) + 8 * ((rho >> 2) & 3) + 4 * ((rho >> 4) & 1) + (rho & 3);
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

// Tiles are counted in 32 bits (a grid has no more): a 64-bit division costs a wave near a thousand cycles.
//
// Contiguous ranges of tiles for each of the 8 XCDs (workgroups are dealt to them in turn), so that
// tiles that share operands share an L2. -1: no tile.
__device__ __forceinline__ int xcd_order(uint32_t id, uint32_t total) {
    const uint32_t x = id & 7, i = id >> 3, q = total >> 3, r = total & 7;
    if (i >= q + (x < r ? 1 : 0)) return -1;
    return (int)(x * q + (x < r ? x : r) + i);
}

// Tile number t of tm x tn tiles, in panels of PANEL tile rows: neighbours share both operands.
template <uint32_t PANEL>
__device__ __forceinline__ void panel_order(uint32_t t, uint32_t tm, uint32_t tn, uint32_t &im, uint32_t &in) {
    const uint32_t per = PANEL * tn, p = t / per, r = t - p * per;
    const uint32_t left = tm - p * PANEL;
    if (left >= PANEL) {
        im = p * PANEL + r % PANEL;
        in = r / PANEL;
    } else {
        in = r / left;
        im = p * PANEL + r - in * left;
    }
}

// Row tiles of every expert, found by each wave from the offsets: expert e owns rows
// [offsets[e], offsets[e+1]) and ceil(rows / bm) tiles; the rows before the first expert and after the last
// are two more stretches, of zeros. order(total) maps the number of row tiles to the one whose place is
// wanted, < 0: none.
template <typename Order>
__device__ __forceinline__ bool find_row_tile(const int32_t *offsets, int experts, int64_t nrows, int bm, Order order,
                                              TilePlace &pl) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = 0;
    const int64_t start = offsets[0] < 0 ? 0 : offsets[0] > nrows ? nrows : offsets[0];
    const int lead = (int)((uint32_t)(start + bm - 1) / (uint32_t)bm);   // tiles before the first expert
    int c = 0, first = 0, total = lead;
    auto stretch = [&](int e0) {                         // those of 64 experts, a lane each
        const int e = e0 + lane;
        lo = hi = 0;
        if (e < experts) {
            lo = offsets[e];
            hi = offsets[e + 1];
        } else if (e == experts) {
            lo = offsets[experts];
            hi = nrows;
        }
        lo = lo < 0 ? 0 : lo > nrows ? nrows : lo;
        hi = hi < lo ? lo : hi > nrows ? nrows : hi;
        c = (int)((uint32_t)(hi - lo + bm - 1) / (uint32_t)bm);
        int inc = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(inc, d);
            inc += lane >= d ? v : 0;
        }
        first = total + inc - c;
        total += __builtin_amdgcn_readlane(inc, 63);
    };
    for (int e0 = 0; e0 <= experts; e0 += 64) stretch(e0);
    const int want = order((uint32_t)total);
    if (want < 0) return false;
    if (want < lead) {
        pl.row0 = (int64_t)want * bm;
        pl.rows = start - pl.row0 < bm ? (int)(start - pl.row0) : bm;
        pl.expert = -1;
        return true;
    }
    const bool again = experts >= 64;                    // the lanes hold the last stretch of several
    total = lead;
    for (int e0 = 0;; e0 += 64) {
        if (again) stretch(e0);
        const uint64_t hit = __ballot(want >= first && want < first + c);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int64_t r0 = lo + (int64_t)(want - first) * bm;
            const int64_t left = hi - r0;
            pl.row0 = (int64_t)uniform64((uint64_t)__shfl((long long)r0, src));
            pl.rows = __builtin_amdgcn_readfirstlane(__shfl((int)(left < bm ? left : bm), src));
            pl.expert = e0 + src < experts ? e0 + src : -1;
            return true;
        }
        if (e0 + 64 > experts) return false;             // not reached: want is below the total
    }
}

// RUN neighbouring columns of one row, rounded once to BF16 or stored as FP32. Rows need no alignment:
// 16-byte stores may start at any element.
template <int RUN>
__device__ __forceinline__ void store_run(const MatmulArgs &p, const TilePlace &pl, int64_t row, int n, const float *v) {
    const int64_t plane = p.mode == kMatmulExpertsK ? pl.expert : pl.split;
    const int64_t at = (plane * p.m + row) * p.n + n;
    if (p.out_bf16) {
        uint16_t *y = (uint16_t *)p.y + at;
        uint32_t w[RUN / 2];
#pragma unroll
        for (int e = 0; e < RUN; e += 2) w[e / 2] = pack_bf16(v[e], v[e + 1]);
        if (n + RUN <= p.n) {
            __builtin_memcpy(y, w, sizeof(w));
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (n + e < p.n) y[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
    } else {
        float *y = (float *)p.y + at;
        if (n + RUN <= p.n) {
            __builtin_memcpy(y, v, RUN * sizeof(float));
        } else {
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (n + e < p.n) y[e] = v[e];
        }
    }
}

// The tile of this workgroup; false: there is none.
__device__ __forceinline__ bool place_tile(const MatmulArgs &p, int bm, int bn, TilePlace &pl) {
    pl.split = 0;
    pl.expert = 0;
    const uint32_t tn = (uint32_t)(p.n + bn - 1) / (uint32_t)bn;
    uint32_t im, in;
    if (p.mode == kMatmulExperts) {
        // all columns of up to 4 row tiles, then the next ones: the row tiles of one expert run together
        const bool found = find_row_tile(p.offsets, p.experts, p.m, bm, [&](uint32_t tiles_m) {
            const int id = xcd_order(blockIdx.x, tiles_m * tn);
            if (id < 0) return -1;
            panel_order<4>((uint32_t)id, tiles_m, tn, im, in);
            return (int)im;
        }, pl);
        if (!found) return false;
        pl.n0 = (int)in * bn;
        pl.k0 = 0;
        pl.k1 = p.k;
    } else {
        const uint32_t tm = (uint32_t)((p.m + bm - 1) / bm), per = tm * tn;
        uint32_t part = 0, t;
        if (p.mode == kMatmulExpertsK) {
            // Experts have unequal ranges of k: each expert's tiles go to all 8 XCDs, in ranges of q (with
            // whole experts for an XCD the CUs stood idle for 38% of the time at 32 experts).
            const uint32_t q = (per + 7) >> 3, i = blockIdx.x >> 3;
            part = i / q;
            t = ((blockIdx.x + part) & 7) * q + i - part * q;
            if (t >= per) return false;
        } else {
            const int id = xcd_order(blockIdx.x, per * (uint32_t)p.splits);
            if (id < 0) return false;
            t = (uint32_t)id;
            if (p.splits > 1) {
                part = t / per;
                t -= part * per;
            }
        }
        // measured with panels of 8 / 4: the experts' two gradients 1310 / 1276 us, dense products within 1%
        if (p.mode == kMatmulExpertsK) panel_order<4>(t, tm, tn, im, in);
        else panel_order<8>(t, tm, tn, im, in);
        pl.row0 = (int64_t)im * bm;
        pl.rows = (int)(p.m - pl.row0 < bm ? p.m - pl.row0 : bm);
        pl.n0 = (int)in * bn;
        if (p.mode == kMatmulExpertsK) {
            pl.expert = (int)part;
            int64_t lo = p.offsets[part], hi = p.offsets[part + 1];
            lo = lo < 0 ? 0 : lo > p.k ? p.k : lo & ~(int64_t)(kBK - 1);
            hi = hi < lo ? lo : hi > p.k ? p.k : hi;
            pl.k0 = lo;
            pl.k1 = hi;
        } else {
            pl.split = (int)part;
            pl.k0 = (int64_t)part * p.split_k;
            pl.k1 = pl.k0 + p.split_k < p.k ? pl.k0 + p.split_k : p.k;
        }
    }
    return true;
}

// The row of a that row r of the tile reads; rows past the end repeat the last one, and a row that
// names no row of a reads row 0 (its result is not stored).
__device__ __forceinline__ int64_t source_row(const MatmulArgs &p, const TilePlace &pl, int r) {
    r = r < pl.rows ? r : pl.rows - 1;
    if (!p.rows) return pl.row0 + r;
    const int64_t v = p.rows[pl.row0 + r];
    return v < 0 || v >= p.a_rows ? 0 : v;
}

// Addresses of a tile's operand loads: piece i of a thread is 16 bytes; the buffers move along k.
template <int KIND, bool EXACT, int BM, int BN, int TN, int NT>
struct TileLoads {
    static constexpr int LA = BM * kBK / 16 / NT, LB = BN * kBK / 16 / NT;
    MovingBuffer ba;
    MovingBufferOf<KIND == kKN> bb;
    uint32_t va[LA], vb[LB], stepb;

    __device__ __forceinline__ void init(const MatmulArgs &p, const TilePlace &pl, int steps, int t) {
        const bool gather = p.rows != nullptr;
        if (gather) {
            ba.base = uniform64((uint64_t)(uintptr_t)p.a);
            ba.left = (uint32_t)(p.a_rows * p.k);
        } else {
            ba.base = uniform64((uint64_t)(uintptr_t)p.a + (uint64_t)(pl.row0 * p.k + pl.k0));
            ba.left = cap31((p.m - pl.row0) * p.k - pl.k0);
        }
        ba.left = __builtin_amdgcn_readfirstlane((int)ba.left);
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int id = i * NT + t, row = id >> 3, ch = (id & 7) ^ swizzle(row);
            va[i] = steps ? (uint32_t)((source_row(p, pl, row) - (gather ? 0 : pl.row0)) * p.k) + 16u * ch : 0u;
        }
        const uint64_t bmat = (uint64_t)(p.mode == kMatmulExperts && pl.expert > 0 ? pl.expert : 0) * (uint64_t)p.n * (uint64_t)p.k;
        if constexpr (KIND == kKN) {
            bb.base = uniform64((uint64_t)(uintptr_t)p.b + bmat + (uint64_t)(pl.k0 * p.n + pl.n0));
            bb.left = uniform64((uint64_t)((p.k - pl.k0) * p.n - pl.n0));
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
                const int id = i * NT + t, row = id >> 3, ch = (id & 7) ^ swizzle(row);
                int n = column_of<EXACT>(row);
                n = n < p.n - pl.n0 ? n : p.n - pl.n0 - 1;
                vb[i] = (uint32_t)n * (uint32_t)p.k + 16u * ch;
            }
            bb.left = __builtin_amdgcn_readfirstlane((int)bb.left);
        }
        stepb = KIND == kKN ? (uint32_t)kBK * (uint32_t)p.n : (uint32_t)kBK;
    }
};

// Row `row` of the output takes no values: its entry in rows names no row of a.
__device__ __forceinline__ bool no_source(const MatmulArgs &p, int64_t row) {
    if (!p.rows) return false;
    const int64_t src = p.rows[row];
    return src < 0 || src >= p.a_rows;
}

// Results of fp32 sums go through LDS to whole rows of BN columns: a store of 16 bytes a lane covers 1 KiB of
// memory, one of 4 bytes 256 bytes in the same time. Lane: column lane % 32, rows 8 q + 4 (lane / 32) + e of a
// 32 x 32 fragment; rows 4-7 of 8 hold columns c ^ 32, so that both halves of a wave write all banks. buf: the
// operand tiles, which every wave has left.
template <int BM, int BN, int TM, int TN, int NT, typename V, int FM, int FN>
__device__ __forceinline__ void store_rows(const MatmulArgs &p, const TilePlace &pl, float *buf, int wm, int wn,
                                           int t, const V (&acc)[FM][FN]) {
    const int lane = t & 63, r32 = lane & 31, h = lane >> 5;
    phase_end();
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = wm * TM + 32 * i + 8 * (e >> 2) + 4 * h + (e & 3), c = wn * TN + 32 * j + r32;
                buf[r * BN + (c ^ (h << 5))] = acc[i][j][e];
            }
    phase_end();
    constexpr int CH = BN / 4, U = BM * CH / NT;         // 16-byte pieces of a row; those of a thread
    const int64_t plane = p.mode == kMatmulExpertsK ? pl.expert : pl.split;
    const int r0 = t / CH, c = 4 * (t % CH), n = pl.n0 + c;
    const int64_t first = (plane * p.m + pl.row0 + r0) * p.n + n, pitch = (int64_t)(NT / CH) * p.n;
    typedef float any4 __attribute__((ext_vector_type(4), aligned(4)));     // rows need no alignment
    static_assert(NT / CH % 8 == 0, "the rows of a thread hold their columns in the same order");
    const float *src = buf + r0 * BN + (c ^ (((r0 >> 2) & 1) << 5));
    if (p.out_bf16) {
        uint16_t *y = (uint16_t *)p.y + first;
#pragma unroll 4
        for (int u = 0; u < U; ++u, y += pitch) {
            const int r = u * (NT / CH) + r0;
            if (r >= pl.rows || n >= p.n) continue;
            const v4f32 v = *(const v4f32 *)(src + u * (NT / CH) * BN);
            const bool zero = no_source(p, pl.row0 + r);
            const uint32_t w[2] = {zero ? 0u : pack_bf16(v[0], v[1]), zero ? 0u : pack_bf16(v[2], v[3])};
            if (n + 4 <= p.n) {
                __builtin_memcpy(y, w, sizeof(w));
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (n + e < p.n) y[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            }
        }
        return;
    }
    float *y = (float *)p.y + first;
    if (pl.rows == BM && pl.n0 + BN <= p.n && !p.rows) {
#pragma unroll
        for (int u = 0; u < U; ++u, y += pitch)
            __builtin_nontemporal_store((any4)*(const v4f32 *)(src + u * (NT / CH) * BN), (any4 *)y);
        return;
    }
#pragma unroll 1
    for (int u = 0; u < U; ++u, y += pitch) {
        const int r = u * (NT / CH) + r0;
        if (r >= pl.rows || n >= p.n) continue;
        v4f32 v = *(const v4f32 *)(src + u * (NT / CH) * BN);
        if (no_source(p, pl.row0 + r)) v = (v4f32)0.0f;
        if (n + 4 <= p.n) {
            __builtin_nontemporal_store((any4)v, (any4 *)y);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < p.n) y[e] = v[e];
        }
    }
}

// Stores a wave's TM x TN values of an FP8 product. Lane: row lane % 16.
template <int KIND, int TM, int TN, typename V, int FM, int FN>
__device__ __forceinline__ void store_tile(const MatmulArgs &p, const TilePlace &pl, int wm, int wn, int lane,
                                           const V (&acc)[FM][FN]) {
    const int g = lane >> 4;
    constexpr int RUN = KIND == kKN || FN == 1 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = wm * TM + 16 * i + (lane & 15);
        if (r >= pl.rows) continue;
        const int64_t row = pl.row0 + r;
        const bool zero = no_source(p, row);
#pragma unroll
        for (int u = 0; u < 4 * FN / RUN; ++u) {
            float v[RUN];
#pragma unroll
            for (int e = 0; e < RUN; ++e) v[e] = zero ? 0.0f : acc[i][u * (RUN / 4) + e / 4][e % 4];
            store_run<RUN>(p, pl, row, pl.n0 + wn * TN + 4 * RUN * u + RUN * g, v);
        }
    }
}

// Scales of a tile for one group of k: thread u < BA loads that of a's row u, u >= BA one of b's, of its
// LDS row u - BA (groups) or of block (u - BA) % BLOCKS. A wave uses one buffer.
template <int KIND, bool EXACT, int BM, int BN, int NT>
struct ScaleLoads {
    static constexpr int BA = BM < 64 ? 64 : BM, BLOCKS = (BN + 127) / 128;
    static_assert(KIND == kGroups ? BA + BN <= NT : BA < NT, "one scale per thread");
    MovingBuffer buf;
    uint32_t off, step;

    __device__ __forceinline__ void init(const MatmulArgs &p, const TilePlace &pl, int t, int wave, int gk, int g0) {
        const int gn = (p.n + 127) / 128, e = pl.expert > 0 ? pl.expert : 0;
        step = 4;
        if (wave < BA / 64) {
            const int64_t first = p.rows ? 0 : pl.row0;
            buf.base = uniform64((uint64_t)(uintptr_t)(p.sa + first * gk + g0));
            const int64_t left = ((p.rows ? p.a_rows : p.m) - first) * gk - g0;
            buf.left = left > 0x3FFFFFFF ? 0xFFFFFFFCu : (uint32_t)left * 4u;
            off = (uint32_t)((source_row(p, pl, t) - first) * gk * 4);
        } else if constexpr (KIND == kGroups) {
            buf.base = uniform64((uint64_t)(uintptr_t)(p.sb + (int64_t)pl.n0 * gk + g0));
            buf.left = cap31(((int64_t)(p.n - pl.n0) * gk - g0) * 4);
            int n = column_of<EXACT>(t - BA);
            n = n < p.n - pl.n0 ? n : p.n - pl.n0 - 1;
            off = (uint32_t)n * (uint32_t)gk * 4u;
        } else {
            const int v = (t - BA) % BLOCKS, nb = v < gn - pl.n0 / 128 ? v : 0;
            if constexpr (KIND == kNK) {
                buf.base = uniform64((uint64_t)(uintptr_t)(p.sb + ((int64_t)e * gn + pl.n0 / 128) * gk + g0));
                buf.left = cap31(((int64_t)(gn - pl.n0 / 128) * gk - g0) * 4);
                off = (uint32_t)nb * (uint32_t)gk * 4u;
            } else {                                     // scales [k/128][n/128]
                buf.base = uniform64((uint64_t)(uintptr_t)(p.sb + ((int64_t)e * gk + g0) * gn + pl.n0 / 128));
                buf.left = cap31(((int64_t)(gk - g0) * gn - pl.n0 / 128) * 4);
                off = (uint32_t)nb * 4u;
                step = (uint32_t)gn * 4u;
            }
        }
        buf.left = __builtin_amdgcn_readfirstlane((int)buf.left);
    }
};

// ---- the tiled kernel ---------------------------------------------------------------------------

// BM x BN outputs per workgroup, WM x WN waves. Operand tiles of 128 bytes of k go straight from
// memory to LDS into a ring of D stages: the loads of step s + D - 1 are issued under the products of
// step s and waited for by count, with one barrier a step. Two workgroups share a CU and fill each
// other's waits. At one a CU (1024 x 4096 x 4096 in 128 x 128 tiles, 33 us) a step of 0.85 us holds 0.25
// us of products; a ring of 4 or 6 stages, twice the waves, or reading the next step's fragments a step
// ahead gave nothing or lost up to 14%.
//
// LDS tiles of rows along k (a, and b unless KN): 128-byte rows of eight 16-byte chunks, chunk c of
// row r at position c ^ swizzle(r). The lanes of the load fetch the permuted chunk, which stays
// inside the same 128 bytes of memory.
// KN: b's tile keeps k as rows of BN bytes (chunk c of row k at c ^ (k & 7)) and the transposing
// LDS read hands each lane 8 codes along k of one column.
// Scales come one step ahead of their codes, as they are; each thread inverts one of them.
template <int FA, int FB, int KIND, int MATH, int BM, int BN, int WM, int WN, int D>
__global__ __launch_bounds__(64 * WM * WN, 2) void matmul_tile_kernel(MatmulArgs p) {
    constexpr int NT = 64 * WM * WN, TM = BM / WM, TN = BN / WN;
    constexpr bool POW2 = MATH == kMathE8m0, EXACT = MATH >= kMathExact;
    constexpr int FR = EXACT ? 32 : 16, FM = TM / FR, FN = TN / FR;      // fragments
    constexpr int kA = BM * kBK, kB = BN * kBK, kStage = kA + kB;
    typedef TileLoads<KIND, EXACT, BM, BN, TN, NT> Loads;
    typedef ScaleLoads<KIND, EXACT, BM, BN, NT> Scales;
    constexpr int LA = Loads::LA, LB = Loads::LB, LT = LA + LB, BA = Scales::BA;
    static_assert(LA * NT * 16 == kA && LB * NT * 16 == kB && (!EXACT || BM * BN * 4 <= D * kStage), "tile and workgroup do not match");
    __shared__ __attribute__((aligned(1024))) uint8_t tiles[D][kStage];
    __shared__ __attribute__((aligned(256))) float raw[D][NT];
    __shared__ __attribute__((aligned(16))) float inv[2][NT];

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, g = lane >> 4;

    TilePlace pl;
    if (!place_tile(p, BM, BN, pl)) return;
    const int steps = pl.expert < 0 || pl.k1 <= pl.k0 ? 0 : (int)((pl.k1 - pl.k0 + kBK - 1) / kBK);
    const int kend = (int)(pl.k1 - pl.k0);
    const int gk = (int)((p.k + kBK - 1) / kBK), g0 = (int)(pl.k0 / kBK);

    constexpr int FV = FR * FR / 64;                     // values of a fragment in a lane
    typedef float frag __attribute__((ext_vector_type(FV)));
    frag acc[FM][FN];
    // FOLD: the scales go into the operands. Seldom a scale is too far from 1 for that; the tile is then done again
    // without. (A choice at each step costs all that folding gains: 525 us for 7168 x 4096 x 8192 in FP32, as without
    // folding, against 465.)
    bool far = false;
    auto all_steps = [&](auto folded) QF8_INLINE {
        constexpr bool FOLD = decltype(folded)::value;
        Loads ld;
        ld.init(p, pl, steps, t);
        Scales ls;
        if (steps) ls.init(p, pl, t, wave, gk, g0);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = (frag)0.0f;

        // The loads of step n_load: piece u of LA + LB, then the scales of step n_load + 1. Past the last
        // step the buffers have length 0: the loads still run, so that counts hold, and leave zeros nobody uses.
        const uint32_t lds0 = __builtin_amdgcn_readfirstlane((int)lds_address(&tiles[0][0])) + (uint32_t)wave * 1024u;
        const uint32_t lds_raw = __builtin_amdgcn_readfirstlane((int)lds_address(&raw[0][0])) + (uint32_t)wave * 256u;
        int n_load = 0, n_scale = 0, at_load = 0, at_scale = 0;              // steps, and their places in the rings
        auto load_scale = [&]() {
            if (n_scale >= steps) ls.buf.left = 0;
            lds_dma4(ls.buf.rsrc(), ls.off, lds_raw + (uint32_t)at_scale * NT * 4u);
            ls.buf.advance(ls.step);
            ++n_scale;
            at_scale = at_scale + 1 == D ? 0 : at_scale + 1;
        };
        auto load_piece = [&](int u) {
            const uint32_t at = lds0 + (uint32_t)at_load * kStage;
            if (u == 0 && n_load >= steps) ld.ba.left = ld.bb.left = 0;
            if (u < LA) lds_dma16(ld.ba.rsrc(), ld.va[u < LA ? u : 0], at + (uint32_t)u * NT * 16u);
            else if (u < LT) lds_dma16(ld.bb.rsrc(), ld.vb[u < LA ? 0 : u - LA], at + kA + (uint32_t)(u - LA) * NT * 16u);
            if (u == LT) {
                ld.ba.advance(kBK);
                ld.bb.advance(ld.stepb);
                load_scale();
                ++n_load;
                at_load = at_load + 1 == D ? 0 : at_load + 1;
            }
        };

        if (steps) {
            load_scale();
#pragma unroll
            for (int d = 0; d < D - 1; ++d)
#pragma unroll
                for (int u = 0; u <= LT; ++u) load_piece(u);
            wait_vmem_but<(D - 1) * (LT + 1)>();
            phase_end();
            const float f = inverse_scale<MATH>(raw[0][t]);
            if constexpr (EXACT && FOLD) far = !near_one(f);
            inv[0][t] = f;
        }
        int at = 0;                                          // stage of step s
        for (int s = 0; s < steps; ++s) {
            wait_vmem_but<(D - 2) * (LT + 1)>();
            phase_end();
            uint8_t *const ta = tiles[at], *const tb = ta + kA;
            const float *const sc = inv[s & 1];
            at = at + 1 == D ? 0 : at + 1;
            const int krem = kend - s * kBK;
            if (krem < kBK) {                               // the last step of a k that is no multiple of 128
#pragma unroll
                for (int i = 0; i < LA; ++i) {
                    const int id = i * NT + t, row = id >> 3, ch = (id & 7) ^ swizzle(row);
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
                        const int row = id >> 3, ch = (id & 7) ^ swizzle(row);
                        if (16 * ch + 16 > krem) *at = keep_bytes(*at, krem - 16 * ch);
                    }
                }
                phase_end();
            }
            float next;                                      // scale of the next step, inverted after the products
            if constexpr (EXACT) {
                // lane (r32, h): row r32 of a fragment; slice u of 16 k holds, for half h, the 8 codes at
                // k = 16 (2 (u / 2) + h) + 8 (u % 2). a comes first, so that a lane ends with one column.
                const int r32 = lane & 31, h = lane >> 5;
                // Folded, a lane's row of each operand carries its own factor.
                float ea[FM], eb[FN];
#pragma unroll
                for (int i = 0; i < FM; ++i) ea[i] = FOLD ? sc[wm * TM + 32 * i + r32] : 1.0f;
#pragma unroll
                for (int j = 0; j < FN; ++j) eb[j] = FOLD ? sc[BA + (KIND == kGroups ? wn * TN + 32 * j + r32 : wn * TN / 128)] : 1.0f;
                v8bf16 fb[FN][8];
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (KIND == kKN) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int kr = 16 * (2 * (u >> 1) + h) + 8 * (u & 1) + (r16 >> 1);
                            const int ch = (wn * TN + 32 * j) / 16 + ((lane >> 4) & 1);
                            const v2i32 q = read_transposed(tb + kr * BN + ((ch ^ (kr & 7)) << 4) + 8 * (r16 & 1));
                            fb[j][u] = codes_to_bf16<FB>((uint32_t)q.x, (uint32_t)q.y, eb[j]);
                        }
                    } else {
                        const int row = wn * TN + 32 * j + r32;
#pragma unroll
                        for (int u = 0; u < 8; u += 2) {
                            const uint4 q = *(const uint4 *)(tb + row * kBK + (((u + h) ^ swizzle(row)) << 4));
                            fb[j][u] = codes_to_bf16<FB>(q.x, q.y, eb[j]);
                            fb[j][u + 1] = codes_to_bf16<FB>(q.z, q.w, eb[j]);
                        }
                    }
                }
                next = raw[at][t];
#pragma unroll
                for (int u = 0; u <= LT; ++u) load_piece(u);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int row = wm * TM + 32 * i + r32;
                    v16f32 part[FN];
#pragma unroll
                    for (int j = 0; j < FN; ++j) part[j] = FOLD ? (v16f32)acc[i][j] : (v16f32)0.0f;
#pragma unroll
                    for (int u = 0; u < 8; u += 2) {
                        const uint4 q = *(const uint4 *)(ta + row * kBK + (((u + h) ^ swizzle(row)) << 4));
                        const v8bf16 f0 = codes_to_bf16<FA>(q.x, q.y, ea[i]), f1 = codes_to_bf16<FA>(q.z, q.w, ea[i]);
#pragma unroll
                        for (int j = 0; j < FN; ++j) part[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f0, fb[j][u], part[j], 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < FN; ++j) part[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f1, fb[j][u + 1], part[j], 0, 0, 0);
                    }
                    if constexpr (FOLD) {
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[i][j] = part[j];
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            v4f32 sa = *(const v4f32 *)(sc + wm * TM + 32 * i + 8 * q + 4 * h);
                            if constexpr (KIND != kGroups) sa *= sc[BA + wn * TN / 128];
#pragma unroll
                            for (int j = 0; j < FN; ++j) {
                                v4f32 f = sa;
                                if constexpr (KIND == kGroups) f *= sc[BA + wn * TN + 32 * j + r32];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[i][j][4 * q + e] = __builtin_fmaf(part[j][4 * q + e], f[e], acc[i][j][4 * q + e]);
                            }
                        }
                    }
                }
                // conversions and scaling run in the shadow of the products: 8 vector instructions a product
#pragma unroll
                for (int m = 0; m < FM * FN * 8; ++m) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, FOLD ? 5 : 9, 0);
                }
            } else {
                // lane (r16, g) holds row r16 of a fragment and k = 16 g + [0, 16) and 64 + 16 g + [0, 16).
                // Products of fragment i run while the fragments of i + 1 are read and the sums of i - 1
                // are scaled; the next step's loads are issued in between, a few at a time, so that no
                // wave stands in a full load queue while the matrix core idles.
                const uint32_t swz = (uint32_t)((g ^ swizzle(r16)) << 4);
                const uint8_t *const pa = ta + (wm * TM + r16) * kBK;
                auto frag_a = [&](int i) {
                    return join16(*(const uint4 *)(pa + i * 16 * kBK + swz), *(const uint4 *)(pa + i * 16 * kBK + (swz ^ 64u)));
                };
                v8i32 fb[FN];
                v8i32 fa = frag_a(0);
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (KIND == kKN) {
                        v2i32 q[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            // 16 lanes read 8 rows of k x 16 columns; two neighbouring lanes cover a row
                            const int kr = (h >> 1) * 64 + 16 * g + 8 * (h & 1) + (r16 >> 1);
                            const int ch = (wn * TN + 16 * j) / 16;
                            q[h] = read_transposed(tb + kr * BN + ((ch ^ (kr & 7)) << 4) + 8 * (r16 & 1));
                        }
                        fb[j] = v8i32{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
                    } else {
                        const uint8_t *src = tb + (wn * TN + r16) * kBK + j * 16 * kBK;
                        fb[j] = join16(*(const uint4 *)(src + swz), *(const uint4 *)(src + (swz ^ 64u)));
                    }
                }
                v4f32 sbg[FN];
                int ebg[FN];
                float sa[FM];
#pragma unroll
                for (int i = 0; i < FM; ++i) sa[i] = sc[wm * TM + 16 * i + r16];
                if constexpr (KIND == kGroups) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        if constexpr (POW2) ebg[j] = __float_as_int(sc[BA + wn * TN + 16 * j + r16]);
                        else sbg[j] = *(const v4f32 *)(sc + BA + wn * TN + 16 * j + 4 * g);
                    }
                } else {
                    const float sbu = sc[BA + wn * TN / 128];
                    if constexpr (POW2) {
#pragma unroll
                        for (int j = 0; j < FN; ++j) ebg[j] = __float_as_int(sbu);
                    } else {
#pragma unroll
                        for (int i = 0; i < FM; ++i) sa[i] *= sbu;
                    }
                }
                next = raw[at][t];
                v4f32 part[2][FN];
                auto scale = [&](int i) {                   // acc += part * (1/Sa 1/Sb)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // the factor first: part times one far scale alone could leave the range
                            if constexpr (KIND == kGroups) acc[i][j][e] = __builtin_fmaf(part[i & 1][j][e], sa[i] * sbg[j][e], acc[i][j][e]);
                            else acc[i][j][e] = __builtin_fmaf(part[i & 1][j][e], sa[i], acc[i][j][e]);
                        }
                };
                constexpr int PI = (LT + FM) / FM;          // load pieces issued per fragment
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    v8i32 next;
                    if (i + 1 < FM) next = frag_a(i + 1);
#pragma unroll
                    for (int u = i * PI; u < (i + 1) * PI && u <= LT; ++u) load_piece(u);
                    if constexpr (POW2) {
#pragma unroll
                        for (int j = 0; j < FN; ++j) {
                            acc[i][j] = mfma_e8m0<FA, FB>(fb[j], fa, acc[i][j], ebg[j], __float_as_int(sa[i]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < FN; ++j) part[i & 1][j] = mfma_raw<FA, FB>(fb[j], fa, v4f32{0.0f, 0.0f, 0.0f, 0.0f});
                        if (i > 0) scale(i - 1);
                    }
                    if (i + 1 < FM) fa = next;
                }
                if constexpr (!POW2) scale(FM - 1);
            }
            asm volatile("" : "+v"(next));
            const float f = inverse_scale<MATH>(next);
            if constexpr (EXACT && FOLD) far = far || (s + 1 < steps && !near_one(f));
            inv[(s + 1) & 1][t] = f;
        }
        wait_vmem();                                        // no load may still write LDS when the workgroup ends
    };
    all_steps(std::integral_constant<bool, MATH == kMathExactPow2>());
    if constexpr (MATH == kMathExactPow2) {
        phase_end();                                    // every wave has left the last step
        raw[0][t] = far ? 1.0f : 0.0f;
        phase_end();
        bool any = false;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) any = any || raw[0][64 * w + lane] != 0.0f;
        if (__any(any)) {
            phase_end();
            all_steps(std::false_type());
        }
    }

    if constexpr (EXACT) store_rows<BM, BN, TM, TN, NT>(p, pl, (float *)&tiles[0][0], wm, wn, t, acc);
    else store_tile<KIND, TM, TN>(p, pl, wm, wn, lane, acc);
}

// ---- the large tile in two alternating groups of waves --------------------------------------------
//
// 256 x 256 outputs, 8 waves of 128 x 64, two on each SIMD: wave w and w + 4. A step of k is four
// phases with a barrier after each, and the second four waves run one phase behind the first:
//
//   P0  read b's fragments and a's first half from LDS      P1  16 MFMAs a wave and their scaling
//   P2  read a's second half                                 P3  16 MFMAs a wave and their scaling
//
// so on every SIMD one wave feeds the matrix core while the other reads. In the plain form of the
// tile both waves of a SIMD wait for the same barrier and the same reads: the matrix core was busy
// 40% of the time on 8192 x 7168 x 18432 (1143 us). Now a pass takes 1052 us, 2.06 PFLOP/s; counted in a
// slower run (1150 us at 1.90 GHz) it was busy 47%, which is 52% of 1052 us at that clock. A phase takes
// 910 cycles, 770 with exponents in place of the FMAs, for 512 of products. Without its loads it takes 705
// and 585, with loads that always hit L2 801 and 613, but at 1.6-1.7 GHz for 1.8-1.9: the card is at its
// power limit, so cycles saved come back as time by half only.
// Loads go to LDS between the products, as soon as a region is free in both groups (the second group reads
// what the first read one phase before):
//   P1 of step s  a's second halves of step s + 1 (2 loads a wave), where those of s - 1 were: last read in
//                 the second group's P2 of s - 1, the first group's P3 of s - 1
//   P3 of step s  b and a's first halves of step s + 2 (6 loads), where those of s were: last read in the
//                 second group's P0 of s, the first group's P1 of s; and the scales of step s + 3 (1 load),
//                 where the same thread read those of s + 1 in P1
// They are waited for by count three phases after: the second halves of s in P0 of s (7 newer loads may be in
// flight), b and the first halves of s + 1 in P2 of s (2 newer, and the scales of s + 2 with them). A wave's
// wait is followed by its group's barrier, the other group's by the next one, and the first read comes two
// barriers after. P1 of step s inverts the scales of s + 1, one per thread; P0 of s + 1 reads them.
template <int FA, int FB, int KIND, int MATH>
__global__ __launch_bounds__(512, 2) void matmul_large_kernel(MatmulArgs p) {
    static_assert(KIND != kGroups && MATH < kMathExact, "one scale of b for each wave and step");
    constexpr int BM = 256, BN = 256, WN = 4, NT = 512, TM = 128, TN = 64, FM = 8, FN = 4;
    constexpr bool POW2 = MATH == kMathE8m0;
    constexpr int kA = BM * kBK, kB = BN * kBK, kStage = kA + kB;
    __shared__ __attribute__((aligned(1024))) uint8_t tiles[2][kStage];
    __shared__ __attribute__((aligned(256))) float raw[2][BM + BN];
    __shared__ __attribute__((aligned(16))) float inv[2][BM + BN];

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, g = lane >> 4;
    TilePlace pl;
    if (!place_tile(p, BM, BN, pl)) return;
    const int steps = pl.expert < 0 || pl.k1 <= pl.k0 ? 0 : (int)((pl.k1 - pl.k0 + kBK - 1) / kBK);
    const int kend = (int)(pl.k1 - pl.k0);
    const int gk = (int)((p.k + kBK - 1) / kBK), g0 = (int)(pl.k0 / kBK);

    v4f32 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};

    if (steps > 0) {
        TileLoads<KIND, false, BM, BN, TN, NT> ld;
        ld.init(p, pl, steps, t);
        ScaleLoads<KIND, false, BM, BN, NT> ls;
        ls.init(p, pl, t, wave, gk, g0);
        const uint32_t lds0 = __builtin_amdgcn_readfirstlane((int)lds_address(&tiles[0][0])) + (uint32_t)wave * 1024u;
        const uint32_t lds_raw = __builtin_amdgcn_readfirstlane((int)lds_address(&raw[0][0])) + (uint32_t)wave * 256u;

        // Each stream of loads has its own position along k; past the last step its buffer has length 0
        // and the loads leave zeros nobody uses.
        MovingBuffer first = ld.ba, second = ld.ba;
        auto cols = ld.bb;
        int n_first = 0, n_second = 0, n_scale = 0;
        auto load_first = [&](int u) QF8_INLINE {                  // piece u of 6: b and a's first halves of step n_first
            const uint32_t at = lds0 + (uint32_t)(n_first & 1) * kStage;
            if (u == 0 && n_first >= steps) first.left = cols.left = 0;
            if (u < 4) lds_dma16(cols.rsrc(), ld.vb[u], at + kA + (uint32_t)u * 8192u);
            else lds_dma16(first.rsrc(), ld.va[2 * (u - 4)], at + (uint32_t)(u - 4) * 2u * 8192u);
            if (u == 5) {
                first.advance(kBK);
                cols.advance(ld.stepb);
                ++n_first;
            }
        };
        auto load_second = [&](int u) QF8_INLINE {                 // piece u of 2: a's second halves of step n_second
            const uint32_t at = lds0 + (uint32_t)(n_second & 1) * kStage;
            if (u == 0 && n_second >= steps) second.left = 0;
            lds_dma16(second.rsrc(), ld.va[2 * u + 1], at + (2u * u + 1u) * 8192u);
            if (u == 1) {
                second.advance(kBK);
                ++n_second;
            }
        };
        auto load_scale = [&]() QF8_INLINE {
            if (n_scale >= steps) ls.buf.left = 0;
            lds_dma4(ls.buf.rsrc(), ls.off, lds_raw + (uint32_t)(n_scale & 1) * (BM + BN) * 4u);
            ls.buf.advance(ls.step);
            ++n_scale;
        };

        load_scale();
#pragma unroll
        for (int u = 0; u < 6; ++u) load_first(u);
        load_scale();
        load_second(0);
        load_second(1);
#pragma unroll
        for (int u = 0; u < 6; ++u) load_first(u);
        wait_vmem_but<6>();
        phase_end();
        inv[0][t] = inverse_scale<MATH>(raw[0][t]);
        phase_end();
        load_scale();                                   // into the place of the scales just read
        if (wave >= 4) phase_end();                     // one phase behind

        const uint32_t swz = (uint32_t)((g ^ swizzle(r16)) << 4);
        v8i32 fa[4], fb[FN];
        // Product m of a phase goes to part[m % 4] and is scaled three products later (the last three
        // in the next phase), when it is complete without a wait.
        v4f32 part[4] = {};
        float sa[4] = {}, late = 0.0f;
        int eb = 0;
        auto scale_one = [&](int i, int j, float f) QF8_INLINE {   // acc += part * (1/Sa 1/Sb)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[j][e], f, acc[i][j][e]);
            asm volatile("" : "+v"(acc[i][j]));         // here, not after a later branch: part is used again
        };
        // codes past k in the last step: chunk g holds k = 16 g + [0, 16) of a fragment, chunk g + 4 64 more
        auto trim = [&](v8i32 f, int krem) QF8_INLINE {
            asm volatile("" : "+s"(krem));              // keeps the masks inside the branch
            const uint4 lo = keep_bytes(make_uint4(f[0], f[1], f[2], f[3]), krem - 16 * g);
            const uint4 hi = keep_bytes(make_uint4(f[4], f[5], f[6], f[7]), krem - 64 - 16 * g);
            return join16(lo, hi);
        };
        auto read_a = [&](const uint8_t *ta, const float *sc, int half) QF8_INLINE {
            const uint8_t *src = ta + (wm * TM + half * 64 + r16) * kBK;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fa[i] = join16(*(const uint4 *)(src + i * 16 * kBK + swz), *(const uint4 *)(src + i * 16 * kBK + (swz ^ 64u)));
#pragma unroll
            for (int i = 0; i < 4; ++i) sa[i] = sc[wm * TM + half * 64 + 16 * i + r16];
            const float sbu = sc[BM + wn / 2];
            eb = __float_as_int(sbu);
            if constexpr (!POW2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sa[i] *= sbu;
                    asm volatile("" : "+v"(sa[i]));     // before the phase ends
                }
            }
        };
        // 16 products. Between them go the loads (a load of 1 KiB takes the path to LDS for 16 cycles:
        // issued in a row they would hold up the wave) and, in the first half, the next step's scales.
        auto between = [&](int half, int m, int s, float &next) QF8_INLINE {
            if (half == 0) {
                if (m == 4 || m == 8) load_second(m / 4 - 1);
                if (m == 5) asm volatile("" : "+v"(next));
                if (m == 11) inv[(s + 1) & 1][t] = inverse_scale<MATH>(next);
            } else {
                if (m % 2 == 0 && m / 2 < 6) load_first(m / 2);
                if (m == 12) load_scale();
            }
        };
        // TAIL, the last tile of some rows: halves of 64 rows past the last one take no products (half 1 then
        // only finishes half 0's scaling). The experts' products on 4096 x 8 rows 1357 -> 1306 us; in one
        // loop with the full tiles it cost those 1-2%.
        const bool left[2] = {wm * TM < pl.rows, wm * TM + 64 < pl.rows};
        auto products = [&](auto tail, int half, int s) QF8_INLINE {
            constexpr bool TAIL = decltype(tail)::value;
            __builtin_amdgcn_s_setprio(1);
            float next = 1.0f;
            if (half == 0) next = raw[(s + 1) & 1][t];
            if (!TAIL || left[half]) {
#pragma unroll
                for (int m = 0; m < 4 * FN; ++m) {
                    const int i = m / FN, j = m % FN, at = half * 4 + i;
                    if constexpr (POW2) {
                        acc[at][j] = mfma_e8m0<FA, FB>(fb[j], fa[i], acc[at][j], eb, __float_as_int(sa[i]));
                        asm volatile("" : "+v"(acc[at][j]));
                    } else {
                        part[j] = mfma_raw<FA, FB>(fb[j], fa[i], v4f32{0.0f, 0.0f, 0.0f, 0.0f});
                        __builtin_amdgcn_sched_barrier(0);
                        if (m < 3) scale_one((half * 4 + 7) % 8, m + 1, late);
                        else scale_one(half * 4 + (m - 3) / FN, (m - 3) % FN, sa[(m - 3) / FN]);
                    }
                    between(half, m, s, next);
                    __builtin_amdgcn_sched_barrier(0);
                }
                late = sa[3];
            } else {
#pragma unroll
                for (int m = 0; m < 4 * FN; ++m) between(half, m, s, next);
                if constexpr (!POW2) {
                    if (half == 1 && left[0]) {
#pragma unroll
                        for (int j = 1; j < FN; ++j) scale_one(3, j, late);
                    }
                }
            }
            __builtin_amdgcn_s_setprio(0);
        };

        auto all_steps = [&](auto tail) QF8_INLINE {
            constexpr bool TAIL = decltype(tail)::value;
            for (int s = 0; s < steps; ++s) {
                const uint8_t *const ta = tiles[s & 1], *const tb = ta + kA;
                const float *const sc = inv[s & 1];
                const int krem = kend - s * kBK;
                // P0
                if (!TAIL || left[0]) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        if constexpr (KIND == kKN) {
                            v2i32 q[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const int kr = (h >> 1) * 64 + 16 * g + 8 * (h & 1) + (r16 >> 1);
                                const int ch = (wn * TN + 16 * j) / 16;
                                q[h] = read_transposed(tb + kr * BN + ((ch ^ (kr & 7)) << 4) + 8 * (r16 & 1));
                            }
                            fb[j] = v8i32{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
                        } else {
                            const uint8_t *src = tb + (wn * TN + r16) * kBK + j * 16 * kBK;
                            fb[j] = join16(*(const uint4 *)(src + swz), *(const uint4 *)(src + (swz ^ 64u)));
                        }
                    }
                    read_a(ta, sc, 0);
                    if (krem < kBK) {
#pragma unroll
                        for (int j = 0; j < FN; ++j) fb[j] = trim(fb[j], krem);
#pragma unroll
                        for (int i = 0; i < 4; ++i) fa[i] = trim(fa[i], krem);
                    }
                }
                wait_vmem_but<7>();                         // a's second halves of this step
                phase_end();
                // P1
                products(tail, 0, s);
                phase_end();
                // P2
                if (!TAIL || left[1]) {
                    read_a(ta, sc, 1);
                    if (krem < kBK) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) fa[i] = trim(fa[i], krem);
                    }
                }
                wait_vmem_but<2>();                         // b and a's first halves of the next
                phase_end();
                // P3
                products(tail, 1, s);
                phase_end();
            }
        };
        if (pl.rows > BM - 64) all_steps(std::false_type());
        else all_steps(std::true_type());
        if constexpr (!POW2) {
#pragma unroll
            for (int j = 1; j < FN; ++j) scale_one(FM - 1, j, late);
        }
        if (wave < 4) phase_end();                      // the others are one phase behind
        wait_vmem();                                    // no load may still write LDS when the workgroup ends
    }
    store_tile<KIND, TM, TN>(p, pl, wm, wn, lane, acc);
}

// ---- launch ----------------------------------------------------------------------------------------

// Tile sizes. fit: workgroups that share a CU.
struct TileSize { int bm, bn, fit; };
constexpr int kTileCount = 4;
constexpr TileSize kTileSizes[kTileCount] = {{256, 256, 1}, {128, 128, 2}, {64, 128, 2}, {32, 128, 2}};

template <int FA, int FB, int KIND, int MATH>
int launch_matmul_tile(const MatmulArgs &p, int size, int64_t groups, hipStream_t s) {
    const dim3 grid((unsigned)groups);
#define QF8_TILE(BM, BN, WM, WN, D) \
    hipLaunchKernelGGL((matmul_tile_kernel<FA, FB, KIND, MATH, BM, BN, WM, WN, D>), grid, dim3(64 * WM * WN), 0, s, p)
    switch (size) {
        case 0:
            if constexpr (MATH >= kMathExact) return QF8_ERR_HIP;        // never planned
            else if constexpr (KIND == kGroups) QF8_TILE(256, 256, 2, 4, 2);
            else hipLaunchKernelGGL((matmul_large_kernel<FA, FB, KIND, MATH>), grid, dim3(512), 0, s, p);
            break;
        case 1: QF8_TILE(128, 128, 2, 2, 2); break;
        case 2: QF8_TILE(64, 128, 1, 4, 3); break;
        default: QF8_TILE(32, 128, 1, 4, 3); break;
    }
#undef QF8_TILE
    return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP;
}

template <int FA, int FB, int KIND>
int launch_matmul_kind(const MatmulArgs &p, int math, int size, int64_t groups, hipStream_t s) {
    if (math == kMathFp8) return launch_matmul_tile<FA, FB, KIND, kMathFp8>(p, size, groups, s);
    if (math == kMathE8m0) return launch_matmul_tile<FA, FB, KIND, kMathE8m0>(p, size, groups, s);
    if (math == kMathExact) return launch_matmul_tile<FA, FB, KIND, kMathExact>(p, size, groups, s);
    return launch_matmul_tile<FA, FB, KIND, kMathExactPow2>(p, size, groups, s);
}

template <int FA, int FB>
int launch_matmul_formats(const MatmulArgs &p, int kind, int math, int size, int64_t groups, hipStream_t s) {
    if (kind == kNK) return launch_matmul_kind<FA, FB, kNK>(p, math, size, groups, s);
    if (kind == kKN) return launch_matmul_kind<FA, FB, kKN>(p, math, size, groups, s);
    return launch_matmul_kind<FA, FB, kGroups>(p, math, size, groups, s);
}

}  // namespace qf8
