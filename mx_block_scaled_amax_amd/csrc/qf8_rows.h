// qf8_rows.h -- pieces of eight neighbouring values of a row, as the row-wise operators (norm, gated activation)
// hold them: loads and stores by type, sums over lanes, and the FP8 codes of 1x128 groups, sixteen lanes each.
#pragma once
#include "qf8_device.h"

namespace qf8 {

// Eight values: one 16-byte piece of BF16, two of FP32. CP: cache policy of BF16's.
template <typename T> struct Eight;
template <> struct Eight<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void stream(const uint16_t *p) { a = ld_stream((const uint4 *)p); }
    __device__ __forceinline__ void values(float *v) const {
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
    }
    static __device__ __forceinline__ uint32_t two(float x, float y) {
        v2bf16 v = {(__bf16)x, (__bf16)y};
        return __builtin_bit_cast(uint32_t, v);
    }
    __device__ __forceinline__ void round(const float *v) {
        a = make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7]));
    }
    template <int CP> __device__ __forceinline__ void from(__amdgpu_buffer_rsrc_t r, int col) { a = buf_load16<CP>(r, col * 2, 0); }
    template <int CP> __device__ __forceinline__ void to(__amdgpu_buffer_rsrc_t r, int col) const { buf_store16<CP>(r, col * 2, 0, a); }
    __device__ __forceinline__ void store_stream(uint16_t *p) const { st_stream((uint4 *)p, a); }
};
// Each of the two pieces fills half of its lines, so loads and stores are cached: non-temporal ones take a line twice. us,
// cached / not: gated activation of FP32 to FP32, 8192 x 2048, 36.7 / 43.0, its gradients 60.6 / 64.8, norm 8192 x 4096 with
// FP32 residual 65.3 / 67.2.
template <> struct Eight<float> {
    uint4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void stream(const float *p) { a = ((const uint4 *)p)[0]; b = ((const uint4 *)p)[1]; }
    __device__ __forceinline__ void values(float *v) const {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
    __device__ __forceinline__ void round(const float *v) {
        a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    }
    template <int CP> __device__ __forceinline__ void from(__amdgpu_buffer_rsrc_t r, int col) {
        a = buf_load16<kCached>(r, col * 4, 0);
        b = buf_load16<kCached>(r, col * 4 + 16, 0);
    }
    template <int CP> __device__ __forceinline__ void to(__amdgpu_buffer_rsrc_t r, int col) const {
        buf_store16<kCached>(r, col * 4, 0, a);
        buf_store16<kCached>(r, col * 4 + 16, 0, b);
    }
    __device__ __forceinline__ void store_stream(float *p) const { ((uint4 *)p)[0] = a; ((uint4 *)p)[1] = b; }
};

// A row of a tensor as a buffer: what lies behind its columns reads as zeros and is not written. No row: no columns.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void *base, int64_t row, int cols, bool there = true) {
    return make_rsrc((const T *)base + row * cols, there ? (uint32_t)cols * (uint32_t)sizeof(T) : 0u);
}

// Sum over the wave, the same bits in every lane (all lanes active): each step adds two partners' equal sums.
__device__ __forceinline__ float sum_wave(float v) {
    v += __uint_as_float(dpp_mov<0xB1>(__float_as_uint(v)));       // quad_perm [1,0,3,2]
    v += __uint_as_float(dpp_mov<0x4E>(__float_as_uint(v)));       // quad_perm [2,3,0,1]
    v += __uint_as_float(dpp_mov<0x141>(__float_as_uint(v)));      // row_half_mirror
    v += __uint_as_float(dpp_mov<0x140>(__float_as_uint(v)));      // row_mirror
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// |amax| bits of a 1x128 group: sixteen lanes of a DPP row, eight values each of those that have some. NaN sorts above every value.
__device__ __forceinline__ uint32_t group_amax(const float *y, bool there = true) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    return max_row16(there ? m : 0);
}
// Bits of the magnitudes that are Inf or NaN once rounded to T: BF16's Inf begins at 255.5 2^120.
template <typename T> constexpr uint32_t kNotFinite = sizeof(T) == 2 ? 0x7F7F8000u : 0x7F800000u;
// The group's scale and this lane's eight codes.
__device__ __forceinline__ float group_scale(uint32_t amax, int fmt, int pow2) {
    if (fmt == kE4M3) return pow2 ? scale_pow2_from_amax_bits<kE4M3>(amax) : scale_from_amax_bits<kE4M3>(amax);
    return pow2 ? scale_pow2_from_amax_bits<kE5M2>(amax) : scale_from_amax_bits<kE5M2>(amax);
}
__device__ __forceinline__ uint2 group_codes(const float *y, float s, int fmt) {
    if (fmt == kE4M3) return make_uint2(cast4<kE4M3>(y[0], y[1], y[2], y[3], s), cast4<kE4M3>(y[4], y[5], y[6], y[7], s));
    return make_uint2(cast4<kE5M2>(y[0], y[1], y[2], y[3], s), cast4<kE5M2>(y[4], y[5], y[6], y[7], s));
}

}  // namespace qf8
