// qf8_gate.hip -- the gated activation between an expert's two products, act(a) * b for a product's two halves
// [a | b], in FP8 codes with 1x128 scales; and the gradients of the halves.
//
//   y = act(a) b;   da = dy b act'(a),  db = dy act(a)
// Sixteen lanes hold a group, eight columns each. One pass over the data, HBM its bound (BF16, 32768 rows of 2 x 2048 to E4M3
// codes 57 us, 5.9 TB/s; the gradients of 16384 rows in E5M2 codes 45 us, 6.0 TB/s; a copy of 256 MB 5.5); the two
// transcendental operations (quarter rate) and the conversions of an element come near it.
#include "qf8_act.h"
#include "qf8_internal.h"
#include "qf8_rows.h"

namespace qf8 {
namespace {

constexpr int kGateThreads = 256, kGatePasses = 4;

// Codes and scale of the group that this lane's eight values belong to, written where they are asked for.
template <typename TX>
__device__ __forceinline__ void leave(const GateArgs &p, const float *y, bool ok, int64_t at, int64_t group) {
    const uint32_t amax = group_amax(y);
    const bool first = (threadIdx.x & 15) == 0 && ok;
    if (p.nonfinite && first && amax >= (p.y ? kNotFinite<TX> : kNotFinite<float>)) *p.nonfinite = 1;
    if (p.y && ok) {
        Eight<TX> e;
        e.round(y);
        e.store_stream((TX *)p.y + at);
    }
    if (p.q) {
        const float s = group_scale(amax, p.fmt, p.pow2);
        const uint2 c = group_codes(y, s, p.fmt);
        if (ok) st_stream((uint2 *)(p.q + at), c);
        if (first) p.scales[group] = s;
    }
}

template <typename TX, int ACT, bool BACKWARD>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs p) {
    constexpr bool EXACT = sizeof(TX) == 4;
    constexpr int GROUPS = kGateThreads / 16, N = BACKWARD ? kGatePasses / 2 : kGatePasses;
    Eight<TX> a[N], b[N], d[N];
    uint32_t row[N], j[N];
    bool ok[N];
    const int cols = (int)p.cols, col0 = (threadIdx.x & 15) * 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t g = (blockIdx.x * N + i) * GROUPS + (threadIdx.x >> 4);
        row[i] = g / p.gcols;
        j[i] = g - row[i] * p.gcols;
        const int col = (int)j[i] * 128 + col0;
        ok[i] = g < p.groups && col < cols;
        a[i].zero(); b[i].zero(); d[i].zero();
        if (ok[i]) {
            const TX *x = (const TX *)p.x + (int64_t)row[i] * 2 * cols + col;
            a[i].stream(x);
            b[i].stream(x + cols);
            if constexpr (BACKWARD) d[i].stream((const TX *)p.dy + (int64_t)row[i] * cols + col);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float av[8], bv[8];
        a[i].values(av);
        b[i].values(bv);
        const int col = (int)j[i] * 128 + col0;
        if constexpr (!BACKWARD) {
#pragma unroll
            for (int k = 0; k < 8; ++k) av[k] = act<ACT, EXACT>(av[k]) * bv[k];
            leave<TX>(p, av, ok[i], (int64_t)row[i] * cols + col, (int64_t)row[i] * p.gcols + j[i]);
        } else {
            float dv[8];
            d[i].values(dv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float slope;
                const float y = act_slope<ACT, EXACT>(av[k], &slope);
                av[k] = dv[k] * bv[k] * slope;
                bv[k] = dv[k] * y;
            }
            // with codes, cols is a multiple of 128 and each half has whole groups
            const int64_t at = (int64_t)row[i] * 2 * cols + col, group = (int64_t)row[i] * 2 * p.gcols + j[i];
            leave<TX>(p, av, ok[i], at, group);
            leave<TX>(p, bv, ok[i], at + cols, group + p.gcols);
        }
    }
}

template <typename TX, int ACT>
int launch_gate_type(const GateArgs &p, int backward, hipStream_t s) {
    const int per = kGateThreads / 16 * (backward ? kGatePasses / 2 : kGatePasses);
    const dim3 grid((p.groups + per - 1) / per), block(kGateThreads);
    if (backward) hipLaunchKernelGGL((gate_kernel<TX, ACT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((gate_kernel<TX, ACT, false>), grid, block, 0, s, p);
    return hipGetLastError() == hipSuccess ? QF8_OK : QF8_ERR_HIP;
}

}  // namespace

int launch_gate(const GateArgs &p, int dtype, int act, int backward, hipStream_t s) {
    if (dtype == QF8_IN_BF16)
        return act == QF8_ACT_SILU ? launch_gate_type<uint16_t, QF8_ACT_SILU>(p, backward, s)
                                   : launch_gate_type<uint16_t, QF8_ACT_GELU>(p, backward, s);
    return act == QF8_ACT_SILU ? launch_gate_type<float, QF8_ACT_SILU>(p, backward, s)
                               : launch_gate_type<float, QF8_ACT_GELU>(p, backward, s);
}

}  // namespace qf8
