// kernels_gated_join.h -- the joining kernel of the gated feed-forward block.
#pragma once

#include "gated_common.h"
#include "gemm_common.h"

namespace fp8k {

// ---------------------------------------------------------------------------
// Gated feed-forward block with K split over workgroups (tiles too few to fill
// the device), or codes of few tokens, whose groups of 128 columns no workgroup
// of kernels_skinny.h holds (S = 1): joins the FP32 partial sums of the gate
// (part[0][s]) and up (part[1][s]) projections, s in order, and forms
// h = act(g) * u.  A wave takes 128 columns of one row (two per lane), the group of the quantized
// form.  A stream of the sums (300 x 2048, 8 splits: 5.4 us with its launch).
// ---------------------------------------------------------------------------
template <bool QOUT, bool POW2>
__global__ __launch_bounds__(256) void gated_join_kernel(GemmParams p, int S) {
    const int64_t groups = (p.N + 127) / 128;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= p.M * groups) return;
    const int lane = threadIdx.x & 63;
    const int64_t m = id / groups, n = (id - m * groups) * 128 + 2 * lane;
    const int64_t mn = p.M * p.N, at = m * p.N + n;
    float g[2] = {0.f, 0.f}, u[2] = {0.f, 0.f}, h[2];
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (n + j < p.N) {
                g[j] += p.part[s * mn + at + j];
                u[j] += p.part[(S + s) * mn + at + j];
            }
#pragma unroll
    for (int j = 0; j < 2; ++j) h[j] = gated_act(p.act, g[j]) * u[j];
    if constexpr (QOUT) {   // N % 128 == 0
        float amax = fmaxf(fabsf(h[0]), fabsf(h[1]));
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
        const float sc = group_scale(amax, POW2);
        *reinterpret_cast<uint16_t*>(p.yq + at) = (uint16_t)cvt_e4m3x2(h[0] / sc, h[1] / sc, 0, false);
        if (lane == 0) p.sy[(n >> 7) * p.M + m] = sc;
    } else {
        const uint32_t hb = pack_bf16x2(h[0], h[1]), gb = pack_bf16x2(g[0], g[1]), ub = pack_bf16x2(u[0], u[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (n + j < p.N) {
                p.y[at + j] = (uint16_t)(hb >> (16 * j));
                if (p.g_out) {
                    p.g_out[at + j] = (uint16_t)(gb >> (16 * j));
                    p.u_out[at + j] = (uint16_t)(ub >> (16 * j));
                }
            }
    }
}

}  // namespace fp8k
