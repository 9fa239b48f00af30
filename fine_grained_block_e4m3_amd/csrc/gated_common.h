// gated_common.h -- the activations of the gated feed-forward operators and
// the BF16 store of a matrix-instruction subtile, for gfx950.
#pragma once

#include "device_common.h"

namespace fp8k {

// Activations of a gated block: h = act(g) * u, act(g) = g * p(g).
//   kActSilu  p = 1 / (1 + e^-g)
//   kActGelu  p = 1 / (1 + e^-t), t = 2 sqrt(2/pi) (g + 0.044715 g^3)
//             (0.5 (1 + tanh(t/2)) written with one exponential)
// For large |g| the exponential overflows to infinity or vanishes, so p
// reaches 0 and 1 exactly and no branch is needed.  The reciprocal is the
// hardware's (1 unit in the last place): the results are rounded to 8 bits or
// fewer, or multiplied into FP32 sums, after it.
enum GatedAct : int { kActSilu = 0, kActGelu = 1 };
constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float gated_sigma(int act, float g) {
    const float t = act == kActSilu ? g : kGeluA * (g + kGeluB * g * g * g);
    return __builtin_amdgcn_rcpf(1.0f + __expf(-t));
}
__device__ __forceinline__ float gated_act(int act, float g) { return g * gated_sigma(act, g); }

// act'(g) = p (1 + g (1 - p) t'(g)), t'(g) = 1 for silu.
__device__ __forceinline__ float gated_act_grad(int act, float g) {
    const float p = gated_sigma(act, g);
    const float dt = act == kActSilu ? 1.0f : kGeluA * (1.0f + 3.0f * kGeluB * g * g);
    // where p is 0 or 1 the second term is 0 (g * dt may be infinite there)
    const float pq = p * (1.0f - p);
    return pq == 0.0f ? p : p + g * dt * pq;
}

// BF16 store of the 16 values a lane holds of a 32x32 subtile: columns
// n + 8 q + (0..3), q = 0..3, of one row of N columns.  8-byte stores, whatever
// the row's alignment (3873 x 3614 x 1280 with g and u: 2-byte ones 198 us,
// so 108).
__device__ __forceinline__ void store_bf16_subtile(uint16_t* row, int64_t n, int64_t N, f32x16 v) {
#pragma unroll
    for (int q = 0; q < 4; ++q, n += 8) {
        const uint32_t lo = pack_bf16x2(v[4 * q], v[4 * q + 1]);
        const uint32_t hi = pack_bf16x2(v[4 * q + 2], v[4 * q + 3]);
        if (n + 3 < N) {
            const uint2 all = make_uint2(lo, hi);
            __builtin_memcpy(row + n, &all, 8);
        } else {
            if (n < N) row[n] = (uint16_t)(lo & 0xFFFF);
            if (n + 1 < N) row[n + 1] = (uint16_t)(lo >> 16);
            if (n + 2 < N) row[n + 2] = (uint16_t)(hi & 0xFFFF);
            if (n + 3 < N) row[n + 3] = (uint16_t)(hi >> 16);
        }
    }
}

// The same values in FP32.
__device__ __forceinline__ void store_f32_subtile(float* row, int64_t n, int64_t N, f32x16 v) {
#pragma unroll
    for (int q = 0; q < 4; ++q, n += 8) {
        if (n + 3 < N) {
            const f32x4 all = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            __builtin_memcpy(row + n, &all, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < N) row[n + j] = v[4 * q + j];
        }
    }
}

}  // namespace fp8k
