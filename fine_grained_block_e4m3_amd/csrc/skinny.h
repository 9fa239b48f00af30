// skinny.h -- launches of the kernels for few tokens (skinny_launch.hip),
// used by the entry points in ffn_api.hip.
#pragma once

#include "host_common.h"

namespace fp8k {

struct SkinnyParams {
    const void* x;          // BF16 (M, K), or E4M3 codes (M, K)
    const float* sa;        // E4M3: activation scales [K/128][M]
    const uint8_t* w[2];    // weight codes; gated: gate, up
    const void* s[2];       // scales
    const uint8_t* z[2];    // 4-bit integers: zero points, or null (8)
    uint16_t* y;            // BF16 (M, N)
    uint16_t* g;            // gated E4M3: also the projections, BF16 (M, N), or null
    uint16_t* u;
    float* part;            // ... or instead of all three their FP32 sums, (2, M, N)
    int64_t M, N, K;
    int32_t act;
};

}  // namespace fp8k

namespace fp8h {

constexpr int64_t kMaxSkinnyM = 16;         // 4-bit weights
constexpr int64_t kMaxSkinnyGatedM = 64;    // the gated block on E4M3 operands

// 16-row weight tiles per workgroup (8 output columns each) and estimated time
// (us) of the gated block on E4M3 operands.
int skinny_gated_e4m3_tiles(int64_t M, int64_t N, int cus);
double skinny_gated_e4m3_us(int64_t M, int64_t N, int64_t K, int cus);

// The gated block on E4M3 operands; 4-bit matrix-vector products, plain and
// gated; the 4-bit integer quantizer.  Arguments are already checked.
fp8_status run_skinny_gated_e4m3(const fp8k::SkinnyParams& p, int cus, hipStream_t stream);
fp8_status run_gemv_w4(const fp8k::SkinnyParams& p, bool gated, int32_t group, hipStream_t stream);
fp8_status run_quant_int4(const float* w, int64_t N, int64_t K, int32_t group, uint8_t* q, uint16_t* s, uint8_t* z,
                          hipStream_t stream);

}  // namespace fp8h
