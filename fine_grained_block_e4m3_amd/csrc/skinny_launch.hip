// skinny_launch.hip -- instances and launches of the kernels for few tokens
// (kernels_skinny.h).
#include "kernels_skinny.h"

namespace {

using namespace fp8h;

// 16-row weight tiles per workgroup: the number that leaves the fullest compute
// unit the fewest tiles, and of those the largest, whose tiles share the x
// operands.  One MI355X, int4 weights with groups of 128, 16 x 24576 x 7168
// (1536 tiles): 6 per workgroup 25 us, 2 28; groups of 64 30 and 37; gated MXFP4
// 1 x 2048 x 7168 (256 tiles): 1 per workgroup 6.4 us, 2 7.7; 3 x 2112 x 7168
// (264): 1 10.9, 2 8.5.
int pick_tiles(int64_t tiles, int cus, std::initializer_list<int> allowed) {
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int rt : allowed) {
        const int64_t c = cdiv(cdiv(tiles, rt), cus) * rt;
        if (c <= cost) {
            cost = c;
            best = rt;
        }
    }
    return best;
}

constexpr int kWaves = 8, kDepth = 2;

template <int FMT, bool GATED, int RT, int GROUP, bool ZEROS, int MB = 1>
fp8_status launch_skinny(const fp8k::SkinnyParams& p, hipStream_t stream) {
    const int64_t cols = GATED ? 8 * RT : 16 * RT;
    hipLaunchKernelGGL((fp8k::skinny_kernel<FMT, GATED, RT, kWaves, kDepth, GROUP, ZEROS, MB>),
                       dim3((unsigned)cdiv(p.N, cols)), dim3(64 * kWaves), 0, stream, p);
    return launch_status();
}

template <int FMT, bool GATED, int GROUP, bool ZEROS>
fp8_status run_skinny(const fp8k::SkinnyParams& p, int cus, hipStream_t stream) {
    const int64_t tiles = cdiv(p.N * (GATED ? 2 : 1), 16);
    const int rt = GATED ? pick_tiles(tiles, cus, {1, 2, 4, 6}) : pick_tiles(tiles, cus, {1, 2, 3, 4, 6});
    switch (rt) {
        case 1: return launch_skinny<FMT, GATED, 1, GROUP, ZEROS>(p, stream);
        case 2: return launch_skinny<FMT, GATED, 2, GROUP, ZEROS>(p, stream);
        case 3:
            if constexpr (!GATED) return launch_skinny<FMT, GATED, 3, GROUP, ZEROS>(p, stream);
            else return FP8_ERR_UNSUPPORTED;
        case 4: return launch_skinny<FMT, GATED, 4, GROUP, ZEROS>(p, stream);
        default: return launch_skinny<FMT, GATED, 6, GROUP, ZEROS>(p, stream);
    }
}

template <bool GATED>
fp8_status run_w4(const fp8k::SkinnyParams& p, int32_t group, int cus, hipStream_t stream) {
    const bool z = p.z[0] != nullptr;
    switch (group) {
        case FP8_W4_MXFP4: return run_skinny<fp8k::kSkinnyMxfp4, GATED, 32, false>(p, cus, stream);
        case 32:
            return z ? run_skinny<fp8k::kSkinnyInt4, GATED, 32, true>(p, cus, stream)
                     : run_skinny<fp8k::kSkinnyInt4, GATED, 32, false>(p, cus, stream);
        case 64:
            return z ? run_skinny<fp8k::kSkinnyInt4, GATED, 64, true>(p, cus, stream)
                     : run_skinny<fp8k::kSkinnyInt4, GATED, 64, false>(p, cus, stream);
        default:
            return z ? run_skinny<fp8k::kSkinnyInt4, GATED, 128, true>(p, cus, stream)
                     : run_skinny<fp8k::kSkinnyInt4, GATED, 128, false>(p, cus, stream);
    }
}

}  // namespace

namespace fp8h {

// E4M3 weights.  Six tiles, read by pairs of lanes, spill 26 registers (one token
// x 24576 x 7168 91 us, four tiles 66; x 1536 20.5 and 18.8, where six tiles
// without the pairs took 17.5).  More than 16 tokens are taken in blocks
// of 16: each weight operand serves all blocks, and with three or four blocks
// only two weight tiles fit the registers.  One MI355X, gated E4M3, before x
// and the weights were read by pairs of lanes: 32 x 7168 x 7168 4 tiles 27 us,
// 2 36; 64 x 7168 x 7168 2 tiles 47, 4 97; 37 x 2112 x 1536 2 tiles 6.4, 1 8.9.
int skinny_gated_e4m3_tiles(int64_t M, int64_t N, int cus) {
    const int64_t tiles = cdiv(N * 2, 16);
    return M <= 32 ? pick_tiles(tiles, cus, {1, 2, 4}) : pick_tiles(tiles, cus, {1, 2});
}

template <int MB>
static fp8_status run_token_blocks(const fp8k::SkinnyParams& p, int cus, hipStream_t stream) {
    const int rt = skinny_gated_e4m3_tiles(p.M, p.N, cus);
    if (rt == 1) return launch_skinny<fp8k::kSkinnyE4m3, true, 1, 128, false, MB>(p, stream);
    if (rt == 2) return launch_skinny<fp8k::kSkinnyE4m3, true, 2, 128, false, MB>(p, stream);
    if constexpr (MB <= 2) return launch_skinny<fp8k::kSkinnyE4m3, true, 4, 128, false, MB>(p, stream);
    else return FP8_ERR_UNSUPPORTED;
}

// Of a K block a workgroup reads and widens its token blocks (0.015 us each) and
// its weight tiles (0.05 each), and multiplies them (0.024 a pair); fitted on
// one MI355X to 1-64 x 512-24576 x 1536 and 7168, within 15% (64 x 512 x 1536
// 5.5 us for 6.0, 64 x 2048 x 7168 14.5 for 14.2, 32 x 7168 x 7168 26.6 for 23.6).
double skinny_gated_e4m3_us(int64_t M, int64_t N, int64_t K, int cus) {
    const int mb = (int)cdiv(M, 16), rt = skinny_gated_e4m3_tiles(M, N, cus);
    return 3.0 + (double)(K / 128 * cdiv(cdiv(cdiv(N * 2, 16), rt), cus)) * (0.015 * mb + rt * (0.05 + 0.024 * mb));
}

fp8_status run_skinny_gated_e4m3(const fp8k::SkinnyParams& p, int cus, hipStream_t stream) {
    switch (cdiv(p.M, 16)) {
        case 1: return run_token_blocks<1>(p, cus, stream);
        case 2: return run_token_blocks<2>(p, cus, stream);
        case 3: return run_token_blocks<3>(p, cus, stream);
        case 4: return run_token_blocks<4>(p, cus, stream);
        default: return FP8_ERR_UNSUPPORTED;
    }
}

fp8_status run_gemv_w4(const fp8k::SkinnyParams& p, bool gated, int32_t group, hipStream_t stream) {
    int cus = 0;
    const fp8_status st = current_device_cus(&cus);
    if (st != FP8_OK) return st;
    return gated ? run_w4<true>(p, group, cus, stream) : run_w4<false>(p, group, cus, stream);
}

fp8_status run_quant_int4(const float* w, int64_t N, int64_t K, int32_t group, uint8_t* q, uint16_t* s, uint8_t* z,
                          hipStream_t stream) {
    const int64_t blocks = cdiv(N * (K / group), 256 / (group / 4));
    if (blocks > 0x7FFFFFFF) return FP8_ERR_INVALID_ARG;
    const dim3 grid((unsigned)blocks), block(256);
    if (group == 32) hipLaunchKernelGGL(fp8k::quant_int4_kernel<32>, grid, block, 0, stream, w, q, s, z, N, K);
    else if (group == 64) hipLaunchKernelGGL(fp8k::quant_int4_kernel<64>, grid, block, 0, stream, w, q, s, z, N, K);
    else hipLaunchKernelGGL(fp8k::quant_int4_kernel<128>, grid, block, 0, stream, w, q, s, z, N, K);
    return launch_status();
}

}  // namespace fp8h
