// ffn_api.hip -- host side of the feed-forward operators of libfp8gemm.so:
// the gated block and its gradient, 4-bit matrix-vector products, and the
// gradient norm with clipping (declared in include/fp8gemm.h).
//
// As in fp8gemm_api.hip every entry point validates on the host, enqueues
// nothing on an error, launches on the caller's stream, and neither
// allocates, frees nor synchronizes.
#include <algorithm>

#include "host_common.h"
#include "kernels_clip.h"
#include "kernels_exact.h"
#include "kernels_gated_grad.h"
#include "kernels_gated_join.h"
#include "skinny.h"

namespace {

using namespace fp8h;


bool act_ok(int32_t act) { return act == FP8_ACT_SILU || act == FP8_ACT_GELU; }

// ---------------------------------------------------------------------------
// Gated block, forward.
// ---------------------------------------------------------------------------
enum GatedOutputs : int32_t { kOutH = 0, kOutSave = 1, kOutQuant = 2 };

// Up to 64 tokens may take a kernel built around the weights' stream
// (kernels_skinny.h), K split inside its workgroups.  Tiles of the rest: rows x
// output columns, and the time of one K block when every compute unit has one
// (one MI355X, K 7168, us).
enum GatedTile : int { kGated256x128, kGated128x128, kGated128x64, kGated64x128, kGated64x64, kGatedTiles };
struct GatedTileInfo {
    int bm, cols;
    double us;
    bool quant;                 // has a quantized-output form (its 128 columns are one group)
};
constexpr GatedTileInfo kGatedTile[kGatedTiles] = {
    {256, 128, 3.54, true}, {128, 128, 1.88, true}, {128, 64, 1.14, false}, {64, 128, 1.12, true}, {64, 64, 0.85, false}};

// The tile, and the workgroups along K per tile (only where the tiles leave
// compute units idle, all in one round), with the least estimated time: the
// rounds' K blocks, 3 us to start and end a round, and for a split a second
// launch (4 us) and its FP32 sums written and read at 4 TB/s.
//
// The kernel for few tokens is the faster one up to 16 tokens (one MI355X, it
// against the tiles: 1 x 2048 x 7168 7.5 us, 16.6; 16 x 24576 x 7168 67, 70).
// More tokens widen x again in each of its workgroups, so that the estimates
// decide (64 x 512 x 1536 6.0, 14.0; 64 x 2048 x 7168 14.2, 19.7; 32 x 7168 x
// 7168 23.6, 28.9; 48 x 7168 x 7168, before its loads were paired, 45, 31); a
// second launch counts 3 us more there, and no tiles are faster than the
// weights arrive (5 TB/s).  Codes are formed by the joining kernel then, whose
// launch it has to make up for.
struct GatedPlan {
    bool skinny;
    GatedTile tile;
    int64_t splits;
    size_t ws_bytes;            // of FP32 sums
};
GatedPlan gated_plan(int64_t M, int64_t N, int64_t K, int32_t outputs, bool may_split, int cus) {
    GatedPlan best{false, kGated256x128, 1, 0};
    const bool quant = outputs == kOutQuant;
    if (M <= 16 && !quant) {
        best.skinny = true;
        return best;
    }
    const int64_t kb = K / 128;
    double few = 1e30;
    if (M <= kMaxSkinnyGatedM && (may_split || !quant)) {
        few = skinny_gated_e4m3_us(M, N, K, cus) + (quant ? 4.0 + 16.0 * (double)(M * N) / 4e6 : 0.0);
        // no tiles can take less: one round of the smallest, split or not
        const double unsplit = 3.0 + kGatedTile[kGated64x64].us * (double)kb;
        const double split = 3.0 + kGatedTile[kGated64x64].us * (double)kb / 8 + 7.0;
        best.skinny = few <= (unsplit < split ? unsplit : split);
    }
    double least = 1e30;
    for (int t = 0; t < kGatedTiles && !best.skinny; ++t) {
        const GatedTileInfo& i = kGatedTile[t];
        const int64_t tiles = cdiv(M, i.bm) * cdiv(N, i.cols);
        for (int64_t s = 1; s <= 8; ++s) {
            if (s > 1 && (!may_split || tiles * s > cus || kb < 4 * s)) break;
            if (s == 1 && quant && !i.quant) continue;
            double us = (double)cdiv(tiles, cus) * (i.us * (double)cdiv(kb, s) + 3.0);
            if (s > 1) us += 4.0 + 16.0 * (double)(s * M * N) / 4e6;
            if (us < least) {
                least = us;
                best.tile = (GatedTile)t;
                best.splits = s;
            }
        }
    }
    if (best.splits > 1) least += 3.0;
    const double stream = 3.0 + (double)(2 * N * K) / 5e6;
    best.skinny = few <= (least > stream ? least : stream);
    if (best.skinny) best.splits = 1;
    if (best.skinny ? quant : best.splits > 1) best.ws_bytes = (size_t)(2 * best.splits * M * N) * sizeof(float);
    return best;
}

// The plan of a call with ws_bytes of workspace.
GatedPlan gated_plan_within(int64_t M, int64_t N, int64_t K, int32_t outputs, size_t ws_bytes, int cus) {
    const GatedPlan pl = gated_plan(M, N, K, outputs, true, cus);
    return pl.ws_bytes > ws_bytes ? gated_plan(M, N, K, outputs, false, cus) : pl;
}

template <int BM, int BN, int WM, int WN, bool POW2, int STAGES, bool QOUT = false>
fp8_status launch_gated_tile(fp8k::GemmParams p, int64_t splits, int cus, hipStream_t stream) {
    p.m_tiles = (int)cdiv(p.M, BM);
    p.n_tiles = (int)cdiv(p.N, BN / 2);
    p.group_m = 4;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    const dim3 grid((unsigned)(tiles < cus ? tiles : cus), (unsigned)splits);
    hipLaunchKernelGGL((fp8k::gemm_exact_kernel<BM, BN, WM, WN, fp8k::kDense, POW2, STAGES, QOUT, true>), grid,
                       dim3(64 * WM * WN), 0, stream, p.xq, p.sa, p.wq, p.sb, p.y, p.m_indices, p.masked_m, p);
    return launch_status();
}

// The joining kernel: K splits' sums to the outputs.
fp8_status launch_gated_join(const fp8k::GemmParams& p, bool quant, bool pow2, int64_t splits, hipStream_t stream) {
    const int64_t blocks = cdiv(p.M * cdiv(p.N, 128), 4);
    if (blocks > 0x7FFFFFFF) return FP8_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks), block(256);
    const int s = (int)splits;
    if (!quant) hipLaunchKernelGGL((fp8k::gated_join_kernel<false, false>), grid, block, 0, stream, p, s);
    else if (pow2) hipLaunchKernelGGL((fp8k::gated_join_kernel<true, true>), grid, block, 0, stream, p, s);
    else hipLaunchKernelGGL((fp8k::gated_join_kernel<true, false>), grid, block, 0, stream, p, s);
    return launch_status();
}

template <bool POW2>
fp8_status run_gated_tiles(const fp8k::GemmParams& p, const GatedPlan& pl, bool quant, int cus, hipStream_t stream) {
    const int64_t s = pl.splits;
    if (s == 1 && quant) {
        switch (pl.tile) {
            case kGated256x128: return launch_gated_tile<256, 256, 4, 2, POW2, 2, true>(p, 1, cus, stream);
            case kGated128x128: return launch_gated_tile<128, 256, 2, 4, POW2, 3, true>(p, 1, cus, stream);
            default: return launch_gated_tile<64, 256, 2, 4, POW2, 3, true>(p, 1, cus, stream);
        }
    }
    fp8_status st;
    switch (pl.tile) {
        case kGated256x128: st = launch_gated_tile<256, 256, 4, 2, POW2, 2>(p, s, cus, stream); break;
        case kGated128x128: st = launch_gated_tile<128, 256, 2, 4, POW2, 3>(p, s, cus, stream); break;
        case kGated128x64: st = launch_gated_tile<128, 128, 4, 2, POW2, 4>(p, s, cus, stream); break;
        case kGated64x128: st = launch_gated_tile<64, 256, 2, 4, POW2, 3>(p, s, cus, stream); break;
        default: st = launch_gated_tile<64, 128, 2, 2, POW2, 4>(p, s, cus, stream); break;
    }
    return st == FP8_OK && s > 1 ? launch_gated_join(p, quant, POW2, s, stream) : st;
}

fp8_status check_gemv(int64_t M, int64_t N, int64_t K, int32_t group) {
    if (!dims_ok(M) || !dims_ok(N) || !dims_ok(K) ||
        !(group == FP8_W4_MXFP4 || group == 32 || group == 64 || group == 128))
        return FP8_ERR_INVALID_ARG;
    if (K % 128 || K == 0 || M > kMaxSkinnyM) return FP8_ERR_SHAPE;
    if (K > kMaxGemmK) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status check_gated(int64_t M, int64_t N, int64_t K, int32_t act, uint32_t flags) {
    if (!dims_ok(M) || !dims_ok(N) || !dims_ok(K) || !act_ok(act) || (flags & ~FP8_FLAG_UE8M0))
        return FP8_ERR_INVALID_ARG;
    if (K % 128) return FP8_ERR_SHAPE;
    if (K > kMaxGemmK) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status run_gated(fp8k::GemmParams& p, int32_t outputs, uint32_t flags, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
    int cus = 0;
    const fp8_status st = current_device_cus(&cus);
    if (st != FP8_OK) return st;
    const bool quant = outputs == kOutQuant, pow2 = flags & FP8_FLAG_UE8M0;
    const GatedPlan pl = gated_plan_within(p.M, p.N, p.K, outputs, ws_bytes, cus);
    if (pl.ws_bytes) p.part = static_cast<float*>(ws);
    if (pl.skinny) {
        fp8k::SkinnyParams q{};
        q.x = p.xq; q.sa = p.sa; q.w[0] = p.wq; q.w[1] = p.wq2; q.s[0] = p.sb; q.s[1] = p.sb2;
        q.y = p.y; q.g = p.g_out; q.u = p.u_out; q.part = p.part;
        q.M = p.M; q.N = p.N; q.K = p.K; q.act = p.act;
        const fp8_status run = run_skinny_gated_e4m3(q, cus, stream);
        return run == FP8_OK && quant ? launch_gated_join(p, true, pow2, 1, stream) : run;
    }
    return pow2 ? run_gated_tiles<true>(p, pl, quant, cus, stream) : run_gated_tiles<false>(p, pl, quant, cus, stream);
}

// ---------------------------------------------------------------------------
// Gradient of the gated block.
// ---------------------------------------------------------------------------
int64_t grad_np(int64_t N) { return cdiv(N, 64) * 64; }

// Tiles and splits of the two products.
struct GradPlan {
    bool dx_wide, dw_wide;      // 128x256 tiles, else 128x128
    bool dw_first;
    int64_t dx_tiles, dw_tiles, dx_splits, dw_splits;
    int64_t arrived;            // tiles with splits
    size_t d_bytes, dx_part, dw_part;   // workspace: dg and du, then FP32 sums, then a count per such tile
    size_t bytes() const { return d_bytes + dx_part + dw_part + (size_t)arrived * sizeof(int32_t); }
};

// Two workgroups of four waves with 128x256 tiles (64x128 per wave) fit a
// compute unit, or three with 128x128 tiles: one multiplies while another
// waits at a barrier, fills its stages or stores.  The wide tile reads a
// quarter less per product; a product takes it where it still gives every
// such slot a tile.  One MI355X, dX / dW columns per tile: 4096x2048x7168
// 256/256 409 us, 128/128 491; 500x2112x7168 (112 and 952 wide tiles) 128/256
// 87, 256/256 100, 128/128 91; 777x500x640 128/128 12.6, 256/256 17.7.  One
// 256x256 workgroup of eight waves per compute unit: 440 us on the first.
GradPlan grad_plan(int64_t M, int64_t N, int64_t K, bool dx, bool dw, int cus) {
    GradPlan pl{};
    const int64_t dx_blocks = 2 * cdiv(N, 32), dw_blocks = cdiv(M, 32);     // of 32 steps
    const int64_t dx_rows = dx ? cdiv(M, 128) : 0, dw_rows = dw ? 2 * cdiv(N, 128) : 0;
    pl.dx_wide = dx_rows * cdiv(K, 256) >= 2 * cus;
    pl.dw_wide = dw_rows * cdiv(K, 256) >= 2 * cus;
    pl.dx_tiles = dx_rows * cdiv(K, pl.dx_wide ? 256 : 128);
    pl.dw_tiles = dw_rows * cdiv(K, pl.dw_wide ? 256 : 128);
    pl.dw_first = dw_blocks > dx_blocks;
    pl.d_bytes = (size_t)(2 * M * grad_np(N)) * sizeof(uint16_t);
    // Split a product whose few tiles have contractions several times the share
    // of a slot (they would run alone at the end), and tiles that leave half of
    // the slots empty; the sums of more splits, written past the caches, cost
    // more than they save.  One MI355X, us: 256x4096x7168 106 (unsplit 145),
    // 384x4096x4096 90 (129), 20x600x1024 15.0 (18.0), 777x500x640 16.1 (18.3);
    // tiles of about a share: 500x2112x7168 92 (87), 1500x1024x2048 53 (39).
    const int64_t slots = (pl.dx_wide || pl.dw_wide ? 2 : 3) * cus;
    const int64_t share = (pl.dx_tiles * dx_blocks * (pl.dx_wide ? 2 : 1) +
                           pl.dw_tiles * dw_blocks * (pl.dw_wide ? 2 : 1)) / slots;
    const int64_t tiles = pl.dx_tiles + pl.dw_tiles;
    // (a product with wide tiles has one for every slot: it is not split)
    auto splits = [&](int64_t n_tiles, int64_t blocks, bool wide) {
        if (!n_tiles || wide) return (int64_t)1;
        int64_t s = blocks / (share > 16 ? share : 16);
        if (s < 2) s = std::min(blocks / 16, slots / tiles);
        return std::clamp(s, (int64_t)1, (int64_t)8);
    };
    pl.dx_splits = splits(pl.dx_tiles, dx_blocks, pl.dx_wide);
    pl.dw_splits = splits(pl.dw_tiles, dw_blocks, pl.dw_wide);
    auto part = [&](int64_t n_tiles, int64_t s) -> size_t {
        if (s == 1) return 0;
        pl.arrived += n_tiles;
        return (size_t)(n_tiles * s * 128 * 128) * sizeof(float);
    };
    pl.dx_part = part(pl.dx_tiles, pl.dx_splits);
    pl.dw_part = part(pl.dw_tiles, pl.dw_splits);
    return pl;
}

template <int BNX, int BNW, int OCC>
fp8_status launch_grad(const fp8k::GatedGradParams& p, bool dw_first, hipStream_t stream) {
    const int64_t wgs = (int64_t)p.dx_tiles * p.dx_splits + (int64_t)p.dw_tiles * p.dw_splits;
    hipLaunchKernelGGL((fp8k::gated_grad_gemm_kernel<128, BNX, BNW, 2, 2, 3, OCC>), dim3((unsigned)wgs), dim3(256), 0,
                       stream, p, dw_first);
    return launch_status();
}

fp8_status run_grad(fp8k::GatedGradParams& p, const GradPlan& pl, uint8_t* ws, hipStream_t s) {
    if (pl.dx_tiles * pl.dx_splits + pl.dw_tiles * pl.dw_splits > 0x7FFFFFFF ||
        cdiv(p.M * (p.NP / 8), 256) > 0x7FFFFFFF)
        return FP8_ERR_UNSUPPORTED;
    p.d = reinterpret_cast<uint16_t*>(ws);
    p.dx_part = reinterpret_cast<float*>(ws + pl.d_bytes);
    p.dw_part = reinterpret_cast<float*>(ws + pl.d_bytes + pl.dx_part);
    p.arrived = reinterpret_cast<int32_t*>(ws + pl.d_bytes + pl.dx_part + pl.dw_part);
    p.arrived_tiles = (int32_t)pl.arrived;
    p.dx_tiles = (int32_t)pl.dx_tiles;
    p.dw_tiles = (int32_t)pl.dw_tiles;
    p.dx_splits = (int32_t)pl.dx_splits;
    p.dw_splits = (int32_t)pl.dw_splits;
    if (pl.dx_tiles + pl.dw_tiles == 0) return FP8_OK;
    fp8_status st = FP8_OK;
    if (p.M && p.N) {
        const dim3 grid((unsigned)cdiv(p.M * (p.NP / 8), 256)), block(256);
        if (p.N % 8 == 0) hipLaunchKernelGGL(fp8k::gated_grad_act_kernel<true>, grid, block, 0, s, p);
        else hipLaunchKernelGGL(fp8k::gated_grad_act_kernel<false>, grid, block, 0, s, p);
        st = launch_status();
    }
    if (st == FP8_OK) {
        if (pl.dx_wide) st = pl.dw_wide ? launch_grad<256, 256, 2>(p, pl.dw_first, s) : launch_grad<256, 128, 2>(p, pl.dw_first, s);
        else st = pl.dw_wide ? launch_grad<128, 256, 2>(p, pl.dw_first, s) : launch_grad<128, 128, 3>(p, pl.dw_first, s);
    }
    return st;
}

// ---------------------------------------------------------------------------
// Gradient clipping.
// ---------------------------------------------------------------------------
int64_t clip_chunks(int64_t n) { return cdiv(n, fp8k::kClipChunk); }
constexpr int64_t kMaxClipChunks = (int64_t)1 << 30;     // per launch: counted in int32, a grid at a time
int clip_grid(int64_t chunks) { return (int)(chunks < fp8k::kClipMaxGrid ? chunks : fp8k::kClipMaxGrid); }

// Calls f(first tensor, tensors, chunks) for each batch of the call, or from
// the last batch to the first.
template <typename F>
fp8_status clip_batches(const int64_t* sizes, int32_t count, bool backwards, F&& f) {
    const int32_t batches = (int32_t)cdiv(count, fp8k::kClipBatch);
    for (int32_t b = 0; b < batches; ++b) {
        const int32_t i = (backwards ? batches - 1 - b : b) * fp8k::kClipBatch;
        const int32_t k = count - i < fp8k::kClipBatch ? count - i : fp8k::kClipBatch;
        int64_t chunks = 0;
        for (int32_t j = 0; j < k; ++j) chunks += clip_chunks(sizes[i + j]);
        if (chunks > kMaxClipChunks) return FP8_ERR_UNSUPPORTED;
        const fp8_status st = f(i, k, chunks);
        if (st != FP8_OK) return st;
    }
    return FP8_OK;
}

}  // namespace

extern "C" {

size_t fp8_gated_workspace_size(int64_t M, int64_t N, int64_t K, int32_t outputs) {
    if (!dims_ok(M) || !dims_ok(N) || !dims_ok(K) || K % 128 || M == 0 || N == 0 || K == 0 || outputs < 0 ||
        outputs > 2)
        return 0;
    int cus = 0;
    if (current_device_cus(&cus) != FP8_OK) return 0;
    return gated_plan(M, N, K, outputs, true, cus).ws_bytes;
}

fp8_status fp8_gated_plan(int64_t M, int64_t N, int64_t K, int32_t outputs, int32_t compute_units,
                          size_t workspace_bytes, fp8_gated_plan_t* plan) {
    if (!plan || !dims_ok(M) || !dims_ok(N) || !dims_ok(K) || outputs < kOutH || outputs > kOutQuant ||
        compute_units <= 0)
        return FP8_ERR_INVALID_ARG;
    if (K % 128 || K == 0 || (outputs == kOutQuant && N % 128)) return FP8_ERR_SHAPE;
    if (K > kMaxGemmK) return FP8_ERR_UNSUPPORTED;
    *plan = fp8_gated_plan_t{};
    if (M == 0 || N == 0) return FP8_OK;
    const GatedPlan pl = gated_plan_within(M, N, K, outputs, workspace_bytes, compute_units);
    plan->few_tokens = pl.skinny;
    plan->tile_m = pl.skinny ? (int32_t)cdiv(M, 16) * 16 : kGatedTile[pl.tile].bm;
    plan->tile_n = pl.skinny ? 8 * skinny_gated_e4m3_tiles(M, N, compute_units) : kGatedTile[pl.tile].cols;
    plan->k_splits = (int32_t)pl.splits;
    plan->joined = pl.ws_bytes != 0;
    plan->tiles = cdiv(M, plan->tile_m) * cdiv(N, plan->tile_n);
    plan->workspace_bytes = pl.ws_bytes;
    return FP8_OK;
}

fp8_status fp8_gated_nt(const uint8_t* xq, const float* sa, const uint8_t* wgq, const float* sbg,
                        const uint8_t* wuq, const float* sbu, uint16_t* h, uint16_t* g, uint16_t* u, int64_t M,
                        int64_t N, int64_t K, int32_t act, uint32_t flags, void* workspace, size_t workspace_bytes,
                        void* stream) {
    const fp8_status st = check_gated(M, N, K, act, flags);
    if (st != FP8_OK) return st;
    if (M == 0 || N == 0) return FP8_OK;
    if (K == 0) return FP8_ERR_SHAPE;
    if (!xq || !sa || !wgq || !sbg || !wuq || !sbu || !h || (!g != !u) || (workspace_bytes && !workspace))
        return FP8_ERR_INVALID_ARG;
    for (const void* p : {(const void*)xq, (const void*)sa, (const void*)wgq, (const void*)sbg, (const void*)wuq,
                          (const void*)sbu, (const void*)h, (const void*)g, (const void*)u, (const void*)workspace})
        if (!aligned16(p)) return FP8_ERR_ALIGNMENT;
    fp8k::GemmParams p{};
    p.xq = xq; p.sa = sa; p.wq = wgq; p.sb = sbg; p.wq2 = wuq; p.sb2 = sbu;
    p.y = h; p.g_out = g; p.u_out = u; p.act = act;
    p.M = M; p.N = N; p.K = K; p.E = 1;
    return run_gated(p, g ? kOutSave : kOutH, flags, workspace, workspace ? workspace_bytes : 0, (hipStream_t)stream);
}

fp8_status fp8_gated_nt_qout(const uint8_t* xq, const float* sa, const uint8_t* wgq, const float* sbg,
                             const uint8_t* wuq, const float* sbu, uint8_t* hq, float* sh, int64_t M, int64_t N,
                             int64_t K, int32_t act, uint32_t flags, void* workspace, size_t workspace_bytes,
                             void* stream) {
    const fp8_status st = check_gated(M, N, K, act, flags);
    if (st != FP8_OK) return st;
    if (N % 128) return FP8_ERR_SHAPE;
    if (M == 0 || N == 0) return FP8_OK;
    if (K == 0) return FP8_ERR_SHAPE;
    if (!xq || !sa || !wgq || !sbg || !wuq || !sbu || !hq || !sh || (workspace_bytes && !workspace))
        return FP8_ERR_INVALID_ARG;
    for (const void* p : {(const void*)xq, (const void*)sa, (const void*)wgq, (const void*)sbg, (const void*)wuq,
                          (const void*)sbu, (const void*)hq, (const void*)sh, (const void*)workspace})
        if (!aligned16(p)) return FP8_ERR_ALIGNMENT;
    fp8k::GemmParams p{};
    p.xq = xq; p.sa = sa; p.wq = wgq; p.sb = sbg; p.wq2 = wuq; p.sb2 = sbu;
    p.yq = hq; p.sy = sh; p.act = act;
    p.M = M; p.N = N; p.K = K; p.E = 1;
    return run_gated(p, kOutQuant, flags, workspace, workspace ? workspace_bytes : 0, (hipStream_t)stream);
}

size_t fp8_gated_grad_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (!dims_ok(M) || !dims_ok(N) || !dims_ok(K) || K % 128 || K > kMaxGemmK || N > kMaxGemmK - 64) return 0;
    int cus = 0;
    if (current_device_cus(&cus) != FP8_OK) return 0;
    // of a call for all gradients, or for some of them
    size_t most = 0;
    for (int which = 1; which <= 3; ++which) {
        const size_t b = grad_plan(M, N, K, which & 1 && M, which & 2 && N, cus).bytes();
        if (b > most) most = b;
    }
    return most;
}

fp8_status fp8_gated_grad_plan(int64_t M, int64_t N, int64_t K, int32_t dx, int32_t dw, int32_t compute_units,
                               fp8_gated_grad_plan_t* plan) {
    if (!plan || !dims_ok(M) || !dims_ok(N) || !dims_ok(K) || compute_units <= 0) return FP8_ERR_INVALID_ARG;
    if (K % 128) return FP8_ERR_SHAPE;
    if (K > kMaxGemmK || N > kMaxGemmK - 64) return FP8_ERR_UNSUPPORTED;
    *plan = fp8_gated_grad_plan_t{};
    if (K == 0 || (!dx && !dw)) return FP8_OK;
    const GradPlan pl = grad_plan(M, N, K, dx && M, dw && N, compute_units);
    plan->dx_tile_n = pl.dx_wide ? 256 : 128;
    plan->dw_tile_n = pl.dw_wide ? 256 : 128;
    plan->dx_splits = (int32_t)pl.dx_splits;
    plan->dw_splits = (int32_t)pl.dw_splits;
    plan->dw_first = pl.dw_first;
    plan->dx_tiles = pl.dx_tiles;
    plan->dw_tiles = pl.dw_tiles;
    plan->workspace_bytes = pl.bytes();
    return FP8_OK;
}

fp8_status fp8_gated_nt_grad(const uint16_t* dh, const uint16_t* g, const uint16_t* u, const uint16_t* x,
                             const uint16_t* wg, const uint16_t* wu, uint16_t* dx, uint16_t* dwg, uint16_t* dwu,
                             int64_t M, int64_t N, int64_t K, int32_t act, void* workspace, size_t workspace_bytes,
                             void* stream) {
    if (!dims_ok(M) || !dims_ok(N) || !dims_ok(K) || !act_ok(act)) return FP8_ERR_INVALID_ARG;
    if (K % 128) return FP8_ERR_SHAPE;
    if (K > kMaxGemmK || N > kMaxGemmK - 64) return FP8_ERR_UNSUPPORTED;
    if (K == 0 || (M == 0 && N == 0) || (!dx && !dwg && !dwu)) return FP8_OK;
    if (!dwg != !dwu) return FP8_ERR_INVALID_ARG;
    if (M && N && (!dh || !g || !u)) return FP8_ERR_INVALID_ARG;
    if ((M && !x && dwg) || (N && (!wg || !wu) && dx)) return FP8_ERR_INVALID_ARG;
    for (const void* p : {(const void*)dh, (const void*)g, (const void*)u, (const void*)x, (const void*)wg,
                          (const void*)wu, (const void*)dx, (const void*)dwg, (const void*)dwu, (const void*)workspace})
        if (!aligned16(p)) return FP8_ERR_ALIGNMENT;
    if (workspace_bytes && !workspace) return FP8_ERR_INVALID_ARG;
    int cus = 0;
    const fp8_status st = current_device_cus(&cus);
    if (st != FP8_OK) return st;
    const GradPlan pl = grad_plan(M, N, K, dx && M, dwg && N, cus);
    if (workspace_bytes < pl.bytes()) return FP8_ERR_SCRATCH;
    fp8k::GatedGradParams p{};
    p.dh = dh; p.g = g; p.u = u; p.x = x; p.w[0] = wg; p.w[1] = wu;
    p.dx = dx; p.dw[0] = dwg; p.dw[1] = dwu;
    p.M = M; p.N = N; p.K = K; p.NP = grad_np(N); p.act = act;
    return run_grad(p, pl, static_cast<uint8_t*>(workspace), (hipStream_t)stream);
}

fp8_status fp8_gemv_w4(const uint16_t* x, const uint8_t* w, const void* s, const uint8_t* z, uint16_t* y, int64_t M,
                       int64_t N, int64_t K, int32_t group, void* stream) {
    const fp8_status st = check_gemv(M, N, K, group);
    if (st != FP8_OK) return st;
    if (M == 0 || N == 0) return FP8_OK;
    if (!x || !w || !s || !y || (z && group == FP8_W4_MXFP4)) return FP8_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)w, s, (const void*)z, (const void*)y})
        if (!aligned16(p)) return FP8_ERR_ALIGNMENT;
    fp8k::SkinnyParams p{};
    p.x = x; p.w[0] = w; p.s[0] = s; p.z[0] = z; p.y = y;
    p.M = M; p.N = N; p.K = K;
    return run_gemv_w4(p, false, group, (hipStream_t)stream);
}

fp8_status fp8_gated_gemv_w4(const uint16_t* x, const uint8_t* wg, const void* sg, const uint8_t* zg,
                             const uint8_t* wu, const void* su, const uint8_t* zu, uint16_t* y, int64_t M, int64_t N,
                             int64_t K, int32_t group, int32_t act, void* stream) {
    const fp8_status st = check_gemv(M, N, K, group);
    if (st != FP8_OK) return st;
    if (!act_ok(act)) return FP8_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return FP8_OK;
    if (!x || !wg || !sg || !wu || !su || !y || (zg && group == FP8_W4_MXFP4) || (!zg != !zu))
        return FP8_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)wg, sg, (const void*)zg, (const void*)wu, su, (const void*)zu,
                          (const void*)y})
        if (!aligned16(p)) return FP8_ERR_ALIGNMENT;
    fp8k::SkinnyParams p{};
    p.x = x; p.w[0] = wg; p.w[1] = wu; p.s[0] = sg; p.s[1] = su; p.z[0] = zg; p.z[1] = zu; p.y = y;
    p.M = M; p.N = N; p.K = K; p.act = act;
    return run_gemv_w4(p, true, group, (hipStream_t)stream);
}

fp8_status fp8_quant_int4(const float* w, int64_t N, int64_t K, int32_t group, uint8_t* q, uint16_t* s, uint8_t* z,
                          void* stream) {
    if (!dims_ok(N) || !dims_ok(K) || !(group == 32 || group == 64 || group == 128)) return FP8_ERR_INVALID_ARG;
    if (K % 128) return FP8_ERR_SHAPE;
    if (N == 0 || K == 0) return FP8_OK;
    if (!w || !q || !s) return FP8_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(q) || !aligned16(s) || !aligned16(z)) return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status st = current_device_cus(&cus);
    if (st != FP8_OK) return st;
    return run_quant_int4(w, N, K, group, q, s, z, (hipStream_t)stream);
}

size_t fp8_clip_workspace_size(const int64_t* sizes, int32_t count) {
    if (count < 0 || (count && !sizes)) return 0;
    size_t slots = 0;
    for (int32_t i = 0; i < count; ++i)
        if (sizes[i] < 0 || sizes[i] > kMaxClipChunks * fp8k::kClipChunk) return 0;
    const fp8_status st = clip_batches(sizes, count, false, [&](int32_t, int32_t, int64_t chunks) {
        slots += (size_t)clip_grid(chunks);
        return FP8_OK;
    });
    if (st != FP8_OK) return 0;
    return 8 * (slots ? slots : 1);
}

fp8_status fp8_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types,
                              int32_t count, float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                              void* stream) {
    if (count < 0 || !(max_norm >= 0.f) || !norm || (count && (!grads || !outs || !sizes || !types)))
        return FP8_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || types[i] < FP8_TYPE_F32 || types[i] > FP8_TYPE_F16) return FP8_ERR_INVALID_ARG;
        if (sizes[i] && (!grads[i] || !outs[i])) return FP8_ERR_INVALID_ARG;
        const uintptr_t mask = types[i] == FP8_TYPE_F32 ? 3 : 1;
        if (((uintptr_t)grads[i] | (uintptr_t)outs[i]) & mask) return FP8_ERR_ALIGNMENT;
    }
    if (((uintptr_t)norm & 3) || ((uintptr_t)workspace & 7)) return FP8_ERR_ALIGNMENT;
    if (!workspace) return FP8_ERR_INVALID_ARG;
    // (every batch is known to be one that can be launched before the first is)
    const size_t need = fp8_clip_workspace_size(sizes, count);
    if (need == 0) return FP8_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return FP8_ERR_SCRATCH;
    int cus = 0;
    fp8_status st = current_device_cus(&cus);
    if (st != FP8_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    double* slots = static_cast<double*>(workspace);
    auto table = [&](int32_t i, int32_t k) {
        fp8k::ClipTable t{};
        int64_t chunks = 0;
        for (int32_t j = 0; j < k; ++j) {
            t.in[j] = grads[i + j];
            t.out[j] = outs[i + j];
            t.n_type[j] = 4 * sizes[i + j] + types[i + j];
            t.first[j] = (int32_t)chunks;
            chunks += clip_chunks(sizes[i + j]);
        }
        t.first[k] = (int32_t)chunks;
        t.count = k;
        return t;
    };
    int64_t used = 0;
    st = clip_batches(sizes, count, false, [&](int32_t i, int32_t k, int64_t chunks) {
        if (chunks == 0) return FP8_OK;
        hipLaunchKernelGGL(fp8k::clip_norm_kernel, dim3(clip_grid(chunks)), dim3(256), 0, s, table(i, k), slots + used);
        used += clip_grid(chunks);
        return launch_status();
    });
    if (st != FP8_OK) return st;
    if (used > fp8k::kClipMaxSlots) {
        hipLaunchKernelGGL(fp8k::clip_join_kernel, dim3(1), dim3(256), 0, s, slots, (int)used);
        st = launch_status();
        if (st != FP8_OK) return st;
        used = 1;
    }
    if (used == 0) {    // nothing to scale: the norm is 0
        hipLaunchKernelGGL(fp8k::clip_scale_kernel, dim3(1), dim3(256), 0, s, fp8k::ClipTable{}, slots, 0, max_norm, norm);
        return launch_status();
    }
    // backwards: what the first pass read last may still be in the last cache
    return clip_batches(sizes, count, true, [&](int32_t i, int32_t k, int64_t chunks) {
        if (chunks == 0) return FP8_OK;
        hipLaunchKernelGGL(fp8k::clip_scale_kernel, dim3(clip_grid(chunks)), dim3(256), 0, s, table(i, k), slots,
                           (int)used, max_norm, norm);
        norm = nullptr;     // written by the first launch
        return launch_status();
    });
}

}  // extern "C"
