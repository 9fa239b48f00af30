// kernels_skinny.h -- products of few tokens with a weight matrix for gfx950:
// matrix-vector products with 4-bit weights and group scales, and the gated
// feed-forward block (4-bit weights: up to 16 tokens; E4M3: up to 64).
//
//   y[m][n] = sum_k x[m][k] w[n][k]
//   gated:  y = act(x Wg^T) * (x Wu^T)
// Weight formats (K % 128 == 0, codes row-major, two 4-bit codes per byte, the
// even element low):
//   kSkinnyMxfp4  w = E2M1 * 2^(e-127) per 32 along K, e packed [K/128][N]
//                 (fp8_quant_mxfp4's layout); x BF16
//   kSkinnyInt4   w = s * (q - z), q = 0..15, per group of 32, 64 or 128:
//                 s BF16 [K/group][N], z u8 [K/group][N] or 8; x BF16
//   kSkinnyE4m3   x and w E4M3 with 1x128 and 128x128 scales
//
// What bounds it: every weight is read once and used M times, so the weight
// stream from HBM.  The kernel is therefore built around that stream:
//   * Weights go from memory straight into the registers in which the matrix
//     instruction takes them: lane (r, q) = (l%16, l/16) of a wave reads the
//     16 bytes q of row r's 64-byte K block (128 4-bit weights), which are
//     the four MFMA steps' operands.  No LDS, no barrier in the K loop.
//   * v_mfma_f32_16x16x32 with the 16 weight rows as A and the tokens as B
//     (4-bit integers: the other way round, so that a lane's results have one
//     scale; up to 4 tokens repeat in groups of 4 rows, and a lane scales one
//     result): tokens past M repeat the last one (their loads coalesce with it) and
//     are not stored.  A vector-FMA form would spend M operations per weight;
//     this one spends the decoding only, whatever M.
//   * The KW waves of a workgroup share its rows and split K; one LDS exchange
//     at the end adds their FP32 sums in wave order.  With few rows this keeps
//     every compute unit reading; no workspace and no second launch.
//   * Every workgroup reads all of x, from its L2: RT 16-row tiles per
//     workgroup share each x operand (the launch picks RT, skinny_launch.hip).
//   * The loads of the D - 1 blocks that follow are in flight while a block is
//     multiplied.
// Exactness: E2M1 times a power of two is a BF16 value (products exact, FP32
// sums; weights of 2^128 and more are infinite, and the scale byte 255 is NaN).
// 4-bit integers enter as the BF16 integers q - z, -15 .. 15, so that a weight
// of zero adds nothing and an infinite x gives what the definition gives; the
// group's sum of x (q - z) is scaled in FP32.  (z applied after the sum, as
// s * (sum x q - z * sum x), takes half the instructions per weight, but
// cancels, and gives NaN for an infinite x.)  E4M3 is widened exactly to FP16.
// Measured (one MI355X, kernel time): gated E4M3 1 x 2048 x 7168 7.4 us
// (29 MB: 4.0 TB/s, the launch's 2.3 us included), MXFP4 1 x 24576 x 7168
// 21 us (4.4 TB/s) and 16 x 24576 x 7168 23 us; int4 1 and 16 x 24576 x 7168
// with groups of 128 24 and 26 us, with zero points 26.3 and 28.7, with
// groups of 64 and zero points 32.5 (16), with groups of 32 and zero points
// 33.3 and 37.9; gated int4 (groups of 64, zero points) 3 x 2112 x 7168 10.8 us.
// With z applied after the sum: 22.1 and 25.0, 22.7 and 25.5, 30.0, 31.4 and
// 39.0; 9.8.  That form with the weights as A for 4-bit integers too, four
// scales and zero points per lane and group: groups of 128 24 and 29 (16 tokens,
// zero points), of 32 45 and 51; gated 11.4.
// Gated E4M3 with g and u stored as well: 1 x 2048 x 7168 7.6 us; with codes
// instead (FP32 sums, then the joining kernel) 11, the tiles 16.6 and 17.2.
#pragma once

#include "gated_common.h"
#include "skinny.h"

namespace fp8k {


enum SkinnyFormat : int { kSkinnyMxfp4 = 0, kSkinnyInt4 = 1, kSkinnyE4m3 = 2 };

// Transposes a 4x4 block of dwords over the four lanes (r, 0..3): afterwards
// v[s] of lane (r, q) is what v[q] of lane (r, s) was.
__device__ __forceinline__ i32x4 transpose_quads(i32x4 v) {
    const auto a = __builtin_amdgcn_permlane32_swap((unsigned)v[0], (unsigned)v[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap((unsigned)v[1], (unsigned)v[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return i32x4{(int)c[0], (int)c[1], (int)d[0], (int)d[1]};
}

// Swaps the second item of even lanes with the first of the odd lane next to
// them.
__device__ __forceinline__ void swap_pair_lanes(i32x4& v0, i32x4& v1, int lane) {
    const bool odd = lane & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int a = v0[j], b = v1[j];
        const int ax = __builtin_amdgcn_mov_dpp(a, 0xB1, 0xF, 0xF, true);
        const int bx = __builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, true);
        v0[j] = odd ? bx : a;
        v1[j] = odd ? b : ax;
    }
}

// Transposes 16-byte items over four registers and the four lanes of a quad:
// afterwards v[s] of quad lane a is what v[a] of quad lane s was.
__device__ __forceinline__ void transpose_quad_lanes(i32x4 (&v)[4], int lane) {
    const bool odd = lane & 1, high = lane & 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int p = 0; p < 4; p += 2) {        // lanes 1 apart
            const int a = v[p][j], b = v[p + 1][j];
            const int ax = __builtin_amdgcn_mov_dpp(a, 0xB1, 0xF, 0xF, true);
            const int bx = __builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, true);
            v[p][j] = odd ? bx : a;
            v[p + 1][j] = odd ? b : ax;
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {           // lanes 2 apart
            const int a = v[p][j], b = v[p + 2][j];
            const int ax = __builtin_amdgcn_mov_dpp(a, 0x4E, 0xF, 0xF, true);
            const int bx = __builtin_amdgcn_mov_dpp(b, 0x4E, 0xF, 0xF, true);
            v[p][j] = high ? bx : a;
            v[p + 2][j] = high ? b : ax;
        }
    }
}

// Eight 4-bit codes of a dword less the zero point z, as BF16 integers in the
// order of the elements.  A half word with nothing but a code in its low bits is
// the FP16 subnormal q * 2^-24 (q * 2^-20 four bits higher), which one
// instruction with FP16 and FP32 operands turns into q - z; BF16 holds that.
__device__ __forceinline__ bf16x8 u4x8_less_zero_to_bf16(int v, float zero) {
    i32x4 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {       // codes 0, 1, 4, 5 and then 2, 3, 6, 7
        const unsigned c = (unsigned)v >> (8 * h);
        const f16x2 a = __builtin_bit_cast(f16x2, c & 0x000F000Fu), b = __builtin_bit_cast(f16x2, c & 0x00F000F0u);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float even = __builtin_fmaf((float)a[j], 0x1p24f, -zero);
            const float odd = __builtin_fmaf((float)b[j], 0x1p20f, -zero);
            r[2 * j + h] = (int)__builtin_amdgcn_perm(__float_as_uint(odd), __float_as_uint(even), 0x07060302u);
        }
    }
    return __builtin_bit_cast(bf16x8, r);
}
// Eight 4-bit codes of a dword less 8, as BF16 values of 1/16 of that, in the
// order of the elements: the hardware converter of a byte's low four bits, taken
// as two's complement, whose FP32 results BF16 holds.
__device__ __forceinline__ bf16x8 u4x8_less8_to_bf16(int v) {
    unsigned lo = (unsigned)v ^ 0x88888888u, hi = lo >> 4;
    asm("" : "+v"(lo), "+v"(hi));       // one shift; then every code is a byte operand
    i32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = __builtin_amdgcn_cvt_off_f32_i4((int)(lo >> (8 * j) & 0xFFu));
        const float b = __builtin_amdgcn_cvt_off_f32_i4((int)(hi >> (8 * j) & 0xFFu));
        r[j] = (int)__builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
    return __builtin_bit_cast(bf16x8, r);
}
// Eight E2M1 codes of a dword times the power of two `scale`, as BF16.
__device__ __forceinline__ bf16x8 e2m1x8_to_bf16(int v, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((unsigned)v, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((unsigned)v, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((unsigned)v, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((unsigned)v, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

// RT: 16-row weight tiles per workgroup; gated: even tiles hold gate rows, odd
// ones the up rows of the same columns, and RT == 1 one tile of 8 gate and 8
// up rows (more workgroups for narrow weights).  KW: waves along K.  D: K
// blocks of a wave in registers.  GROUP: group size of 4-bit integers.  MB:
// blocks of 16 tokens (E4M3).
template <int FMT, bool GATED, int RT, int KW, int D, int GROUP, bool ZEROS, int MB = 1>
__global__ __launch_bounds__(64 * KW) void skinny_kernel(SkinnyParams p) {
    constexpr bool kMixed = GATED && RT == 1;
    constexpr int COLS = GATED ? 8 * RT : 16 * RT;      // output columns of a workgroup
    constexpr int WL = FMT == kSkinnyE4m3 ? 2 : 1;      // 16-byte weight loads per lane and block
    constexpr int XL = FMT == kSkinnyE4m3 ? 2 : 4;      // 16-byte x loads per lane and block
    constexpr bool kTranspose = FMT == kSkinnyInt4 && GROUP < 128;
    constexpr int NG = FMT == kSkinnyInt4 ? 128 / GROUP : 1;   // groups per block
    static_assert(!GATED || RT == 1 || RT % 2 == 0, "gate and up tiles in pairs");
    static_assert(MB == 1 || FMT == kSkinnyE4m3, "token blocks");
    __shared__ f32x4 sums[KW][RT * MB][64];

    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int64_t N = p.N;
    const int KB = (int)(p.K / 128);
    // workgroup b of a dispatch wave lands on XCD b % 8: each XCD takes a run of
    // consecutive rows, so that the lines of the scale tables (16 rows take a
    // part of one) are fetched into one L2 only
    const int G = gridDim.x, per = G / 8, rest = G % 8, xcd = blockIdx.x % 8;
    const int64_t n0 = (int64_t)(xcd * per + min(xcd, rest) + (int)(blockIdx.x / 8)) * COLS;

    // operand row of this lane in each tile (rows past N repeat the last one;
    // they are not stored)
    const uint8_t* wrow[RT][WL];
    const uint32_t* erow[RT];       // MXFP4: this lane's scale dwords
    const uint16_t* srow[RT];       // 4-bit integers: scales and zero points
    const uint8_t* zrow[RT];        // of group q % NG of a block
    const float* brow[RT];          // E4M3: the block scales of the lane's 4 result rows
    const int64_t row_bytes = FMT == kSkinnyE4m3 ? p.K : p.K / 2;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int wi = kMixed ? r >> 3 : GATED ? t & 1 : 0;
        auto row = [&](int i) FP8K_INLINE {
            return min(n0 + (kMixed ? i & 7 : 16 * (GATED ? t >> 1 : t) + i), N - 1);
        };
        const int64_t n = row(r);
        if constexpr (WL == 1) wrow[t][0] = p.w[wi] + n * row_bytes + 16 * q;
        else
#pragma unroll
            for (int i = 0; i < WL; ++i) wrow[t][i] = p.w[wi] + row((r & 14) + i) * row_bytes + 32 * q + 16 * (r & 1);
        erow[t] = reinterpret_cast<const uint32_t*>(p.s[wi]) + n;
        const int ri = kMixed ? q >> 1 : GATED ? t & 1 : 0;
        const int64_t nr = n0 + (kMixed ? 4 * (q & 1) : 16 * (GATED ? t >> 1 : t) + 4 * q);
        srow[t] = static_cast<const uint16_t*>(p.s[wi]) + (q % NG) * N + n;
        zrow[t] = ZEROS ? p.z[wi] + (q % NG) * N + n : nullptr;
        brow[t] = static_cast<const float*>(p.s[ri]) + (min(nr, N - 1) >> 7) * KB;
    }
    // x of this lane's token: 4-bit with whole-block groups and E4M3: the 32
    // elements 32q ..; transposed: elements 32 s + 8 q of step s.
    // A load whose neighbouring lanes read different rows takes a cycle per
    // lane, and x outweighs the weights of a workgroup with few tiles.  With
    // more than a few tokens (4-bit formats) the four lanes of a quad read 64
    // contiguous bytes, a token of the quad per load, and exchange them in
    // registers; the two lanes of a pair do so for E4M3 (and always for its
    // weights).  One MI355X, K 7168, us: MXFP4 16 x 500 10.5 -> 6.4, 1 x 500
    // 6.0 -> 6.4; int4 (128) 16 x 24576 27.9 -> 24.5, 1 x 500 6.4 -> 7.9; with
    // groups of 64, whose x is transposed once more, 16 x 500 11.6 -> 9.3, 1 x
    // 500 7.3 -> 9.6.  Gated E4M3 16 x 2048 10.2 -> 9.0, 48 x 2048 17.2 -> 13.3,
    // with the weights 1 x 2048 8.0 -> 7.5, 16 x 2048 -> 7.8, 48 x 2048 -> 12.0.
    const bool four = FMT == kSkinnyInt4 && p.M <= 4;   // token m in operand rows 4m .. 4m + 3
    const bool quads = MB > 1 || p.M > (kTranspose ? 8 : 4);
    const uint8_t* xrow[MB * XL];
    const float* sarow[MB];
    if constexpr (FMT == kSkinnyE4m3) {
#pragma unroll
        for (int c = 0; c < MB; ++c) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t m = min((int64_t)(16 * c + (quads ? (r & 14) + i : r)), p.M - 1);
                xrow[2 * c + i] = static_cast<const uint8_t*>(p.x) + m * p.K + 32 * q + 16 * (quads ? r & 1 : i);
            }
            sarow[c] = p.sa + min((int64_t)(16 * c + r), p.M - 1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int64_t m = min((int64_t)(quads ? 4 * (r >> 2) + i : four ? r >> 2 : r), p.M - 1);
            xrow[i] = static_cast<const uint8_t*>(p.x) + m * p.K * 2 +
                      (quads ? 64 * q + 16 * (r & 3) : kTranspose ? 16 * q + 64 * i : 64 * q + 16 * i);
        }
    }

    struct Block {
        i32x4 w[RT][WL];
        i32x4 x[MB][XL];
        uint32_t e[RT];             // MXFP4: scale dword of the operand row
        uint16_t s[RT];             // int4: BF16 scale and zero point of one group
        uint8_t z[RT];
        float sa[MB], sb[RT];       // E4M3: scales of the token and of the result rows
    };
    auto load = [&](Block& b, int kb) FP8K_INLINE {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
            for (int i = 0; i < WL; ++i)
                b.w[t][i] = *reinterpret_cast<const i32x4*>(wrow[t][i] + (int64_t)kb * 64 * WL);
            if constexpr (FMT == kSkinnyMxfp4) b.e[t] = erow[t][(int64_t)kb * N];
            if constexpr (FMT == kSkinnyE4m3) b.sb[t] = brow[t][kb];
            if constexpr (FMT == kSkinnyInt4) {
                const int64_t at = (int64_t)kb * NG * N;
                b.s[t] = srow[t][at];
                if constexpr (ZEROS) b.z[t] = zrow[t][at];
            }
        }
#pragma unroll
        for (int c = 0; c < MB; ++c) {
            if constexpr (FMT == kSkinnyE4m3) b.sa[c] = sarow[c][(int64_t)kb * p.M];
#pragma unroll
            for (int i = 0; i < XL; ++i)
                b.x[c][i] = *reinterpret_cast<const i32x4*>(xrow[XL * c + i] +
                                                            (int64_t)kb * (FMT == kSkinnyE4m3 ? 128 : 256));
        }
    };

    f32x4 acc[RT][MB];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < MB; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](Block& b) FP8K_INLINE {
        if constexpr (FMT == kSkinnyE4m3) {
#pragma unroll
            for (int t = 0; t < RT; ++t) swap_pair_lanes(b.w[t][0], b.w[t][1], lane);
            if (quads)
#pragma unroll
                for (int c = 0; c < MB; ++c) swap_pair_lanes(b.x[c][0], b.x[c][1], lane);
        } else
            if (quads) {
                transpose_quad_lanes(b.x[0], lane);
                if constexpr (kTranspose)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const i32x4 y = transpose_quads(i32x4{b.x[0][0][j], b.x[0][1][j], b.x[0][2][j], b.x[0][3][j]});
#pragma unroll
                        for (int i = 0; i < 4; ++i) b.x[0][i][j] = y[i];
                    }
            }
        if constexpr (FMT == kSkinnyE4m3) {
            f32x4 part[RT][MB];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                f16x8 xv[MB];
#pragma unroll
                for (int c = 0; c < MB; ++c)
                    xv[c] = e4m3x8_to_f16(b.x[c][s >> 1][2 * (s & 1)], b.x[c][s >> 1][2 * (s & 1) + 1]);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const f16x8 wv = e4m3x8_to_f16(b.w[t][s >> 1][2 * (s & 1)], b.w[t][s >> 1][2 * (s & 1) + 1]);
#pragma unroll
                    for (int c = 0; c < MB; ++c)
                        part[t][c] =
                            __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, xv[c], s ? part[t][c] : f32x4{}, 0, 0, 0);
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int c = 0; c < MB; ++c) {
                    const float f = b.sa[c] * b.sb[t];
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[t][c][v] = __builtin_fmaf(f, part[t][c][v], acc[t][c][v]);
                }
        } else if constexpr (FMT == kSkinnyMxfp4) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const bf16x8 xv = __builtin_bit_cast(bf16x8, b.x[0][s]);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    // the lane's 32 weights are group q: its scale byte as an FP32 exponent
                    const float sc = __uint_as_float((b.e[t] >> (8 * q) & 0xFFu) << 23);
                    acc[t][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e2m1x8_to_bf16(b.w[t][0][s], sc), xv, acc[t][0],
                                                                        0, 0, 0);
                }
            }
        } else {
            i32x4 wt[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) wt[t] = kTranspose ? transpose_quads(b.w[t][0]) : b.w[t][0];
            // the block's groups' scales (high half) and zero points, from the
            // lanes that loaded them to all
            uint32_t sz[RT][4];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                sz[t][0] = (uint32_t)b.s[t] << 16 | (ZEROS ? b.z[t] & 15u : 0u);
                if constexpr (NG == 4) {
                    const auto h = __builtin_amdgcn_permlane32_swap(sz[t][0], sz[t][0], false, false);
                    const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
                    const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
                    sz[t][0] = lo[0]; sz[t][1] = lo[1]; sz[t][2] = hi[0]; sz[t][3] = hi[1];
                } else if constexpr (NG == 2) {
                    const auto h = __builtin_amdgcn_permlane16_swap(sz[t][0], sz[t][0], false, false);
                    sz[t][0] = h[0]; sz[t][1] = h[1];
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 part[RT];
                float zero[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    part[t] = f32x4{};
                    zero[t] = (float)(sz[t][g] & 0xFFu);
                }
#pragma unroll
                for (int i = 0; i < 4 / NG; ++i) {
                    const int s = g * (4 / NG) + i;
                    const bf16x8 xv = __builtin_bit_cast(bf16x8, b.x[0][s]);
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            xv, ZEROS ? u4x8_less_zero_to_bf16(wt[t][s], zero[t]) : u4x8_less8_to_bf16(wt[t][s]), part[t],
                            0, 0, 0);
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const float sc = __uint_as_float(sz[t][g] & 0xFFFF0000u);
                    acc[t][0][0] = __builtin_fmaf(sc, part[t][0], acc[t][0][0]);
                    if (!four)
#pragma unroll
                        for (int v = 1; v < 4; ++v) acc[t][0][v] = __builtin_fmaf(sc, part[t][v], acc[t][0][v]);
                }
            }
        }
    };

    // This wave's blocks, D - 1 of them in flight ahead of the one multiplied:
    // every KW-th pair of blocks (the two 64-byte halves of a row's 128-byte
    // line, one right after the other), counted from a start that differs from
    // workgroup to workgroup, so that the workgroups, which all read the same
    // x, do not ask for the same lines at the same time.
    const int rot = (int)((unsigned)blockIdx.x * 6u % (unsigned)KB);
    const int pairs = (KB + 1) / 2, mine = pairs > wave ? (pairs - wave + KW - 1) / KW : 0;
    const int nb = 2 * mine - (mine && (KB & 1) && wave + (mine - 1) * KW == pairs - 1);
    auto block_of = [&](int j) FP8K_INLINE {
        const int kb = 2 * (wave + (j >> 1) * KW) + (j & 1) + rot;
        return kb < KB ? kb : kb - KB;
    };
    Block b[D];
#pragma unroll
    for (int j = 0; j < D - 1; ++j)
        if (j < nb) load(b[j], block_of(j));
    int at = 0;
    for (; at + 2 * D - 2 < nb; at += D) {      // every load of the round is one of a block
#pragma unroll
        for (int j = 0; j < D; ++j) {
            load(b[(j + D - 1) % D], block_of(at + j + D - 1));
            multiply(b[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 2 * D - 2; ++j) {
        if (at + j + D - 1 < nb) load(b[(j + D - 1) % D], block_of(at + j + D - 1));
        if (at + j < nb) multiply(b[j % D]);
    }

    // ---- join the waves' sums, in wave order; tile t by wave t % KW ----
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < MB; ++c) sums[wave][t * MB + c][lane] = acc[t][c];
    __syncthreads();
    auto total = [&](int t, int l) FP8K_INLINE {
        f32x4 v{};
        if constexpr (FMT == kSkinnyInt4) {
            // weights are the columns there: four lanes' sums of one token
            const int m = l & 15, from = (four ? 16 * (m & 3) : 16 * (m >> 2)) + 4 * (l >> 4), e = four ? 0 : m & 3;
            for (int w = 0; w < KW; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += sums[w][t][from + i][e];
            // (sums of 1/16 of the weights: what their subnormals lose, BF16 would too)
            if constexpr (!ZEROS) v *= 16.f;
        } else {
            for (int w = 0; w < KW; ++w) v += sums[w][t][l];
        }
        return v;
    };
    constexpr int OT = GATED ? (RT + 1) / 2 : RT;       // result tiles
    for (int o = wave; o < OT * MB; o += KW) {
        const int t = o / MB, c = o - t * MB;
        const int64_t m = 16 * c + r, n = n0 + 16 * t + 4 * q;
        auto store = [&](uint16_t* out, f32x4 v) FP8K_INLINE {
            const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
            if (n + 3 < N) {
                const uint2 all = make_uint2(lo, hi);
                __builtin_memcpy(out, &all, 8);
            } else {
                if (n < N) out[0] = (uint16_t)(lo & 0xFFFF);
                if (n + 1 < N) out[1] = (uint16_t)(lo >> 16);
                if (n + 2 < N) out[2] = (uint16_t)(hi & 0xFFFF);
                if (n + 3 < N) out[3] = (uint16_t)(hi >> 16);
            }
        };
        if constexpr (GATED) {
            if (kMixed && q >= 2) continue;             // the up rows' lanes
            const f32x4 g = total((kMixed ? 0 : 2 * t) * MB + c, lane);
            const f32x4 u = total((kMixed ? 0 : 2 * t + 1) * MB + c, kMixed ? lane + 32 : lane);
            if (m >= p.M) continue;
            if constexpr (FMT == kSkinnyE4m3) {
                if (p.part) {                           // N % 128 == 0
                    if (n < N) {
                        *reinterpret_cast<f32x4*>(p.part + m * N + n) = g;
                        *reinterpret_cast<f32x4*>(p.part + (p.M + m) * N + n) = u;
                    }
                    continue;
                }
                if (p.g) {
                    store(p.g + m * N + n, g);
                    store(p.u + m * N + n, u);
                }
            }
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = gated_act(p.act, g[i]) * u[i];
            store(p.y + m * N + n, v);
        } else {
            const f32x4 v = total(t, lane);
            if (m < p.M) store(p.y + m * N + n, v);
        }
    }
}

// ---------------------------------------------------------------------------
// 4-bit integer weights with group scales.  Asymmetric: lo = min(w, 0),
// hi = max(w, 0), s = BF16((hi - lo) / 15), z = round(-lo / s) in [0, 15];
// symmetric: s = BF16(amax / 7), z = 8; q = clamp(round(w / s) + z, 0, 15).
// All roundings to nearest, ties to even, quotients correctly rounded; the
// scale is at least BF16(1e-8), so a group of zeros is z everywhere.
// One group per 8 lanes of 4 elements (group 32), 16 or 32 lanes; a stream:
// 24576 x 7168 204-218 us, 7168 x 2048 20-24 (one MI355X: 3.7-3.9 and 2.8-3.4
// TB/s; with zero points the slower ones).
// ---------------------------------------------------------------------------
template <int GROUP>
__global__ __launch_bounds__(256) void quant_int4_kernel(const float* __restrict__ w, uint8_t* __restrict__ qd,
                                                         uint16_t* __restrict__ s, uint8_t* __restrict__ z,
                                                         int64_t N, int64_t K) {
    constexpr int L = GROUP / 4;                        // lanes per group
    const int64_t groups = K / GROUP;
    const int64_t id = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int64_t total = N * groups;
    const int64_t at = min(id, total - 1);              // whole sub-waves stay active for the shuffles
    const int64_t n = at / groups, g = at - n * groups;
    const int i = (int)(threadIdx.x % L);
    const f32x4 v = *reinterpret_cast<const f32x4*>(w + n * K + g * GROUP + 4 * i);
    float lo = fminf(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), 0.f);
    float hi = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), 0.f);
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, o, L));
        hi = fmaxf(hi, __shfl_xor(hi, o, L));
    }
    const float wide = z ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
    const uint32_t sb = pack_bf16x2(fmaxf(wide, 1e-8f), 0.f) & 0xFFFFu;
    const float sc = bf16_bits_to_f32(sb);
    const float zp = z ? fminf(fmaxf(rintf(-lo / sc), 0.f), 15.f) : 8.f;
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c |= (uint32_t)fminf(fmaxf(rintf(v[j] / sc) + zp, 0.f), 15.f) << (4 * j);
    if (id >= total) return;
    *reinterpret_cast<uint16_t*>(qd + (n * K + g * GROUP) / 2 + 2 * i) = (uint16_t)c;
    if (i == 0) {
        s[g * N + n] = (uint16_t)sb;
        if (z) z[g * N + n] = (uint8_t)zp;
    }
}

}  // namespace fp8k
