// kernels_adapter.h -- low-rank adapters of many requests beside one
// projection, for gfx950:
//   out[t] = y[t] + scale[a] * (x[t] A_a^T) B_a^T,  a the adapter of token t.
//
// The tokens come sorted by adapter in tiles of 16 rows (src: the token of a
// row or -1, index: its adapter), which is one dimension of the matrix
// instruction.  Two kernels:
//   down  z[row] = x[src[row]] A_a^T, K split over waves and workgroups where
//         the tiles are few; FP32 sums, one buffer per workgroup along K
//   up    the sums of z, scaled, times B_a^T, added to y and rounded once
// Both are bounded by memory: x, y and the adapters that occur are read once
// from memory (tiles of one adapter share them through the caches); the
// products are a few operations per byte.  z enters the second product as the
// sum of two BF16 values, which keeps 16 bits of it (one part would cost 2^-9
// of the added term) and costs only instructions that wait anyway.
//
// The index of a tile is that of its first row with a token; a row of another
// index is not computed.  Rows of an index outside the adapters take y as it is.
#pragma once

#include "rows_common.h"

namespace fp8k {

struct AdapterParams {
    const uint16_t* x;          // (T, K)
    const uint16_t* a;          // (L, R, K)
    const uint16_t* b;          // (L, N, R)
    const float* scale;         // (L)
    const int32_t* src;         // (16 tiles)
    const int32_t* index;       // (16 tiles)
    const uint16_t* y;          // (T, N)
    uint16_t* out;              // (T, N), may be y
    float* z;                   // [splits][16 tiles][R]
    int64_t T, N, K, tiles;
    int64_t k_range;            // elements of K per workgroup, a multiple of 128
    int64_t n_range;            // columns per workgroup of the second kernel
    int32_t L, R, splits;
};

constexpr int kAdapterMaxR = 128;

// A tile's rows: lane l holds row l % 16.
struct AdapterTile {
    int64_t token;              // of the lane's row, or of a row that has one
    int32_t index;              // of the tile
    bool any, valid;            // the tile has a token; the lane's row is one of the tile's index
};
__device__ __forceinline__ AdapterTile adapter_tile(const AdapterParams& p, int64_t tile, int lane) {
    AdapterTile t;
    const int64_t row = tile * 16 + (lane & 15);
    const int32_t src = tile < p.tiles ? p.src[row] : -1;
    const bool has = src >= 0 && src < p.T;
    const int32_t idx = has ? p.index[row] : -1;
    const uint64_t m = __ballot(has);
    t.any = m != 0;
    const int first = t.any ? __builtin_ctzll(m) : 0;
    t.index = __builtin_amdgcn_readlane(idx, first);
    t.valid = has && idx == t.index;
    const int32_t safe = __builtin_amdgcn_readlane(src, first);
    t.token = t.valid ? src : safe;
    return t;
}

// First kernel.  WK waves of a workgroup share a tile's K range, 4 / WK tiles.
// A step is 32 of K: lane l reads 16 bytes of token l % 16 (or of row l % 16
// of A) from element 8 (l / 16) on, four steps in flight.  Rows without a
// token read another row's and are not stored, rows of A behind R the last one's.
template <int RT, int WK>
__global__ __launch_bounds__(256) void adapter_down_kernel(AdapterParams p) {
    __shared__ float part[WK > 1 ? 3 : 1][RT][64][4];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t tile = WK > 1 ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
    const AdapterTile t = adapter_tile(p, tile, lane);
    const bool work = t.any && t.index >= 0 && t.index < p.L;
    if (WK > 1 && !work) return;            // (the whole workgroup)
    f32x4 acc[RT] = {};
    if (work) {
        const int64_t k0 = (int64_t)blockIdx.y * p.k_range, k1 = k0 + p.k_range < p.K ? k0 + p.k_range : p.K;
        const uint16_t* x = p.x + t.token * p.K + 8 * (lane >> 4);
        const uint16_t* a[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = 16 * r + (lane & 15);
            a[r] = p.a + ((int64_t)t.index * p.R + (row < p.R ? row : p.R - 1)) * p.K + 8 * (lane >> 4);
        }
        for (int64_t k = k0 + (WK > 1 ? wave * 128 : 0); k < k1; k += WK * 128) {
            bf16x8 xv[4], av[RT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[i] = *reinterpret_cast<const bf16x8*>(x + k + 32 * i);
#pragma unroll
                for (int r = 0; r < RT; ++r) av[r][i] = *reinterpret_cast<const bf16x8*>(a[r] + k + 32 * i);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[r][i], xv[i], acc[r], 0, 0, 0);
        }
    }
    if constexpr (WK > 1) {
        if (wave > 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[wave - 1][r][lane][i] = acc[r][i];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] += part[w][r][lane][i];
    }
    // lane l: token l % 16, elements 16 r + 4 (l / 16) + i
    if (!work || !t.valid) return;
    float* z = p.z + ((int64_t)blockIdx.y * p.tiles * 16 + tile * 16 + (lane & 15)) * p.R + 4 * (lane >> 4);
#pragma unroll
    for (int r = 0; r < RT; ++r)
        if (16 * r + 4 * (lane >> 4) < p.R) *reinterpret_cast<f32x4*>(z + 16 * r) = acc[r];
}

// Second kernel.  A wave forms 64 columns of a tile at a time: four products
// whose rows are the columns 16 (i / 4) + 4 j + i % 4 (i the row, j the
// product), so that a lane ends with 16 columns of one token in a row.
// RS: 32s of R.
template <int RS, bool SHARE>
__global__ __launch_bounds__(256) void adapter_up_kernel(AdapterParams p) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t tile = SHARE ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    const AdapterTile t = adapter_tile(p, tile, lane);
    if (!t.any) return;
    const bool adds = t.index >= 0 && t.index < p.L;
    if (!adds && p.out == p.y) return;
    const int g = lane >> 4;
    // z of the lane's token, elements 32 s + 8 g + 0..7, as two BF16 parts
    bf16x8 hi[RS], lo[RS];
    if (adds) {
        const float c = p.scale[t.index];
        const float* z = p.z + (tile * 16 + (lane & 15)) * p.R + 8 * g;
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            float f[8] = {};
            if (t.valid && 32 * s + 8 * g < p.R) {
                for (int i = 0; i < p.splits; ++i) {
                    const float* zi = z + (int64_t)i * p.tiles * 16 * p.R + 32 * s;
                    const f32x4 u = *reinterpret_cast<const f32x4*>(zi), v = *reinterpret_cast<const f32x4*>(zi + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[e] += u[e];
                        f[4 + e] += v[e];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = c * f[e];
                hi[s][e] = (__bf16)v;
                lo[s][e] = (__bf16)(v - (float)hi[s][e]);
            }
        }
    }
    const int64_t n_lo = (int64_t)blockIdx.y * p.n_range, n_end = n_lo + p.n_range < p.N ? n_lo + p.n_range : p.N;
    const int i0 = lane & 15;
    const uint16_t* b = p.b + (int64_t)(adds ? t.index : 0) * p.N * p.R + 8 * g;
    const uint16_t* y = p.y + t.token * p.N;
    uint16_t* out = p.out + t.token * p.N;
    for (int64_t n = n_lo + (SHARE ? 0 : wave * 64); n < n_end; n += SHARE ? 64 : 256) {
        f32x4 acc[4] = {};
        const int64_t c0 = n + 16 * g;      // the lane's first column
        i32x4 base[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (t.valid && c0 + 8 * h < p.N) base[h] = load_row16<uint16_t>(y + c0 + 8 * h, p.N - c0 - 8 * h);
        if (adds) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int64_t col = n + 16 * (i0 >> 2) + 4 * j + (i0 & 3);
                col = col < p.N ? col : p.N - 1;        // (not stored)
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    bf16x8 w{};
                    if (32 * s + 8 * g < p.R) w = *reinterpret_cast<const bf16x8*>(b + col * p.R + 32 * s);
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, hi[s], acc[j], 0, 0, 0);
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, lo[s], acc[j], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (t.valid && c0 + 8 * h < p.N) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = RowElem<uint16_t>::get(base[h], e) + acc[2 * h + (e >> 2)][e & 3];
                // (without an adapter y goes through as it is, the sign of a zero too)
                store_row16<uint16_t>(out + c0 + 8 * h, p.N - c0 - 8 * h, adds ? RowElem<uint16_t>::pack(f) : base[h]);
            }
        }
    }
}

}  // namespace fp8k
