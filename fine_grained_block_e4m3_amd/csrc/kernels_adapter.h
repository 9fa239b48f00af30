// kernels_adapter.h -- low-rank adapters of many requests beside one
// projection, for gfx950:
//   out[t] = y[t] + scale[a] * (x[t] A_a^T) B_a^T,  a the adapter of token t.
//
// The tokens come sorted by adapter in tiles of 16 rows (src: the token of a
// row or -1, index: its adapter), which is one dimension of the matrix
// instruction.  Three forms:
//   whole   one kernel, a few workgroups per tile that each form z = x A^T of
//           their tokens by dot products: a token or two per adapter
//   tiles   two kernels: the first forms z, K split over waves and workgroups,
//           the second adds z's sums, multiplies by B^T and adds y, N split; a
//           workgroup per tile and split.  Few tokens per adapter: A and B are
//           most of what is read, and the operands come straight into registers
//   groups  the two kernels with a workgroup per four tiles, which mostly share
//           an adapter: x and y are most of what is read, in whole 128-byte
//           pieces of their rows through LDS.
// (The matrix instruction's layout, 16 rows of 64 bytes per load, comes at 36
// GB/s per compute unit from L2, pieces of 128 bytes at 80, whole kilobytes at
// 105, measured: that is why whole multiplies by rows, and why many tokens go
// through LDS.)
// All are bounded by memory otherwise; the products are a few operations per
// byte.  z enters the second product as the sum of three BF16 values, which hold
// all of an FP32 value (one could cost 2^-8 of the added term, two 2^-16); they
// cost matrix instructions where the kernels wait for memory.
//
// Measured (one MI355X, K 7168): 1 token, R 16, N 2048 6.1 us (one kernel); 100
// tokens of 64 adapters, N 2112 10.0 (one kernel); 8192 tokens of 8, R 64, N 2048 28 + 26
// (two; 4.2 and 3.1 TB/s).
//
// The index of a tile is that of its first row with a token; a row of another
// index is not computed.  Rows of an index outside the adapters take y as it is.
#pragma once

#include "gemm_common.h"
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
    int64_t k_range;            // elements of K per workgroup of the first kernel, a multiple of 128
    int64_t n_range;            // columns per workgroup of the second kernel, a multiple of 256
    int32_t L, R;
    int32_t splits, parts;      // workgroups along K and along N
};

constexpr int kAdapterMaxR = 128;

// A tile's rows: lane l holds row l % 16.
struct AdapterTile {
    int64_t token;              // of the lane's row, or of a row that has one
    int32_t index;              // of the tile
    bool any;                   // the tile has a token
    bool adds;                  // and its index is an adapter
    bool valid;                 // the lane's row is one of the tile's index
};
__device__ __forceinline__ AdapterTile adapter_tile(const AdapterParams& p, int64_t tile, int lane) {
    AdapterTile t;
    const int64_t row = (tile < p.tiles ? tile : 0) * 16 + (lane & 15);
    const int32_t src = p.src[row], idx = p.index[row];
    const bool has = tile < p.tiles && src >= 0 && src < p.T;
    const uint64_t m = __ballot(has);
    t.any = m != 0;
    const int first = t.any ? __builtin_ctzll(m) : 0;
    t.index = __builtin_amdgcn_readlane(idx, first);
    t.adds = t.any && t.index >= 0 && t.index < p.L;
    t.valid = has && idx == t.index;
    const int32_t safe = __builtin_amdgcn_readlane(src, first);
    t.token = t.valid ? src : safe;
    return t;
}

// First product.  A step is 32 of K: lane l reads 16 bytes of token l % 16 (and
// of row l % 16 of each 16 of A) from element 8 (l / 16) on.  Lanes whose row
// has no token read another row's and are not used (leaving them out saves
// nothing that could be measured), rows of A behind R the last one's.  The
// lane's results are elements 16 r + 4 (l / 16) + i of token l % 16.
__device__ __forceinline__ const uint16_t* adapter_x(const AdapterParams& p, const AdapterTile& t, int lane) {
    return p.x + t.token * p.K + 8 * (lane >> 4);
}
__device__ __forceinline__ const uint16_t* adapter_a(const AdapterParams& p, const AdapterTile& t, int r, int lane) {
    const int row = 16 * r + (lane & 15);
    return p.a + ((int64_t)t.index * p.R + (row < p.R ? row : p.R - 1)) * p.K + 8 * (lane >> 4);
}
__device__ __forceinline__ bf16x8 load_bf16x8(const uint16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

// z over the chunks of 32 G elements c, c + step, ..., below `end`; the next
// chunk's loads are under way while one is multiplied.
template <int RT, int G>
__device__ __forceinline__ void adapter_down(const uint16_t* x, const uint16_t* const (&a)[RT], int64_t c, int64_t step,
                                             int64_t end, f32x4 (&acc)[RT]) {
    bf16x8 xv[2][G], av[2][G][RT];
    auto load = [&](int h, int64_t at) FP8K_INLINE {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int64_t k = at * (32 * G) + 32 * i;
            xv[h][i] = load_bf16x8(x + k);
#pragma unroll
            for (int r = 0; r < RT; ++r) av[h][i][r] = load_bf16x8(a[r] + k);
        }
    };
    auto multiply = [&](int h) FP8K_INLINE {
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int r = 0; r < RT; ++r)
                acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[h][i][r], xv[h][i], acc[r], 0, 0, 0);
    };
    if (c >= end) return;
    load(0, c);
    for (;;) {
        if (c + step >= end) {
            multiply(0);
            return;
        }
        load(1, c + step);
        multiply(0);
        c += 2 * step;
        if (c >= end) {
            multiply(1);
            return;
        }
        load(0, c);
        multiply(1);
    }
}

// Second product.  B's rows are the columns col(j), j = 0..3, of the lane's row
// of each of four products.  RS: 32s of R.
template <int RS, typename F>
__device__ __forceinline__ void adapter_b_load(const AdapterParams& p, int32_t index, F col, int g, bf16x8 (&w)[4][RS]) {
    const uint16_t* b = p.b + (int64_t)index * p.N * p.R;
    int at[RS];                             // (lanes whose elements lie behind R load others, times a z of 0 ...)
#pragma unroll
    for (int s = 0; s < RS; ++s) at[s] = 32 * s + 8 * g < p.R ? 32 * s + 8 * g : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t c = col(j) < p.N ? col(j) : p.N - 1;      // (not stored)
#pragma unroll
        for (int s = 0; s < RS; ++s) w[j][s] = load_bf16x8(b + c * p.R + at[s]);
    }
    // ... which an infinity there would make a NaN
#pragma unroll
    for (int s = 0; s < RS; ++s)
        if (32 * s + 32 > p.R) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (32 * s + 8 * g >= p.R) w[j][s] = bf16x8{};
        }
}
template <int RS>
__device__ __forceinline__ void adapter_multiply(const bf16x8 (&w)[4][RS], const bf16x8 (&z)[RS][3], f32x4 (&acc)[4]) {
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j][s], z[s][h], acc[j], 0, 0, 0);
}

// The scaled z of the lane's token, elements 32 s + 8 (l / 16) + 0..7, as three
// BF16 parts, each the next eight bits of it, cut: together all 24 of an FP32
// value.  (Two parts left 2^-16 of it, which shows where y takes away the
// leading bits of what is added.)  No finite value becomes an infinity by the
// cut; an infinity or NaN stands in the first part alone.  Elements behind R
// take a scale of 0, as an infinite one would make NaN of their zeros.
__device__ __forceinline__ void adapter_parts(const float (&f)[8], float scale, bf16x8 (&z)[3]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float v = scale * f[e];
        const bool finite = __builtin_isfinite(v);
#pragma unroll
        for (int h = 0; h < 3; ++h) {
            const float cut = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
            z[h][e] = __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(v) >> 16));
            v = h == 0 && !finite ? 0.f : v - cut;
        }
    }
}

template <int RT, int G>
__global__ __launch_bounds__(256) void adapter_down_kernel(AdapterParams p) {
    __shared__ __attribute__((aligned(16))) float part[3][RT][64][4];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t tile = blockIdx.x / p.splits, split = blockIdx.x - tile * p.splits;
    const AdapterTile t = adapter_tile(p, tile, lane);
    if (!t.adds) return;                    // (the whole workgroup)
    f32x4 acc[RT] = {};
    const int64_t k0 = split * p.k_range, k1 = k0 + p.k_range < p.K ? k0 + p.k_range : p.K;
    const uint16_t* a[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) a[r] = adapter_a(p, t, r, lane);
    adapter_down<RT, G>(adapter_x(p, t, lane), a, k0 / (32 * G) + wave, 4, k1 / (32 * G), acc);
    if (wave > 0) {
#pragma unroll
        for (int r = 0; r < RT; ++r) *reinterpret_cast<f32x4*>(part[wave - 1][r][lane]) = acc[r];
    }
    __syncthreads();
    if (wave > 0 || !t.valid) return;
    float* z = p.z + (split * p.tiles * 16 + tile * 16 + (lane & 15)) * p.R + 4 * (lane >> 4);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int w = 0; w < 3; ++w) acc[r] += *reinterpret_cast<const f32x4*>(part[w][r][lane]);
        if (16 * r + 4 * (lane >> 4) < p.R) *reinterpret_cast<f32x4*>(z + 16 * r) = acc[r];
    }
}

// z of groups of four tiles: a product of 64 rows of x with A's R rows, K in
// chunks of CHUNK elements.  Both come into registers in whole 256-byte (128-byte)
// pieces of their rows, A one chunk ahead and x XD - 1, and from there as the
// matrix instruction's operands through LDS: a wave's 16 rows of x for itself,
// A, which all waves share, in two places in turn.  A group of several adapters
// goes through K once for each.
// Three chunks of x in registers at R 33 to 64, two at others, and chunks of 64
// above 64, measured (K 7168, 8192 tokens, us): R 64 two 35.2, three 32.2, chunks
// of 64 33.4; R 16 26.7, 27.3, 31.1; R 128 29.8, 30.6 and in chunks of 128 39.8.  With x
// straight in the operands' layout, 16 rows of 64 bytes per load, R 64 35.3, R 16
// 28.0; through LDS by direct loads, three stages of 64 elements of x and A 34.6, 28.9.
// LDS row of 2 CHUNK bytes: its 16-byte pieces at place piece ^ adapter_swz(row).
template <int CHUNK>
__device__ __forceinline__ int adapter_swz(int row) {       // 16 rows at one piece cover all banks
    return CHUNK == 128 ? row & 15 : (row >> 1) & 7;
}
template <int RT, int CHUNK, int XD>
__global__ __launch_bounds__(256, RT <= 4 ? 4 : 2) void adapter_down_group_kernel(AdapterParams p, int64_t groups) {
    constexpr int PIECES = CHUNK / 8, ROW = 2 * CHUNK;
    constexpr int XROWS = 64 / PIECES, XN = 16 / XROWS;             // rows of a wave's load of x, and its loads
    constexpr int AROWS = 256 / PIECES, AN = (16 * RT + AROWS - 1) / AROWS;
    constexpr int STAGE = AN * AROWS * ROW;
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE + 64 * ROW];
    __shared__ int32_t adapter[4];          // of the tiles, -1: none
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t per = (groups * p.splits + 7) / 8, work = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= per || work >= groups * p.splits) return;
    const int64_t group = work / p.splits, split = work - group * p.splits;
    const AdapterTile t = adapter_tile(p, group * 4 + wave, lane);
    if (lane == 0) adapter[wave] = t.adds ? t.index : -1;
    __syncthreads();
    const int64_t k0 = split * p.k_range, k1 = k0 + p.k_range < p.K ? k0 + p.k_range : p.K;
    const int chunks = (int)((k1 - k0) / CHUNK);
    const int piece = threadIdx.x % PIECES;         // the thread's, of row x_row of every XROWS and a_row of every AROWS
    const int x_row = lane / PIECES, a_row = threadIdx.x / PIECES;
    uint8_t* xs = smem + 2 * STAGE + wave * 16 * ROW;
    const uint16_t* x[XN];
#pragma unroll
    for (int j = 0; j < XN; ++j)
        x[j] = p.x + (int64_t)__shfl((int)t.token, XROWS * j + x_row) * p.K + k0 + 8 * piece;
    f32x4 acc[RT] = {};
    int of[4], todo = 0;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        of[m] = uniform(adapter[m]);
        todo |= of[m] >= 0 ? 1 << m : 0;
    }
    while (todo) {
        int index = 0;                      // this pass's adapter
#pragma unroll
        for (int m = 3; m >= 0; --m)
            if (todo >> m & 1) index = of[m];
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (of[m] == index) todo &= ~(1 << m);
        const bool mine = t.adds && t.index == index;
        const uint16_t* a[AN];
#pragma unroll
        for (int j = 0; j < AN; ++j) {
            const int row = AROWS * j + a_row;
            a[j] = p.a + ((int64_t)index * p.R + (row < p.R ? row : p.R - 1)) * p.K + k0 + 8 * piece;
        }
        bf16x8 av[AN], xv[XD][XN];
        auto load_a = [&](int c) FP8K_INLINE {
#pragma unroll
            for (int j = 0; j < AN; ++j) av[j] = load_bf16x8(a[j] + (int64_t)c * CHUNK);
        };
        auto load_x = [&](int h, int c) FP8K_INLINE {
#pragma unroll
            for (int j = 0; j < XN; ++j) xv[h][j] = load_bf16x8(x[j] + (int64_t)c * CHUNK);
        };
        auto put = [&](uint8_t* rows, int row, bf16x8 v) FP8K_INLINE {
            *reinterpret_cast<bf16x8*>(rows + row * ROW + 16 * (piece ^ adapter_swz<CHUNK>(row))) = v;
        };
        auto get = [&](const uint8_t* rows, int row, int s) FP8K_INLINE {
            return *reinterpret_cast<const bf16x8*>(rows + row * ROW + 16 * ((4 * s + (lane >> 4)) ^ adapter_swz<CHUNK>(row)));
        };
        load_a(0);
        if (mine) {
#pragma unroll
            for (int u = 0; u < XD - 1; ++u)
                if (u < chunks) load_x(u, u);
        }
        for (int c0 = 0; c0 < chunks; c0 += XD) {
#pragma unroll
            for (int u = 0; u < XD; ++u) {
                const int c = c0 + u;
                if (c >= chunks) break;
                uint8_t* as = smem + (c & 1) * STAGE;       // (read two chunks ago, before the last barrier)
#pragma unroll
                for (int j = 0; j < AN; ++j) put(as, AROWS * j + a_row, av[j]);
                if (mine) {
#pragma unroll
                    for (int j = 0; j < XN; ++j) put(xs, XROWS * j + x_row, xv[u][j]);
                }
                if (c + 1 < chunks) load_a(c + 1);
                if (mine && c + XD - 1 < chunks) load_x((u + XD - 1) % XD, c + XD - 1);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // (the last chunk's reads too)
                lds_barrier();
                if (mine) {
#pragma unroll
                    for (int s = 0; s < CHUNK / 32; ++s) {
                        const bf16x8 v = get(xs, lane & 15, s);
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(get(as, 16 * r + (lane & 15), s), v, acc[r], 0, 0, 0);
                    }
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        lds_barrier();                      // (before another pass's first chunk)
    }
    if (!t.adds || !t.valid) return;
    float* z = p.z + (split * p.tiles * 16 + (group * 4 + wave) * 16 + (lane & 15)) * p.R + 4 * (lane >> 4);
#pragma unroll
    for (int r = 0; r < RT; ++r)
        if (16 * r + 4 * (lane >> 4) < p.R) *reinterpret_cast<f32x4*>(z + 16 * r) = acc[r];
}

// The sum of eight elements of z over the splits.
__device__ __forceinline__ void adapter_z_sum(const AdapterParams& p, int64_t row, int e0, float (&f)[8]) {
    const float* z = p.z + row * p.R + e0;
    const int64_t next = p.tiles * 16 * p.R;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    // (eight splits' loads at a time)
    for (int i0 = 0; i0 < p.splits; i0 += 8) {
        f32x4 u[8][2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u[i][h] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (i0 + i < p.splits) u[i][h] = *reinterpret_cast<const f32x4*>(z + (i0 + i) * next + 4 * h);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += u[i][e >> 2][e & 3];
    }
}

// Second kernel for a tile: 64 columns at a time, by four products whose rows
// are the columns 16 (i / 4) + 4 j + i % 4 (i the row, j the product), so that a
// lane ends with 16 columns in a row of token l % 16.
template <int RS>
__device__ __forceinline__ void adapter_up_load(const AdapterParams& p, const AdapterTile& t, int64_t n, int lane,
                                                bf16x8 (&w)[4][RS], i32x4 (&base)[2]) {
    const int g = lane >> 4, i = lane & 15;
    if (t.adds) adapter_b_load<RS>(p, t.index, [&](int j) FP8K_INLINE { return n + 16 * (i >> 2) + 4 * j + (i & 3); }, g, w);
    const int64_t c0 = n + 16 * g;
    const uint16_t* y = p.y + t.token * p.N + c0;
    if (n + 64 <= p.N) {                    // (lanes without a token of their own read another's)
#pragma unroll
        for (int h = 0; h < 2; ++h) __builtin_memcpy(&base[h], y + 8 * h, 16);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            base[h] = i32x4{0, 0, 0, 0};
            if (c0 + 8 * h < p.N) base[h] = load_row16<uint16_t>(y + 8 * h, p.N - c0 - 8 * h);
        }
    }
}
template <int RS>
__device__ __forceinline__ void adapter_up_store(const AdapterParams& p, const AdapterTile& t, int64_t n, int lane,
                                                 const bf16x8 (&w)[4][RS], const bf16x8 (&z)[RS][3], const i32x4 (&base)[2]) {
    f32x4 acc[4] = {};
    if (t.adds) adapter_multiply<RS>(w, z, acc);
    if (!t.valid) return;
    const int64_t c0 = n + 16 * (lane >> 4);
    uint16_t* out = p.out + t.token * p.N + c0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = RowElem<uint16_t>::get(base[h], e) + acc[2 * h + (e >> 2)][e & 3];
        // (without an adapter y goes through as it is, the sign of a zero too)
        const i32x4 v = t.adds ? RowElem<uint16_t>::pack(f) : base[h];
        if (n + 64 <= p.N) __builtin_memcpy(out + 8 * h, &v, 16);
        else if (c0 + 8 * h < p.N) store_row16<uint16_t>(out + 8 * h, p.N - c0 - 8 * h, v);
    }
}

template <int RS>
__global__ __launch_bounds__(256) void adapter_up_kernel(AdapterParams p) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, i = lane & 15;
    const int64_t tile = blockIdx.x / p.parts, n_lo = (blockIdx.x - tile * p.parts) * p.n_range;
    const int64_t n_end = n_lo + p.n_range < p.N ? n_lo + p.n_range : p.N, n0 = n_lo + wave * 64;
    if (n0 >= n_end) return;
    const AdapterTile t = adapter_tile(p, tile, lane);
    if (!t.any || (!t.adds && p.out == p.y)) return;
    bf16x8 w[4][RS], z[RS][3];
    i32x4 base[2];
    adapter_up_load<RS>(p, t, n0, lane, w, base);
    if (t.adds) {
        const float c = p.scale[t.index];
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            float f[8] = {};
            if (t.valid && 32 * s + 8 * g < p.R) adapter_z_sum(p, tile * 16 + i, 32 * s + 8 * g, f);
            adapter_parts(f, 32 * s + 8 * g < p.R ? c : 0.f, z[s]);
        }
    }
    for (int64_t n = n0; n < n_end; n += 256) {
        if (n > n0) adapter_up_load<RS>(p, t, n, lane, w, base);
        adapter_up_store<RS>(p, t, n, lane, w, z, base);
    }
}

// One kernel for few tokens per adapter: `parts` workgroups per tile (a power of
// two) share its tokens, then N, and each forms z of its tokens for itself: A is
// read as often, but from its die's L2, and no z goes through memory, which
// costs a second launch and 2 us.  16 waves, one workgroup per compute unit.
//
// z by dot products over whole kilobytes of A's rows: a wave takes eight rows
// and every KP-th 512 elements, NT tokens at a time, and leaves its sums in
// zs[kp][row of the tile][R].
__device__ __forceinline__ float add_across(float a, float b, bool half) {
    // lanes below: a of both halves; lanes above: b (of 64 lanes, or of each 32)
    const auto s = half ? __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false)
                        : __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
template <int CTRL>
__device__ __forceinline__ float lane_shift(float f) {
    return __uint_as_float(lane_shift0<CTRL, 0xF>(__float_as_uint(f)));
}
template <int NT>
__device__ __forceinline__ void adapter_dots(const AdapterParams& p, const uint16_t* a, const int (&row)[NT],
                                             const int (&token)[NT], int kp, int KP, int r0, int lane, float* zs) {
    float acc[NT][8] = {};
    for (int64_t c = (int64_t)kp * 512; c < p.K; c += (int64_t)KP * 512) {
        const bool in = c + 8 * lane < p.K;
        const int64_t k = in ? c + 8 * lane : 0;
        bf16x8 av[8], xv[NT];
#pragma unroll
        for (int r = 0; r < 8; ++r) av[r] = load_bf16x8(a + r * p.K + k);
#pragma unroll
        for (int q = 0; q < NT; ++q) xv[q] = load_bf16x8(p.x + (int64_t)token[q] * p.K + k);
        if (!in) {                          // (both: zero times an infinity is no zero)
#pragma unroll
            for (int r = 0; r < 8; ++r) av[r] = bf16x8{};
#pragma unroll
            for (int q = 0; q < NT; ++q) xv[q] = bf16x8{};
        }
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    acc[q][r] = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{av[r][e], av[r][e + 1]}, bf16x2{xv[q][e], xv[q][e + 1]},
                                                                acc[q][r], false);
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        // sums over the lanes, halving the rows that a lane holds: row lane / 8 in the end
        float u[4], v[2];
#pragma unroll
        for (int r = 0; r < 4; ++r) u[r] = add_across(acc[q][r], acc[q][r + 4], true);
#pragma unroll
        for (int r = 0; r < 2; ++r) v[r] = add_across(u[r], u[r + 2], false);
        const bool upper = lane & 8;
        float f = (upper ? v[1] : v[0]) + lane_shift<0x128>(upper ? v[0] : v[1]);   // lane ^ 8
        f += lane_shift<0x141>(f);          // mirrored in 8 lanes
        f += lane_shift<0x4E>(f);           // lane ^ 2
        f += lane_shift<0xB1>(f);           // lane ^ 1
        if ((lane & 7) == 0) zs[(kp * 16 + row[q]) * p.R + r0 + (lane >> 3)] = f;
    }
}

constexpr int kWholeWaves = 16;

template <int RS>
__global__ __launch_bounds__(64 * kWholeWaves) void adapter_whole_kernel(AdapterParams p) {
    __shared__ __attribute__((aligned(16))) float zs[kWholeWaves * 16 * 8];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, i = lane & 15;
    // (a tile's workgroups on one die, whose L2 then holds the adapter)
    const int part = (int)(blockIdx.x >> 3) & (p.parts - 1);
    const int64_t tile = (int64_t)((blockIdx.x >> 3) >> __builtin_ctz(p.parts)) * 8 + (blockIdx.x & 7);
    AdapterTile t = adapter_tile(p, tile, lane);
    if (!t.any || (!t.adds && p.out == p.y)) return;
    // Shares of the tokens, each over parts / shares parts of N: the cheapest of
    // the powers of two.  Cost of a compute unit (measured, in units of R / 8.6 ps):
    // 28 per 1024 columns times 1024, and per element of K 12 for four tokens,
    // 7, 9 and 12 for one to three.
    const uint32_t all = (uint32_t)__ballot(t.valid) & 0xFFFFu;
    const int log_parts = __builtin_ctz(p.parts), count = __builtin_popcount(all);
    int log_shares = 0;
    float least = INFINITY;
    for (int l = 0; l <= log_parts; ++l) {
        const int each = (count + (1 << l) - 1) >> l, rest = each & 3;
        const int columns = 10 + log_parts - l;         // log2 of those that a share's parts do at once
        const float cost = (float)p.K * (float)(each / 4 * 12 + (rest ? (5 + 2 * rest + rest / 3) : 0)) +
                           (float)((p.N + (1ll << columns) - 1) >> columns) * (28.f * 1024.f);
        if (cost < least) {
            least = cost;
            log_shares = l;
        }
    }
    const int shares = 1 << log_shares;
    t.valid = t.valid && ((__builtin_popcount(all & ((1u << i) - 1)) ^ part) & (shares - 1)) == 0;
    uint32_t left = (uint32_t)__ballot(t.valid) & 0xFFFFu;
    if (!left) return;
    const int log_range = 6 + log_parts - log_shares;
    const int64_t n_range = (p.N + (1ll << log_range) - 1) >> log_range << 6, n_lo = (part >> log_shares) * n_range;
    const int64_t n_end = n_lo + n_range < p.N ? n_lo + n_range : p.N;
    const int blocks = p.R / 8, KP = kWholeWaves / blocks;
    if (t.adds && wave < KP * blocks) {
        const int kp = wave / blocks, r0 = 8 * (wave - kp * blocks);
        const uint16_t* a = p.a + ((int64_t)t.index * p.R + r0) * p.K;
        auto next = [&](int& row, int& token) FP8K_INLINE {
            if (left) {                     // (the last one twice)
                row = __builtin_ctz(left);
                token = __builtin_amdgcn_readlane((int)t.token, row);
                left &= left - 1;
            }
        };
        while (left) {
            const int n = __builtin_popcount(left);
            int row[4] = {}, token[4] = {};
            if (n == 1) {
                next(row[0], token[0]);
                adapter_dots<1>(p, a, {row[0]}, {token[0]}, kp, KP, r0, lane, zs);
            } else if (n == 2) {
                next(row[0], token[0]);
                next(row[1], token[1]);
                adapter_dots<2>(p, a, {row[0], row[1]}, {token[0], token[1]}, kp, KP, r0, lane, zs);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q > 0) row[q] = row[q - 1], token[q] = token[q - 1];
                    next(row[q], token[q]);
                }
                adapter_dots<4>(p, a, row, token, kp, KP, r0, lane, zs);
            }
        }
    }
    bf16x8 w[4][RS], z[RS][3];
    i32x4 base[2];
    int64_t n = n_lo + 64 * wave;
    if (n < n_end) adapter_up_load<RS>(p, t, n, lane, w, base);
    __syncthreads();
    if (n >= n_end) return;
    if (t.adds) {
        const float c = p.scale[t.index];
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            float f[8] = {};
            const int e0 = 32 * s + 8 * g;
            if (e0 < p.R && t.valid) {
#pragma unroll 4
                for (int k = 0; k < KP; ++k) {
                    const float* sum = zs + (k * 16 + i) * p.R + e0;
                    const f32x4 u = *reinterpret_cast<const f32x4*>(sum), v = *reinterpret_cast<const f32x4*>(sum + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] += e < 4 ? u[e] : v[e - 4];
                }
            }
            adapter_parts(f, e0 < p.R ? c : 0.f, z[s]);
        }
    }
    while (n < n_end) {
        adapter_up_store<RS>(p, t, n, lane, w, z, base);
        n += 64 * kWholeWaves;
        if (n < n_end) adapter_up_load<RS>(p, t, n, lane, w, base);
    }
}

// Second kernel for a group: z's parts of its 64 rows lie in LDS; a wave forms
// 64 columns of the four tiles, B's loads shared by tiles of one adapter, and
// each tile's results change places in LDS so that 8 lanes hold 64 columns of a
// row and y is read and written in whole 128-byte pieces.  STREAM: those are
// whole cache lines, read and written with the nontemporal hint (8192 tokens,
// N 2048, both kernels, three sets of x, y and out in turn: R 64 64.4 us without,
// 57.9 with it, R 16 51.6, 44.9, R 128 104.3, 97.6; 3000 tokens, R 64 31.5, 30.4).
// Eight waves above R 32, so that z, 64 R values per split for each workgroup,
// is read half as often (both kernels, four waves / eight, us: R 64, 8192 tokens,
// N 2048 54.0 / 51.7, 4000, N 7168 58.3 / 48.7; R 128 80.5 / 79.8; R 32 41.3 / 42.5, R 16
// 39.3 / 40.2: four there).
constexpr int adapter_up_waves(int RS) { return RS == 1 ? 4 : 8; }

template <int RS, bool STREAM>
__global__ __launch_bounds__(64 * adapter_up_waves(RS), RS <= 2 ? 4 : 2) void adapter_up_group_kernel(AdapterParams p, int64_t groups) {
    constexpr int ZROW = 32 * RS + 8;       // elements; 16 rows at one place cover all banks
    constexpr int DROW = 68, WAVES = adapter_up_waves(RS);
    __shared__ __attribute__((aligned(16))) uint16_t zp[3][64][ZROW];
    __shared__ __attribute__((aligned(16))) float ds[WAVES][16][DROW];
    __shared__ int32_t token[64], adapter[4];       // -1: none
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, i = lane & 15;
    const int64_t per = (groups * p.parts + 7) / 8, work = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= per || work >= groups * p.parts) return;
    const int64_t group = work / p.parts, n_lo = (work - group * p.parts) * p.n_range;
    const int64_t n_end = n_lo + p.n_range < p.N ? n_lo + p.n_range : p.N;
    if (wave < 4) {
        const AdapterTile t = adapter_tile(p, group * 4 + wave, lane);
        if (lane < 16) token[16 * wave + lane] = t.valid ? (int32_t)t.token : -1;
        if (lane == 0) adapter[wave] = t.adds ? t.index : -1;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 64 * 4 * RS; k += 64 * WAVES) {
        const int row = k / (4 * RS), e0 = 8 * (k % (4 * RS)), a = adapter[row >> 4];
        float f[8] = {};
        bf16x8 z[3];
        if (a >= 0 && token[row] >= 0 && e0 < p.R) adapter_z_sum(p, group * 64 + row, e0, f);
        adapter_parts(f, a >= 0 && e0 < p.R ? p.scale[a] : 0.f, z);
#pragma unroll
        for (int h = 0; h < 3; ++h) *reinterpret_cast<bf16x8*>(&zp[h][row][e0]) = z[h];
    }
    __syncthreads();
    const int r8 = lane >> 3, c8 = 8 * (lane & 7);      // the lane's rows r8 and r8 + 8, and its columns
    for (int64_t n = n_lo + wave * 64; n < n_end; n += 64 * WAVES) {
        const bool full = n + 64 <= p.N;
        i32x4 base[4][2];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // (a row without a token reads another's)
                const uint16_t* y = p.y + (int64_t)max(token[16 * m + 8 * h + r8], 0) * p.N + n + c8;
                if (full) {
                    base[m][h] = load_row16<uint16_t, STREAM>(y, 8);
                } else {
                    base[m][h] = i32x4{0, 0, 0, 0};
                    if (n + c8 < p.N) base[m][h] = load_row16<uint16_t>(y, p.N - n - c8);
                }
            }
        bf16x8 w[4][RS];
        int held = -1;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int a = uniform(adapter[m]);
            if (a >= 0) {
                if (a != held) {
                    adapter_b_load<RS>(p, a, [&](int j) FP8K_INLINE { return n + 16 * j + i; }, g, w);
                    held = a;
                }
                bf16x8 z[RS][3];
#pragma unroll
                for (int s = 0; s < RS; ++s)
#pragma unroll
                    for (int h = 0; h < 3; ++h) z[s][h] = *reinterpret_cast<const bf16x8*>(&zp[h][16 * m + i][32 * s + 8 * g]);
                f32x4 acc[4] = {};
                adapter_multiply<RS>(w, z, acc);
                // (the wave's own buffer: its LDS operations run in order)
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4*>(&ds[wave][i][16 * j + 4 * g]) = acc[j];
                __builtin_amdgcn_wave_barrier();
            } else if (p.out == p.y) {
                continue;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = token[16 * m + 8 * h + r8];
                i32x4 v = base[m][h];
                if (a >= 0) {
                    const f32x4 d0 = *reinterpret_cast<const f32x4*>(&ds[wave][8 * h + r8][c8]);
                    const f32x4 d1 = *reinterpret_cast<const f32x4*>(&ds[wave][8 * h + r8][c8 + 4]);
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = RowElem<uint16_t>::get(base[m][h], e) + (e < 4 ? d0[e] : d1[e - 4]);
                    v = RowElem<uint16_t>::pack(f);
                }
                uint16_t* out = p.out + (int64_t)t * p.N + n + c8;
                if (t >= 0) {
                    if (full) store_row16<uint16_t, STREAM>(out, 8, v);
                    else if (n + c8 < p.N) store_row16<uint16_t>(out, p.N - n - c8, v);
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

}  // namespace fp8k
