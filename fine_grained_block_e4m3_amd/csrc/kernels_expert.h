// kernels_expert.h -- tokens sorted by expert and back, with the gradients,
// for gfx950.  A pair p = t * k + j is token t's j-th expert; pos[p] is its row
// in the experts' buffer (-1: none), src[row] the pair of a row (-1: none).
//   sort       row = start of the expert's segment + number of earlier pairs
//              of the expert (a stable counting sort)
//   dispatch   xs[pos[t][j]] = x[t], as it is or as E4M3 codes and 1x128 scales
//   combine    out[t] = sum_j w[t][j] * y[pos[t][j]]
//   its gradient  dy[pos[t][j]] = w[t][j] * dout[t],
//                 dw[t][j] = <dout[t], y[pos[t][j]]>
// The combine with unit weights is the dispatch's gradient.
//
// All but the sort are streams bounded by memory: every row of x is read once
// and written to its k places (a quantizing dispatch forms its codes once),
// every row of y is read once.  A wave moves a run of one row; the places are
// wave-uniform and come through the scalar cache.  Rows outside [0, rows) are
// nowhere written or read, whatever the tables hold.
// Measured (one MI355X, kernel time): sort of 65536 pairs over 256 experts 10.8
// us, of up to 512 3.2; 8192 x 8 rows of 7168: codes 119 (5.1 TB/s), combine
// 179 (5.9 TB/s); 4096 x 2: combine 30, gradient 53 (5.8 TB/s); 3001 x 4 rows of
// 1530 copied 11.6 (4.6 TB/s).
#pragma once

#include "rows_common.h"

namespace fp8k {

// ---------------------------------------------------------------------------
// The sort.
// ---------------------------------------------------------------------------
constexpr int kSortMaxExperts = 1024;
constexpr int kSortBins = kSortMaxExperts + 1;      // and one for pairs kept without an expert

struct SortParams {
    const void* ids;            // int32, or int64
    int32_t* pos;               // may be NULL
    int32_t* src;
    int32_t* m_indices;         // contiguous layout
    int32_t* counts;            // of each expert; masked layout: at most max_m; may be NULL
    int32_t* hist;              // [bins][chunks4], with more than one chunk
    int64_t pairs, rows;
    int64_t chunk;              // pairs of a workgroup
    int32_t E, bins;            // bins: E, or E + 1 where pairs without an expert get rows too
    int32_t chunks, chunks4;    // chunks4: rounded up to a multiple of 4
    int32_t align;              // contiguous
    int64_t max_m;              // masked
    bool contiguous;            // else masked
    bool wide;                  // ids are int64
};

// Bin of a pair, or -1.
__device__ __forceinline__ int sort_bin(const SortParams& p, int64_t i) {
    const int64_t id = p.wide ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
    if (id >= 0 && id < p.E) return (int)id;
    return p.bins > p.E ? p.E : -1;
}

// -1 to every row's entries, by all threads of `groups` workgroups; the rows of
// pairs are written after it.
template <int THREADS>
__device__ __forceinline__ void sort_clear(const SortParams& p, int group, int groups) {
    const i32x4 none{-1, -1, -1, -1};
    for (int64_t r = 4 * ((int64_t)group * THREADS + threadIdx.x); r < p.rows; r += (int64_t)4 * groups * THREADS) {
        if (r + 4 <= p.rows) {              // (at any alignment)
            __builtin_memcpy(p.src + r, &none, 16);
            if (p.contiguous) __builtin_memcpy(p.m_indices + r, &none, 16);
        } else {
            for (int64_t i = r; i < p.rows; ++i) {
                p.src[i] = -1;
                if (p.contiguous) p.m_indices[i] = -1;
            }
        }
    }
}

// Pairs per bin of one chunk; and all rows cleared.
__global__ __launch_bounds__(1024) void expert_count_kernel(SortParams p) {
    __shared__ int32_t hist[kSortBins];
    const int64_t lo = blockIdx.x * p.chunk, end = lo + p.chunk < p.pairs ? lo + p.chunk : p.pairs;
    const int64_t i0 = lo + threadIdx.x;
    const int first = i0 < end ? sort_bin(p, i0) : -1;      // (its load runs while the counts are cleared)
    for (int b = threadIdx.x; b < p.bins; b += 1024) hist[b] = 0;
    sort_clear<1024>(p, blockIdx.x, gridDim.x);
    __syncthreads();
    if (first >= 0) atomicAdd(&hist[first], 1);
    for (int64_t i = i0 + 1024; i < end; i += 1024) {
        const int b = sort_bin(p, i);
        if (b >= 0) atomicAdd(&hist[b], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.bins; b += 1024) p.hist[(int64_t)b * p.chunks4 + blockIdx.x] = hist[b];
    if (blockIdx.x == 0) {                  // (what a row of four is filled up with)
        for (int b = threadIdx.x; b < p.bins; b += 1024)
            for (int c = p.chunks; c < p.chunks4; ++c) p.hist[(int64_t)b * p.chunks4 + c] = 0;
    }
}

// Inclusive sum over the 64 lanes.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

// Lanes whose key (of `bits` bits) is the lane's own.
__device__ __forceinline__ uint64_t same_key(uint32_t key, int bits) {
    uint64_t same = ~0ull;
    for (int k = 0; k < bits; ++k) {
        const bool bit = key >> k & 1u;
        const uint64_t m = __ballot(bit);
        same &= bit ? m : ~m;
    }
    return same;
}

// Rows of one chunk's pairs.  Each wave takes a run of the chunk, 64 pairs at a
// time; a lane's rank among them is the number of lower lanes with its bin, and
// a count per wave and bin numbers the pairs of a run.  The counts of the waves
// before it and of the chunks before this one then make the first row of a
// wave's bin.  ROUNDS: times 64 pairs that a wave keeps in registers between
// the two passes, or 0 (any number, formed twice).  No result depends on the
// order of atomics.
template <int WAVES, int ROUNDS>
__global__ __launch_bounds__(64 * WAVES) void expert_place_kernel(SortParams p) {
    constexpr int THREADS = 64 * WAVES;
    __shared__ int32_t next[WAVES][kSortBins];  // per wave: counts, then the first row
    __shared__ int32_t total[kSortBins];        // per bin: all chunks' pairs
    __shared__ int32_t earlier[kSortBins];      // ... and those of the chunks before this one
    __shared__ int32_t sums[WAVES];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = blockIdx.x;
    const int bits = 32 - __builtin_clz(p.bins);        // a bin and "none" (= bins) fit
    const int64_t lo = c * p.chunk, end = lo + p.chunk < p.pairs ? lo + p.chunk : p.pairs;
    const int64_t run = ((end - lo + WAVES - 1) / WAVES + 63) / 64 * 64;
    const int64_t w_lo = lo + wave * run, w_end = w_lo + run < end ? w_lo + run : end;
    int bin[ROUNDS > 0 ? ROUNDS : 1], at[ROUNDS > 0 ? ROUNDS : 1];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int64_t i = w_lo + 64 * r + lane;
        bin[r] = i < w_end ? sort_bin(p, i) : -1;
    }
    if (p.chunks == 1) sort_clear<THREADS>(p, 0, 1);    // (else the first kernel has)
    // (a wave clears and counts its own bins; LDS operations of a wave run in order)
    for (int b = lane; b < p.bins; b += 64) next[wave][b] = 0;
    // Numbers of 64 pairs within the wave's run.
    auto number = [&](int b) FP8K_INLINE {
        const uint64_t same = same_key(b >= 0 ? (uint32_t)b : (uint32_t)p.bins, bits);
        const int rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
        int k = 0;
        if (b >= 0) k = next[wave][b] + rank;
        __builtin_amdgcn_wave_barrier();        // (every lane has read before the last one of its bin writes)
        if (b >= 0 && rank == n - 1) next[wave][b] = k + 1;
        __builtin_amdgcn_wave_barrier();
        return k;
    };
    if constexpr (ROUNDS > 0) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) at[r] = number(bin[r]);
    } else {
        for (int64_t i = w_lo + lane; i < w_end; i += 64) {
            const int b = sort_bin(p, i);
            if (b >= 0) atomicAdd(&next[wave][b], 1);
        }
    }
    if (p.chunks > 1) {
        // all chunks' pairs of a bin, and those of the chunks before this one, by 2^k threads a bin
        int per = 1;
        while (per < 16 && per * 2 * p.bins <= THREADS) per *= 2;
        for (int b0 = 0; b0 < p.bins; b0 += THREADS / per) {
            const int b = b0 + threadIdx.x / per;
            int all = 0, before = 0;
            if (b < p.bins) {
                const i32x4* h = reinterpret_cast<const i32x4*>(p.hist + (int64_t)b * p.chunks4);
#pragma unroll 4
                for (int k = threadIdx.x % per; k < p.chunks4 / 4; k += per) {
                    const i32x4 n = h[k];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        all += n[e];
                        before += 4 * k + e < c ? n[e] : 0;
                    }
                }
            }
            for (int o = per / 2; o >= 1; o /= 2) {
                all += __shfl_xor(all, o);
                before += __shfl_xor(before, o);
            }
            if (b < p.bins && threadIdx.x % per == 0) {
                total[b] = all;
                earlier[b] = before;
            }
        }
    }
    __syncthreads();
    // the rows that each bin's segment takes
    int carry = 0;
    for (int b0 = 0; b0 < p.bins; b0 += THREADS) {
        const int b = b0 + threadIdx.x;
        int before = 0, all = 0, take = 0;
        if (b < p.bins) {
            if (p.chunks > 1) {
                all = total[b];
                before = earlier[b];
            } else {
#pragma unroll
                for (int w = 0; w < WAVES; ++w) all += next[w][b];
            }
            if (c == 0 && b < p.E && p.counts) p.counts[b] = p.contiguous || all < p.max_m ? all : (int)p.max_m;
            take = p.contiguous ? (all + p.align - 1) / p.align * p.align : 0;
        }
        const int upto = wave_scan(take, lane);
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        int first = carry + upto - take;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            first += w < wave ? sums[w] : 0;
            carry += sums[w];
        }
        if (b < p.bins) {
            // (rows and pairs together stay below 2^31)
            if (!p.contiguous) first = (int)(b * p.max_m);
            int row = first + before;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const int n = next[w][b];
                next[w][b] = row;
                row += n;
            }
        }
        __syncthreads();
    }
    auto place = [&](int64_t i, int b, int row) FP8K_INLINE {
        const bool held = b >= 0 && row < p.rows && (p.contiguous || row < (b + 1) * p.max_m);
        if (p.pos) p.pos[i] = held ? row : -1;
        if (held) {
            p.src[row] = (int32_t)i;
            if (p.contiguous) p.m_indices[row] = b < p.E ? b : -1;
        }
    };
    if constexpr (ROUNDS > 0) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int64_t i = w_lo + 64 * r + lane;
            if (i < w_end) place(i, bin[r], (bin[r] >= 0 ? next[wave][bin[r]] : 0) + at[r]);
        }
    } else {
        for (int64_t i0 = w_lo; i0 < w_end; i0 += 64) {
            const int64_t i = i0 + lane;
            const int b = i < w_end ? sort_bin(p, i) : -1;
            const int row = number(b);
            if (i < w_end) place(i, b, row);
        }
    }
}

// ---------------------------------------------------------------------------
// Moving rows.
// ---------------------------------------------------------------------------
struct RowsParams {
    const void* x;              // dispatch: x (T, W); combine: y (rows, W); gradient: dout (T, W)
    const void* y;              // gradient: y (rows, W)
    void* out;                  // dispatch: xs (rows, W); combine: out (T, W); gradient: dy (rows, W), or NULL
    const int32_t* pos;         // (T, k)
    const int32_t* src;         // (rows), or NULL: rows without a pair stay as they are
    const float* w;             // (T, k), or NULL: 1
    float* dw;                  // (T, k), or NULL
    float* sa;                  // quantizing dispatch: [W/128][rows]
    int64_t T, rows, W;
    int64_t segs;               // runs per row
    int64_t work;               // waves (workgroups of the gradient) that move rows; those behind them clear rows
    int32_t k;
};

// Rows of the experts' buffer that one wave looks through for cleared ones.
constexpr int kClearRows = 8;

// Zeros to the rows of a group of kClearRows that no pair has.
template <typename T, bool STREAM = false>
__device__ __forceinline__ void clear_rows(const RowsParams& p, int64_t group, int lane) {
    const int64_t r0 = group * kClearRows;
    const bool none = lane < kClearRows && r0 + lane < p.rows && p.src[r0 + lane] < 0;
    uint64_t left = __ballot(none);
    while (left) {
        const int64_t r = r0 + __builtin_ctzll(left);
        left &= left - 1;
        T* row = static_cast<T*>(p.out) + r * p.W;
        for (int64_t n = lane * RowElem<T>::VN; n < p.W; n += 64 * RowElem<T>::VN)
            store_row16<T, STREAM>(row + n, p.W - n, i32x4{0, 0, 0, 0});
    }
}

constexpr int kRowVecs = 4;     // 16-byte vectors of a lane per run: 4 KB per wave

template <typename T>
__global__ __launch_bounds__(256) void expert_dispatch_kernel(RowsParams p) {
    constexpr int VN = RowElem<T>::VN;
    const int64_t u = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (u >= p.work) {
        if (p.src) clear_rows<T>(p, u - p.work, lane);
        return;
    }
    const int64_t t = u / p.segs, n0 = (u - t * p.segs) * (64 * VN * kRowVecs) + lane * VN;
    const T* x = static_cast<const T*>(p.x) + t * p.W;
    i32x4 v[kRowVecs];
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i) {
        const int64_t n = n0 + i * 64 * VN;
        if (n < p.W) v[i] = load_row16<T>(x + n, p.W - n);
    }
    for (int j = 0; j < p.k; ++j) {
        const int64_t row = uniform(p.pos[t * p.k + j]);
        if (row < 0 || row >= p.rows) continue;
        T* out = static_cast<T*>(p.out) + row * p.W;
#pragma unroll
        for (int i = 0; i < kRowVecs; ++i) {
            const int64_t n = n0 + i * 64 * VN;
            if (n < p.W) store_row16<T>(out + n, p.W - n, v[i]);
        }
    }
}

// A wave forms the codes of 8 groups of a token (a lane 16 elements, 8 lanes a
// group) and stores them at the token's k places.  The scales of one K block
// lie beside those of the expert's neighbouring tokens, 4 bytes each: every die
// takes a run of consecutive tokens, whose pieces of a line then meet in its
// cache (1024 x 8 of 64 experts, K 7168: tokens dealt out to the dies in turn
// 17.7 us, so 14.6).  STREAM: codes that do not fit the last-level cache are
// stored past the caches, which then keep those lines (8192 x 8 of 256 experts,
// 470 MB of codes: 150 us, so 120, as long as without any scales; 67 MB: no
// difference).
template <typename T, bool POW2, bool STREAM>
__global__ __launch_bounds__(256) void expert_dispatch_quant_kernel(RowsParams p) {
    constexpr int VN = RowElem<T>::VN;
    // (a grid of whole 8s: block b runs on die b % 8)
    const int64_t u = ((int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)) * 4 + uniform(threadIdx.x >> 6);
    if (u >= p.work) return;
    const int lane = threadIdx.x & 63;
    const int64_t t = u / p.segs, kb = (u - t * p.segs) * 8 + (lane >> 3);
    const bool in = kb < p.W / 128;
    const int64_t n = kb * 128 + (lane & 7) * 16;
    float f[16];
#pragma unroll
    for (int i = 0; i < 16 / VN; ++i) {
        i32x4 v{0, 0, 0, 0};
        if (in) v = *reinterpret_cast<const i32x4*>(static_cast<const T*>(p.x) + t * p.W + n + i * VN);
#pragma unroll
        for (int e = 0; e < VN; ++e) f[i * VN + e] = RowElem<T>::get(v, e);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 8));
    const float s = group_scale(amax, POW2), r = 1.0f / s;
    i32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = (int)cvt_e4m3x4_quot<POW2>(f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]}, s, r);
    for (int j = 0; j < p.k; ++j) {
        const int64_t row = uniform(p.pos[t * p.k + j]);
        if (row < 0 || row >= p.rows || !in) continue;
        i32x4* out = reinterpret_cast<i32x4*>(static_cast<uint8_t*>(p.out) + row * p.W + n);
        if constexpr (STREAM) __builtin_nontemporal_store(q, out);
        else *out = q;
        if ((lane & 7) == 0) p.sa[kb * p.rows + row] = s;
    }
}

constexpr int kCombineVecs = 2; // 16-byte vectors of a lane per row and run

// STREAM: rows of whole cache lines are read with the nontemporal hint, each
// once (8192 x 8, N 7168: 209 us without, 195 with it; 4096 x 2 35.5, 30.9; rows
// of 3060 bytes, which share lines, 11.1, 12.6).
template <typename T, bool STREAM>
__global__ __launch_bounds__(256) void expert_combine_kernel(RowsParams p) {
    constexpr int VN = RowElem<T>::VN;
    const int64_t u = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    if (u >= p.work) return;
    const int lane = threadIdx.x & 63;
    const int64_t t = u / p.segs, n0 = (u - t * p.segs) * (64 * VN * kCombineVecs) + lane * VN;
    float acc[kCombineVecs][VN] = {};
    for (int j0 = 0; j0 < p.k; j0 += 4) {
        i32x4 v[4][kCombineVecs];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = t * p.k + j0 + j;
            const int64_t row = j0 + j < p.k ? (int64_t)uniform(p.pos[at]) : -1;
            const bool held = row >= 0 && row < p.rows;
            w[j] = held ? (p.w ? p.w[at] : 1.0f) : 0.f;
#pragma unroll
            for (int i = 0; i < kCombineVecs; ++i) {
                const int64_t n = n0 + i * 64 * VN;
                v[j][i] = i32x4{0, 0, 0, 0};
                if (held && n < p.W) v[j][i] = load_row16<T, STREAM>(static_cast<const T*>(p.x) + row * p.W + n, p.W - n);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < kCombineVecs; ++i)
#pragma unroll
                for (int e = 0; e < VN; ++e) acc[i][e] = fmaf(w[j], RowElem<T>::get(v[j][i], e), acc[i][e]);
    }
#pragma unroll
    for (int i = 0; i < kCombineVecs; ++i) {
        const int64_t n = n0 + i * 64 * VN;
        if (n < p.W) store_row16<T>(static_cast<T*>(p.out) + t * p.W + n, p.W - n, RowElem<T>::pack(acc[i]));
    }
}

// A workgroup takes a token: dout is read once per PAIRS of its pairs, each row
// of y once.  STREAM: rows of whole cache lines are read and written with the
// nontemporal hint (4096 x 2, N 7168: 66 us without, 55 with it, and 117, 115
// with a pass that reads dy; 1024 x 8 86, 76; 8192 x 8 510, 496; rows of 3060
// bytes 26.4, 26.9).  With 8 pairs at a time the compiler keeps up to 43 scalars
// (rows and their bases) in lanes of vector registers; nothing goes to memory.
template <typename T, int PAIRS, bool STREAM>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(RowsParams p) {
    constexpr int VN = RowElem<T>::VN;
    __shared__ float part[4][PAIRS];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t t = blockIdx.x;
    if (t >= p.work) {
        if (p.src) clear_rows<T, STREAM>(p, (t - p.work) * 4 + wave, lane);
        return;
    }
    const T* dout = static_cast<const T*>(p.x) + t * p.W;
    for (int j0 = 0; j0 < p.k; j0 += PAIRS) {
        int64_t row[PAIRS];
        float w[PAIRS], acc[PAIRS] = {};
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            const int64_t at = t * p.k + j0 + j;
            row[j] = j0 + j < p.k ? (int64_t)uniform(p.pos[at]) : -1;
            if (row[j] >= p.rows) row[j] = -1;
            w[j] = row[j] >= 0 && p.w ? p.w[at] : 1.0f;
        }
        for (int64_t n = threadIdx.x * VN; n < p.W; n += 256 * VN) {
            const i32x4 d = load_row16<T>(dout + n, p.W - n);
            i32x4 v[PAIRS];
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                v[j] = i32x4{0, 0, 0, 0};
                if (p.dw && row[j] >= 0) v[j] = load_row16<T, STREAM>(static_cast<const T*>(p.y) + row[j] * p.W + n, p.W - n);
            }
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                float s[VN];
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    const float g = RowElem<T>::get(d, e);
                    acc[j] = fmaf(g, RowElem<T>::get(v[j], e), acc[j]);
                    s[e] = w[j] * g;
                }
                if (p.out && row[j] >= 0)
                    store_row16<T, STREAM>(static_cast<T*>(p.out) + row[j] * p.W + n, p.W - n, RowElem<T>::pack(s));
            }
        }
        if (p.dw) {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                // (a pair without a row has no product, even of an infinite dout)
                const float s = wave_sum(acc[j]);
                if (lane == 0) part[wave][j] = row[j] >= 0 ? s : 0.f;
            }
            __syncthreads();
            const int j = threadIdx.x;
            if (j < PAIRS && j0 + j < p.k)
                p.dw[t * p.k + j0 + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
            __syncthreads();
        }
    }
}

}  // namespace fp8k
