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
#pragma once

#include "rows_common.h"

namespace fp8k {

// ---------------------------------------------------------------------------
// The sort.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMaxExperts = 1024;
constexpr int kSortBins = kSortMaxExperts + 1;      // and one for pairs kept without an expert

struct SortParams {
    const void* ids;            // int32, or int64
    int32_t* pos;
    int32_t* src;
    int32_t* m_indices;         // contiguous layout
    int32_t* counts;            // of each expert; masked layout: at most max_m
    int32_t* hist;              // [chunks][bins], with more than one chunk
    int64_t pairs, rows;
    int64_t chunk;              // pairs of a workgroup
    int32_t E, bins;            // bins: E, or E + 1 where pairs without an expert get rows too
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

// Pairs per bin of one chunk.
__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(SortParams p) {
    __shared__ int32_t hist[kSortBins];
    for (int b = threadIdx.x; b < p.bins; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * p.chunk, end = lo + p.chunk < p.pairs ? lo + p.chunk : p.pairs;
    for (int64_t i = lo + threadIdx.x; i < end; i += kSortThreads) {
        const int b = sort_bin(p, i);
        if (b >= 0) atomicAdd(&hist[b], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.bins; b += kSortThreads) p.hist[(int64_t)blockIdx.x * p.bins + b] = hist[b];
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

// Rows of one chunk's pairs.  Each wave counts and then places a run of the
// chunk's pairs: the bins' counts of the waves before it and of the chunks
// before this one make the first row of its own, and within 64 pairs a lane's
// rank is the number of lower lanes with its bin (a mask that one ballot per
// bit of the bin narrows).  No result depends on the order of the counting
// atomics.
__global__ __launch_bounds__(kSortThreads) void expert_place_kernel(SortParams p) {
    __shared__ int32_t next[kSortWaves][kSortBins];     // per wave: counts, then the next row
    __shared__ int32_t total[kSortBins];
    __shared__ int32_t start[kSortBins + 1];
    __shared__ int32_t sums[kSortWaves];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int chunks = gridDim.x, c = blockIdx.x;
    for (int b = lane; b < p.bins; b += 64) next[wave][b] = 0;
    const int64_t lo = c * p.chunk, end = lo + p.chunk < p.pairs ? lo + p.chunk : p.pairs;
    const int64_t run = ((end - lo + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    const int64_t w_lo = lo + wave * run, w_end = w_lo + run < end ? w_lo + run : end;
    for (int64_t i = w_lo + lane; i < w_end; i += 64) {
        const int b = sort_bin(p, i);
        if (b >= 0) atomicAdd(&next[wave][b], 1);
    }
    __syncthreads();
    // totals, and the rows that a bin's segment takes
    int carry = 0;
    for (int b0 = 0; b0 < p.bins; b0 += kSortThreads) {
        const int b = b0 + threadIdx.x;
        int before = 0, all = 0, take = 0;
        if (b < p.bins) {
            if (chunks > 1) {
#pragma unroll 8
                for (int i = 0; i < chunks; ++i) {
                    const int n = p.hist[(int64_t)i * p.bins + b];
                    all += n;
                    before += i < c ? n : 0;
                }
            } else {
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w) all += next[w][b];
            }
            total[b] = all;
            take = p.contiguous ? (all + p.align - 1) / p.align * p.align : 0;
        }
        const int upto = wave_scan(take, lane);
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        int first = carry + upto - take;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            first += w < wave ? sums[w] : 0;
            carry += sums[w];
        }
        if (b < p.bins) {
            // (rows past 2^31 do not exist: a masked buffer has fewer, and so has a contiguous one)
            if (!p.contiguous) first = (int)(b * p.max_m);
            start[b] = first;
            int at = first + before;
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const int n = next[w][b];
                next[w][b] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) start[p.bins] = carry;
    __syncthreads();
    const int bits = 32 - __builtin_clz(p.bins);        // a bin and "none" (= bins) fit
    for (int64_t i0 = w_lo; i0 < w_end; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < w_end;
        const int b = in ? sort_bin(p, i) : -1;
        const uint32_t key = b >= 0 ? (uint32_t)b : (uint32_t)p.bins;
        uint64_t same = ~0ull;
        for (int k = 0; k < bits; ++k) {
            const bool bit = key >> k & 1u;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
        int at = 0;
        if (b >= 0) at = next[wave][b] + rank;
        __builtin_amdgcn_wave_barrier();                // (every lane has read before the last one of its bin writes)
        if (b >= 0 && rank == n - 1) next[wave][b] = at + 1;
        __builtin_amdgcn_wave_barrier();
        if (in) {
            const bool held = b >= 0 && at < p.rows && (p.contiguous || at < (b + 1) * p.max_m);
            p.pos[i] = held ? at : -1;
            if (held) {
                p.src[at] = (int32_t)i;
                if (p.contiguous) p.m_indices[at] = b < p.E ? b : -1;
            }
        }
    }
    // what no pair has: counts, and the rows behind a segment's pairs
    for (int b = c * kSortWaves + wave; b < p.bins; b += chunks * kSortWaves) {
        const int n = total[b];
        if (lane == 0 && b < p.E) p.counts[b] = p.contiguous || n < p.max_m ? n : (int)p.max_m;
        const int64_t s = start[b];
        int64_t to = p.contiguous ? s + (int64_t)(n + p.align - 1) / p.align * p.align : s + p.max_m;
        to = to < p.rows ? to : p.rows;
        for (int64_t r = s + n + lane; r < to; r += 64) {
            p.src[r] = -1;
            if (p.contiguous) p.m_indices[r] = -1;
        }
    }
    if (p.contiguous) {
        for (int64_t r = start[p.bins] + (int64_t)c * kSortThreads + threadIdx.x; r < p.rows; r += (int64_t)chunks * kSortThreads) {
            p.src[r] = -1;
            p.m_indices[r] = -1;
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
template <typename T>
__device__ __forceinline__ void clear_rows(const RowsParams& p, int64_t group, int lane) {
    const int64_t r0 = group * kClearRows;
    const bool none = lane < kClearRows && r0 + lane < p.rows && p.src[r0 + lane] < 0;
    uint64_t left = __ballot(none);
    while (left) {
        const int64_t r = r0 + __builtin_ctzll(left);
        left &= left - 1;
        T* row = static_cast<T*>(p.out) + r * p.W;
        for (int64_t n = lane * RowElem<T>::VN; n < p.W; n += 64 * RowElem<T>::VN)
            store_row16<T>(row + n, p.W - n, i32x4{0, 0, 0, 0});
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
// group) and stores them at the token's k places.
template <typename T, bool POW2>
__global__ __launch_bounds__(256) void expert_dispatch_quant_kernel(RowsParams p) {
    constexpr int VN = RowElem<T>::VN;
    const int64_t u = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
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
        *reinterpret_cast<i32x4*>(static_cast<uint8_t*>(p.out) + row * p.W + n) = q;
        if ((lane & 7) == 0) p.sa[kb * p.rows + row] = s;
    }
}

constexpr int kCombineVecs = 2; // 16-byte vectors of a lane per row and run

template <typename T>
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
                if (held && n < p.W) v[j][i] = load_row16<T>(static_cast<const T*>(p.x) + row * p.W + n, p.W - n);
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

// A workgroup takes a token: dout is read once per 4 of its pairs, each row of
// y once.
constexpr int kGradPairs = 4;

template <typename T>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(RowsParams p) {
    constexpr int VN = RowElem<T>::VN;
    __shared__ float part[4][kGradPairs];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t t = blockIdx.x;
    if (t >= p.work) {
        if (p.src) clear_rows<T>(p, (t - p.work) * 4 + wave, lane);
        return;
    }
    const T* dout = static_cast<const T*>(p.x) + t * p.W;
    for (int j0 = 0; j0 < p.k; j0 += kGradPairs) {
        int64_t row[kGradPairs];
        float w[kGradPairs], acc[kGradPairs] = {};
#pragma unroll
        for (int j = 0; j < kGradPairs; ++j) {
            const int64_t at = t * p.k + j0 + j;
            row[j] = j0 + j < p.k ? (int64_t)uniform(p.pos[at]) : -1;
            if (row[j] >= p.rows) row[j] = -1;
            w[j] = row[j] >= 0 && p.w ? p.w[at] : 1.0f;
        }
        for (int64_t n = threadIdx.x * VN; n < p.W; n += 256 * VN) {
            const i32x4 d = load_row16<T>(dout + n, p.W - n);
            i32x4 v[kGradPairs];
#pragma unroll
            for (int j = 0; j < kGradPairs; ++j) {
                v[j] = i32x4{0, 0, 0, 0};
                if (p.dw && row[j] >= 0) v[j] = load_row16<T>(static_cast<const T*>(p.y) + row[j] * p.W + n, p.W - n);
            }
#pragma unroll
            for (int j = 0; j < kGradPairs; ++j) {
                float s[VN];
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    const float g = RowElem<T>::get(d, e);
                    acc[j] = fmaf(g, RowElem<T>::get(v[j], e), acc[j]);
                    s[e] = w[j] * g;
                }
                if (p.out && row[j] >= 0)
                    store_row16<T>(static_cast<T*>(p.out) + row[j] * p.W + n, p.W - n, RowElem<T>::pack(s));
            }
        }
        if (p.dw) {
#pragma unroll
            for (int j = 0; j < kGradPairs; ++j) {
                // (a pair without a row has no product, even of an infinite dout)
                const float s = wave_sum(acc[j]);
                if (lane == 0) part[wave][j] = row[j] >= 0 ? s : 0.f;
            }
            __syncthreads();
            const int j = threadIdx.x;
            if (j < kGradPairs && j0 + j < p.k)
                p.dw[t * p.k + j0 + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
            __syncthreads();
        }
    }
}

}  // namespace fp8k
