// kernels_route.h -- the router's choice of experts and its gradient, for
// gfx950:
//   ids[t][j]  the expert of row t's j-th largest logit (ties: lowest expert)
//   w[t][j] = scale * p[ids[t][j]] / (renorm ? sum_i p[ids[t][i]] : 1),
//   p = softmax(logits[t])
// and, with G = sum_j w_j dw_j / scale,
//   dlogits[e] = sum over j with ids_j = e of w_j (dw_j - (renorm ? G : 0))
//                - (renorm ? 0 : scale p_e G).
//
// What bounds it: the k dependent steps of a choice for one token, the logits'
// stream for many.  A wave takes one row; lane l holds the PER consecutive
// experts from PER * l as integers that compare as the logits do, so one
// maximum over the wave (six lane shifts, no LDS) finds the next expert and
// the first lane that holds it is the lowest index.  The selection compares
// logits, not probabilities: it is exact.
// Measured (one MI355X, kernel time): 1 row of 256 experts, k 8, 3.0 us; 8192
// rows BF16 7.6; 4095 x 162, k 6, 5.7 and the gradient 5.6.
#pragma once

#include "rows_common.h"

namespace fp8k {

struct RouteParams {
    const void* logits;
    float* w;
    int32_t* ids;
    const float* dw;
    void* dlogits;
    int64_t T;
    int32_t E, k;
    float scale;
    bool renorm;
    bool vec;                   // lanes' experts can be loaded as whole vectors
};

// Logits as integers in their order: NaN above everything, -0 as 0, -infinity
// (an expert that is masked out) and places behind the last expert 0.
__device__ __forceinline__ uint32_t route_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    if (b == 0xFF800000u) return 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float route_value(uint32_t key) {
    return __uint_as_float(key == 0xFFFFFFFFu ? 0x7FC00000u : key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The lane's PER logits, -infinity behind the row's end.
template <typename T, int PER>
__device__ __forceinline__ void route_load(const RouteParams& p, int64_t row, int lane, float* v) {
    const T* l = static_cast<const T*>(p.logits) + row * p.E;
    const int e0 = lane * PER;
    T raw[PER];
    if (p.vec) {                // E is a multiple of PER and every lane's place is aligned
        if (e0 < p.E) {
            __builtin_memcpy(raw, __builtin_assume_aligned(l + e0, PER * sizeof(T) < 16 ? PER * sizeof(T) : 16), sizeof(raw));
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = RowElem<T>::get1(raw[i]);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = e0 + i < p.E ? RowElem<T>::get1(l[e0 + i]) : -INFINITY;
    }
}

template <typename T, int PER>
__global__ __launch_bounds__(256) void route_topk_kernel(RouteParams p) {
    const int64_t row = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    if (row >= p.T) return;
    const int lane = threadIdx.x & 63;
    float v[PER];
    uint32_t key[PER];
    route_load<T, PER>(p, row, lane, v);
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = route_key(v[i]);
        best = key[i] > best ? key[i] : best;
    }
    // lane j keeps the j-th choice
    uint32_t mine = 0, first = 0;
    int32_t id = -1;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t m = wave_max_u32(best);
        if (j == 0) first = m;
        if (m == 0) break;
        const int from = __builtin_ctzll(__ballot(best == m));
        int at = 0;
        if (lane == from) {
            best = 0;
            bool found = false;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (!found && key[i] == m) {
                    found = true;
                    at = i;
                    key[i] = 0;
                }
                best = key[i] > best ? key[i] : best;
            }
        }
        at = __builtin_amdgcn_readlane(at, from);
        if (lane == j) {
            id = from * PER + at;
            mine = m;
        }
    }
    const float top = route_value(first);
    const float e = id >= 0 ? expf(route_value(mine) - top) : 0.f;
    float sum = e;
    if (!p.renorm) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += expf(v[i] - top);
    }
    sum = wave_sum(sum);
    if (lane < p.k) {
        p.ids[row * p.k + lane] = id;
        // (a row without any expert has no sum either)
        p.w[row * p.k + lane] = id >= 0 ? p.scale * (e / sum) : 0.f;
    }
}

// The choice is read back from ids; its probabilities are formed again.  An
// index outside the experts adds nothing, one that stands twice counts twice.
template <typename T, int PER>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteParams p) {
    const int64_t row = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    if (row >= p.T) return;
    const int lane = threadIdx.x & 63;
    const int id = lane < p.k ? p.ids[row * p.k + lane] : -1;
    const bool chosen = id >= 0 && id < p.E;
    const T* l = static_cast<const T*>(p.logits) + row * p.E;
    const float mine = chosen ? RowElem<T>::get1(l[id]) : -INFINITY;
    float v[PER];
    uint32_t top_key = route_key(mine);
    if (!p.renorm) {
        route_load<T, PER>(p, row, lane, v);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t k = route_key(v[i]);
            top_key = k > top_key ? k : top_key;
        }
    }
    top_key = wave_max_u32(top_key);
    // (no expert at all: every exponential is 0 then, not the difference of two infinities)
    const float top = top_key ? route_value(top_key) : 0.f;
    const float e = chosen ? expf(mine - top) : 0.f;
    float sum = e;
    if (!p.renorm) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = expf(v[i] - top);
            sum += v[i];
        }
    }
    sum = wave_sum(sum);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    const float w = e * inv;
    const float dw = chosen ? p.dw[row * p.k + lane] : 0.f;
    const float total = wave_sum(w * dw);
    const float add = p.renorm ? w * (dw - total) : w * dw;
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = p.renorm ? 0.f : -(v[i] * inv) * total;
    for (int j = 0; j < p.k; ++j) {
        const int at = __builtin_amdgcn_readlane(chosen ? id : -1, j) - lane * PER;
        const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(add), j));
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] += at == i ? a : 0.f;
    }
    T* out = static_cast<T*>(p.dlogits) + row * p.E;
    const int e0 = lane * PER;
    T raw[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) raw[i] = RowElem<T>::put1(p.scale * d[i]);
    if (p.vec) {
        if (e0 < p.E) __builtin_memcpy(__builtin_assume_aligned(out + e0, PER * sizeof(T) < 16 ? PER * sizeof(T) : 16), raw, sizeof(raw));
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e0 + i < p.E) out[e0 + i] = raw[i];
    }
}

}  // namespace fp8k
