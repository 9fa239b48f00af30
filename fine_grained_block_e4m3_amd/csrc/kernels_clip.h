// kernels_clip.h -- global gradient norm over many tensors, and clipping, for
// gfx950:  norm = sqrt(sum over tensors and elements of g^2),
//          out = g * min(1, max_norm / (norm + 1e-6)).
//
// What bounds it: memory, two passes over the gradients (the factor depends
// on all of them) and one write.  The tensors reach the kernels as a table in
// the kernel arguments, so a call needs no copy to the device; a batch holds
// kClipBatch tensors, cut into chunks of kClipChunk elements that the
// workgroups take in turn (the tensor of a chunk is found by bisection of the
// first chunks), so many small tensors and a few large ones keep every
// compute unit equally busy.
//   * Squares are summed in FP64, which a stream leaves time for: no overflow
//     or underflow for any finite FP32 gradient.  Every workgroup writes its
//     sum to its own slot and the slots are added in a fixed order, so equal
//     inputs give equal results.
//   * The second pass runs backwards, over what the first read last, of which
//     the 256 MB last-level cache still holds a part.
//   * Vector loads of 16 bytes at any element alignment (gradients are often
//     views of a flat buffer).
// Measured (one MI355X, kernel time): 300 tensors of 400 M elements in both
// types, 1.14 GB, 703-710 us out of place (3.43 GB at 4.8 TB/s; the norm pass
// alone 5.6 TB/s with what the last-level cache holds; forwards 727); 24
// tensors of 0.26 M elements 10.5 us, two launches.
#pragma once

#include "gated_common.h"

namespace fp8k {

constexpr int kClipBatch = 120;             // tensors per launch (kernel arguments stay below 4 KB)
constexpr int kClipChunk = 8192;            // elements
constexpr int kClipMaxGrid = 2048;          // workgroups per launch
constexpr int kClipMaxSlots = 2048;         // sums that every workgroup of the second pass adds by itself

enum ClipType : int { kClipF32 = 0, kClipBf16 = 1, kClipF16 = 2 };

struct ClipTable {
    const void* in[kClipBatch];
    void* out[kClipBatch];
    int64_t n_type[kClipBatch];             // 4 * elements + type
    int32_t first[kClipBatch + 1];          // first chunk of each tensor; last: all chunks
    int32_t count;
};
static_assert(sizeof(ClipTable) <= 3856, "kernel arguments");

__device__ __forceinline__ int clip_tensor_of(const ClipTable& t, int chunk) {
    int lo = 0, hi = t.count;               // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Element type traits: VN elements per 16-byte vector.
template <int TYPE>
struct ClipElem {
    using T = uint16_t;
    static constexpr int VN = 8;
    static __device__ __forceinline__ float get(i32x4 v, int i) {
        const uint32_t b = (uint32_t)v[i >> 1] >> (16 * (i & 1)) & 0xFFFFu;
        if constexpr (TYPE == kClipBf16) return __uint_as_float(b << 16);
        else return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        if constexpr (TYPE == kClipBf16) return pack_bf16x2(a, b);
        else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    }
    static __device__ __forceinline__ i32x4 scale(i32x4 v, float c) {
        i32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = (int)pack(get(v, 2 * j) * c, get(v, 2 * j + 1) * c);
        return r;
    }
    static __device__ __forceinline__ float get1(T b) { return get(i32x4{(int)b, 0, 0, 0}, 0); }
    static __device__ __forceinline__ T put1(float a) { return (T)(pack(a, 0.f) & 0xFFFFu); }
};
template <>
struct ClipElem<kClipF32> {
    using T = float;
    static constexpr int VN = 4;
    static __device__ __forceinline__ float get(i32x4 v, int i) { return __int_as_float(v[i]); }
    static __device__ __forceinline__ i32x4 scale(i32x4 v, float c) {
        i32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = __float_as_int(__int_as_float(v[j]) * c);
        return r;
    }
    static __device__ __forceinline__ float get1(T b) { return b; }
    static __device__ __forceinline__ T put1(float a) { return a; }
};

// Sum of v over the workgroup's 256 threads, in every thread, in a fixed order.
__device__ __forceinline__ double clip_block_sum(double v, double* shared) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (shared[0] + shared[1]) + (shared[2] + shared[3]);
    __syncthreads();
    return v;
}

template <int TYPE>
__device__ __forceinline__ double clip_chunk_squares(const void* in, int64_t n) {
    using E = ClipElem<TYPE>;
    const typename E::T* g = static_cast<const typename E::T*>(in);
    double s = 0.0;
    const int nv = (int)(n / E::VN);
#pragma unroll 4
    for (int i = threadIdx.x; i < nv; i += 256) {
        i32x4 v;
        __builtin_memcpy(&v, g + (int64_t)i * E::VN, 16);
#pragma unroll
        for (int j = 0; j < E::VN; ++j) {
            const double d = (double)E::get(v, j);
            s = __builtin_fma(d, d, s);
        }
    }
    const int i = nv * E::VN + (int)threadIdx.x;
    if (i < n) {
        const double d = (double)E::get1(g[i]);
        s = __builtin_fma(d, d, s);
    }
    return s;
}

__global__ __launch_bounds__(256) void clip_norm_kernel(ClipTable t, double* __restrict__ slots) {
    __shared__ double shared[4];
    double s = 0.0;
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = clip_tensor_of(t, c);
        const int64_t nt = t.n_type[i], at = (int64_t)(c - t.first[i]) * kClipChunk;
        const int64_t n = min((nt >> 2) - at, (int64_t)kClipChunk);
        const int type = (int)(nt & 3);
        if (type == kClipF32) s += clip_chunk_squares<kClipF32>(static_cast<const float*>(t.in[i]) + at, n);
        else if (type == kClipBf16) s += clip_chunk_squares<kClipBf16>(static_cast<const uint16_t*>(t.in[i]) + at, n);
        else s += clip_chunk_squares<kClipF16>(static_cast<const uint16_t*>(t.in[i]) + at, n);
    }
    s = clip_block_sum(s, shared);
    if (threadIdx.x == 0) slots[blockIdx.x] = s;
}

// All slots into slot 0 (one workgroup), where there are more than every
// workgroup of the second pass should add by itself.
__global__ __launch_bounds__(256) void clip_join_kernel(double* __restrict__ slots, int n) {
    __shared__ double shared[4];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) s += slots[i];
    s = clip_block_sum(s, shared);
    if (threadIdx.x == 0) slots[0] = s;
}

template <int TYPE>
__device__ __forceinline__ void clip_chunk_scale(const void* in, void* out, int64_t n, float c) {
    using E = ClipElem<TYPE>;
    const typename E::T* g = static_cast<const typename E::T*>(in);
    typename E::T* o = static_cast<typename E::T*>(out);
    const int nv = (int)(n / E::VN);
#pragma unroll 4
    for (int i = threadIdx.x; i < nv; i += 256) {
        i32x4 v;
        __builtin_memcpy(&v, g + (int64_t)i * E::VN, 16);
        v = E::scale(v, c);
        __builtin_memcpy(o + (int64_t)i * E::VN, &v, 16);
    }
    const int i = nv * E::VN + (int)threadIdx.x;
    if (i < n) o[i] = E::put1(E::get1(g[i]) * c);
}

__global__ __launch_bounds__(256) void clip_scale_kernel(ClipTable t, const double* __restrict__ slots, int nslots,
                                                         float max_norm, float* __restrict__ norm_out) {
    __shared__ double shared[4];
    double s = 0.0;
    for (int i = threadIdx.x; i < nslots; i += 256) s += slots[i];
    const double norm = sqrt(clip_block_sum(s, shared));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    // a NaN norm stays a NaN factor; an infinite norm gives 0
    const double r = (double)max_norm / (norm + 1e-6);
    const float c = r > 1.0 ? 1.0f : (float)r;
    for (int b = blockIdx.x; b < t.first[t.count]; b += gridDim.x) {
        const int k = t.first[t.count] - 1 - b;
        const int i = clip_tensor_of(t, k);
        if (c == 1.0f && t.in[i] == t.out[i]) continue;   // in place, nothing to clip
        const int64_t nt = t.n_type[i], at = (int64_t)(k - t.first[i]) * kClipChunk;
        const int64_t n = min((nt >> 2) - at, (int64_t)kClipChunk);
        const int type = (int)(nt & 3);
        if (type == kClipF32)
            clip_chunk_scale<kClipF32>(static_cast<const float*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, n, c);
        else if (type == kClipBf16)
            clip_chunk_scale<kClipBf16>(static_cast<const uint16_t*>(t.in[i]) + at,
                                        static_cast<uint16_t*>(t.out[i]) + at, n, c);
        else
            clip_chunk_scale<kClipF16>(static_cast<const uint16_t*>(t.in[i]) + at,
                                       static_cast<uint16_t*>(t.out[i]) + at, n, c);
    }
}

}  // namespace fp8k
