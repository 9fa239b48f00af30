// rows_common.h -- helpers of the kernels that move rows of tokens (routing,
// the experts' rows, adapters): vectors of 16 bytes at any element alignment,
// and reductions over a wave, for gfx950.
#pragma once

#include "device_common.h"

namespace fp8k {

// Element types of rows: VN elements per 16-byte vector, widened to FP32.
template <typename T>
struct RowElem;
template <>
struct RowElem<float> {
    static constexpr int VN = 4;
    static __device__ __forceinline__ float get(i32x4 v, int i) { return __int_as_float(v[i]); }
    static __device__ __forceinline__ i32x4 pack(const float* f) {
        return i32x4{__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]), __float_as_int(f[3])};
    }
    static __device__ __forceinline__ float get1(float b) { return b; }
    static __device__ __forceinline__ float put1(float f) { return f; }
};
template <>
struct RowElem<uint16_t> {      // BF16 bits
    static constexpr int VN = 8;
    static __device__ __forceinline__ float get(i32x4 v, int i) {
        const uint32_t w = (uint32_t)v[i >> 1];
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
    static __device__ __forceinline__ i32x4 pack(const float* f) {
        return i32x4{(int)pack_bf16x2(f[0], f[1]), (int)pack_bf16x2(f[2], f[3]), (int)pack_bf16x2(f[4], f[5]),
                     (int)pack_bf16x2(f[6], f[7])};
    }
    static __device__ __forceinline__ float get1(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ uint16_t put1(float f) { return (uint16_t)(pack_bf16x2(f, 0.f) & 0xFFFFu); }
};

// The 16 bytes at p, of which `left` elements (more than none) belong to the
// row: whole vectors at any alignment, a row's last ones element by element.
// STREAM: with the nontemporal hint, for what is read once or does not fit the
// caches.
typedef i32x4 i32x4_any __attribute__((aligned(2)));

template <typename T, bool STREAM = false>
__device__ __forceinline__ i32x4 load_row16(const T* p, int64_t left) {
    i32x4 v{0, 0, 0, 0};
    if (left >= RowElem<T>::VN) {
        if constexpr (STREAM) v = __builtin_nontemporal_load(reinterpret_cast<const i32x4_any*>(p));
        else __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < RowElem<T>::VN - 1; ++i) {
            if (i < left) {
                if constexpr (sizeof(T) == 4) v[i] = __float_as_int(p[i]);
                else v[i >> 1] |= (int)((uint32_t)p[i] << (16 * (i & 1)));
            }
        }
    }
    return v;
}
template <typename T, bool STREAM = false>
__device__ __forceinline__ void store_row16(T* p, int64_t left, i32x4 v) {
    if (left >= RowElem<T>::VN) {
        if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<i32x4_any*>(p));
        else __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int i = 0; i < RowElem<T>::VN - 1; ++i) {
            if (i < left) {
                if constexpr (sizeof(T) == 4) p[i] = __int_as_float(v[i]);
                else p[i] = (uint16_t)((uint32_t)v[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

// Reductions over the 64 lanes in a fixed order, by lane shifts within rows of
// 16 and broadcasts between them; every lane gets the result.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_shift0(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    auto up = [](uint32_t a, uint32_t b) FP8K_INLINE { return a > b ? a : b; };
    v = up(v, lane_shift0<0x111, 0xF>(v));
    v = up(v, lane_shift0<0x112, 0xF>(v));
    v = up(v, lane_shift0<0x114, 0xF>(v));
    v = up(v, lane_shift0<0x118, 0xF>(v));
    v = up(v, lane_shift0<0x142, 0xA>(v));
    v = up(v, lane_shift0<0x143, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float f) {
    auto add = [](float a, uint32_t b) FP8K_INLINE { return a + __uint_as_float(b); };
    f = add(f, lane_shift0<0x111, 0xF>(__float_as_uint(f)));
    f = add(f, lane_shift0<0x112, 0xF>(__float_as_uint(f)));
    f = add(f, lane_shift0<0x114, 0xF>(__float_as_uint(f)));
    f = add(f, lane_shift0<0x118, 0xF>(__float_as_uint(f)));
    f = add(f, lane_shift0<0x142, 0xA>(__float_as_uint(f)));
    f = add(f, lane_shift0<0x143, 0xC>(__float_as_uint(f)));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), 63));
}

}  // namespace fp8k
