// Eight values of a bf16 or fp32 row in a lane, and rows of a paged cache.
#pragma once

#include "fp8_values.h"

namespace dg {

__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const f32x4_t a = reinterpret_cast<const f32x4_t*>(p)[0], b = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}

// Stored past the caches (store8) or through them (put8).
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2(x[2 * i], x[2 * i + 1]);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    f32x4_t a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x[i], b[i] = x[4 + i];
    __builtin_nontemporal_store(a, reinterpret_cast<f32x4_t*>(p));
    __builtin_nontemporal_store(b, reinterpret_cast<f32x4_t*>(p) + 1);
}

__device__ __forceinline__ void put8(uint16_t* p, const float (&x)[8]) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<u32x4_t*>(p) = w;
}

__device__ __forceinline__ void put8(float* p, const float (&x)[8]) {
    f32x4_t a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x[i], b[i] = x[4 + i];
    reinterpret_cast<f32x4_t*>(p)[0] = a;
    reinterpret_cast<f32x4_t*>(p)[1] = b;
}

// Row of the pool ([page][head][offset], in rows) of a slot and head.
__device__ __forceinline__ int64_t pool_row(int slot, int h, int H, int page_shift) {
    const int64_t page = slot >> page_shift;
    const int at = slot & ((1 << page_shift) - 1);
    return ((page * H + h) << page_shift) + at;
}

// The value of another lane, by a DPP control; and the sum of a value over the LPR lanes
// that hold a row (4, 8, 16 or 32 lanes, on a multiple of that).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

template <int LPR>
__device__ __forceinline__ float sum_of_row(float v) {
    v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));                     // lane ^ 1
    v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));                     // lane ^ 2
    if constexpr (LPR >= 8) v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));     // the other four of eight
    if constexpr (LPR >= 16) v += __uint_as_float(dpp<0x140>(__float_as_uint(v)));    // the other eight of sixteen
    if constexpr (LPR >= 32) {
        const u32x2_t s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(s.x) + __uint_as_float(s.y);
    }
    return v;
}

}  // namespace dg
