// Device helpers on e4m3 codes and bf16 fragments shared by the few-token
// kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Two e4m3 bytes of a word (the low or the high half) as two bf16: exact,
// every e4m3 value is a bf16 value.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}

// The same as two fp16, exact too.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}

// Eight consecutive e4m3 bytes as an MFMA fragment of eight bf16.
__device__ __forceinline__ bf16x8_t e4m3x8_to_bf16x8(uint32_t lo, uint32_t hi) {
    u32x4_t r;
    r.x = e4m3x2_to_bf16x2<false>(lo);
    r.y = e4m3x2_to_bf16x2<true>(lo);
    r.z = e4m3x2_to_bf16x2<false>(hi);
    r.w = e4m3x2_to_bf16x2<true>(hi);
    return __builtin_bit_cast(bf16x8_t, r);
}

// Two fp32 as two bf16 in a word, each rounded to nearest even.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float a, float b) {
    bf16x2_t r;
    r.x = (__bf16)a;
    r.y = (__bf16)b;
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float a, float b) {
    f16x2_t r;
    r.x = (_Float16)a;
    r.y = (_Float16)b;
    return __builtin_bit_cast(uint32_t, r);
}

// 16 rows x 32 K of bf16 by 16 columns x 32 K, added to acc: lane l passes
// eight K values of row (and of column) l & 15, the same ones for both
// operands; it gets out[4 * (l >> 4) + i][l & 15], i = 0..3.
__device__ __forceinline__ f32x4_t mfma_bf16(bf16x8_t rows, bf16x8_t cols, f32x4_t acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(rows, cols, acc, 0, 0, 0);
}

__device__ __forceinline__ f32x4_t mfma_f16(f16x8_t rows, f16x8_t cols, f32x4_t acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(rows, cols, acc, 0, 0, 0);
}

// The largest and the sum of a value over lanes l, l ^ 16, l ^ 32 and l ^ 48.
__device__ __forceinline__ float max_of_groups(float v) {
    u32x2_t s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __builtin_fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
    s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_fmaxf(__uint_as_float(s.x), __uint_as_float(s.y));
}

__device__ __forceinline__ float sum_of_groups(float v) {
    u32x2_t s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s.x) + __uint_as_float(s.y);
    s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s.x) + __uint_as_float(s.y);
}

// An input at a uniform place, which the launch does not write: a scalar load,
// also where the kernel has stores behind it, outside the vector loads' order.
__device__ __forceinline__ int uniform_input(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

// A copy of v that the compiler cannot see through: what is derived from it is
// computed where the copy is taken, and not kept in registers across a loop that
// needs them.
__device__ __forceinline__ int fresh(int v) {
    int r;
    asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "v"(v));
    return r;
}

// The value of lane 4 (l / 4) + I, in every lane l.
template <int I>
__device__ __forceinline__ float of_quad(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), I * 0x55, 0xF, 0xF, true));
}

// Inclusive sum of v over the wave's lanes up to each.
__device__ __forceinline__ uint32_t sum_up_to_lane(uint32_t v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
    return v;
}

// Between a wave's LDS writes and reads of the same place by its other lanes:
// the hardware keeps their order, this keeps the compiler from changing it.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace dg
