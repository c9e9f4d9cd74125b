// The FP4 key/value cache on gfx950: rows quantised as they are written to their
// slots, and read back.
//
// A row is the D values of one token and head, in blocks of 32.  Written:
//   s    = the least 2^e, -125 <= e <= 125, with max |x| <= 6 s over the block; 1 where
//          the block is all zeros
//   code = the e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to
//          x / s, at most 6 in size, ties to the even mantissa;
// a block that holds a NaN or an infinity gets the scale NaN and codes 0.  Read back:
// code * s, which is a number of bf16.
//
// s comes from the exponent and mantissa of the largest |x|: 1.m 2^E is at most
// 6 * 2^(E - 2) where 1.m <= 1.5, else at most 6 * 2^(E - 1).  x / s is a shift of the
// exponent, so the conversion instruction, which divides by a power of two and rounds
// once, is the definition itself.
//
// Bound: memory, one pass with 16-byte accesses to the rows: a lane holds 8 values,
// four lanes a block, D / 8 a row.  The scale bytes of 128 values meet in one lane,
// which stores them as a word.  Keys and values share a launch (gridDim.y = 2).
#include "fp8_values.h"
#include "row_access.h"
#include "serve_internal.h"

namespace dg {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kLeastScale = 2, kLargestScale = 252;     // 2^-125 and 2^125, biased by 127

struct CopyArgs {
    const int32_t* slots;
    void* rows[2];
    uint8_t* codes[2];
    uint8_t* sf[2];
    int64_t stride[2];
    int64_t total;                  // rows: tokens * H
    int64_t slot_count;             // num_pages * page_size
    int H, page_shift;
};

// The value of lane l + N of the same 16 lanes, in lane l.
template <int N>
__device__ __forceinline__ uint32_t from_right(uint32_t v) {
    return dpp<0x100 + N>(v);
}

template <typename In, int D>
__global__ __launch_bounds__(kThreads) void kv4_cache_write_kernel(CopyArgs a) {
    constexpr int LPR = D / 8;
    const int kv = blockIdx.y;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const int part = threadIdx.x % LPR;
    if (r >= a.total) return;                  // whole rows: LPR divides a wave
    const int64_t t = r / a.H;
    const int h = (int)(r - t * a.H);
    const int slot = a.slots[t];
    float x[8];
    load8(static_cast<const In*>(a.rows[kv]) + t * a.stride[kv] + (int64_t)h * D + part * 8, x);
    // the maximum of the bit patterns of |x| in the block: NaN and infinity come out on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    m = max(m, dpp<0xB1>(m));                  // lane ^ 1
    m = max(m, dpp<0x4E>(m));                  // lane ^ 2
    const bool finite = m < 0x7F800000u;
    const int e = (int)(m >> 23) - 2 + ((m & 0x7FFFFFu) > 0x400000u);
    uint32_t s = (uint32_t)min(max(e, (int)kLeastScale), (int)kLargestScale);
    if (m == 0) s = 127;
    const float scale = __uint_as_float(s << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
    if (!finite) w = 0, s = 255;
    uint32_t sf = s | from_right<4>(s) << 8;
    if constexpr (D > 64) sf |= from_right<8>(s) << 16 | from_right<12>(s) << 24;
    if (slot < 0 || slot >= a.slot_count) return;
    const int64_t row = pool_row(slot, h, a.H, a.page_shift);
    *reinterpret_cast<uint32_t*>(a.codes[kv] + row * (D / 2) + part * 4) = w;
    if constexpr (D == 64) {
        if (part == 0) *reinterpret_cast<uint16_t*>(a.sf[kv] + row * 2) = (uint16_t)sf;
    } else if (part % 16 == 0) {
        *reinterpret_cast<uint32_t*>(a.sf[kv] + row * (D / 32) + part / 4) = sf;
    }
}

// The eight values of a word of codes, stored past the caches.
__device__ __forceinline__ void store_values(uint16_t* p, uint32_t w, float scale) {
    const u32x4_t v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
}

__device__ __forceinline__ void store_values(float* p, uint32_t w, float scale) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1),
                  c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    const float x[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    store8(p, x);
}

template <typename Out, int D>
__global__ __launch_bounds__(kThreads) void kv4_cache_read_kernel(CopyArgs a) {
    constexpr int LPR = D / 8;
    const int kv = blockIdx.y;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const int part = threadIdx.x % LPR;
    if (r >= a.total) return;
    const int64_t t = r / a.H;
    const int h = (int)(r - t * a.H);
    const int slot = a.slots[t];
    uint32_t w = 0, s = 127;
    if (slot >= 0 && slot < a.slot_count) {
        const int64_t row = pool_row(slot, h, a.H, a.page_shift);
        w = *reinterpret_cast<const uint32_t*>(a.codes[kv] + row * (D / 2) + part * 4);
        s = a.sf[kv][row * (D / 32) + part / 4];
    }
    store_values(static_cast<Out*>(a.rows[kv]) + t * a.stride[kv] + (int64_t)h * D + part * 8, w, __uint_as_float(s << 23));
}

template <int D>
hipError_t launch_piece(const CopyArgs& a, bool f32, bool write, hipStream_t stream) {
    constexpr int64_t rows = kThreads / (D / 8);
    const dim3 grid((unsigned)((a.total + rows - 1) / rows), 2), block(kThreads);
    if (write) {
        if (f32) hipLaunchKernelGGL((kv4_cache_write_kernel<float, D>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((kv4_cache_write_kernel<uint16_t, D>), grid, block, 0, stream, a);
    } else {
        if (f32) hipLaunchKernelGGL((kv4_cache_read_kernel<float, D>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((kv4_cache_read_kernel<uint16_t, D>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

// A grid has fewer than 2^32 threads, so tokens beyond 2^31 threads' take further launches.
template <int D>
hipError_t launch(const CopyArgs& a, int64_t T, bool f32, bool write, hipStream_t stream) {
    const int64_t piece = (1ll << 31) / (a.H * (D / 8));         // H is at most 65535
    for (int64_t t = 0; t < T; t += piece) {
        CopyArgs b = a;
        b.slots = a.slots + t;
        for (int i = 0; i < 2; ++i) b.rows[i] = static_cast<char*>(a.rows[i]) + t * a.stride[i] * (f32 ? 4 : 2);
        b.total = (T - t < piece ? T - t : piece) * a.H;
        const hipError_t e = launch_piece<D>(b, f32, write, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch(const KvCopy& p, bool write, hipStream_t stream) {
    CopyArgs a;
    a.slots = p.slots;
    a.rows[0] = p.k; a.rows[1] = p.v;
    a.codes[0] = p.cache.k_codes; a.codes[1] = p.cache.v_codes;
    a.sf[0] = static_cast<uint8_t*>(p.cache.k_sf); a.sf[1] = static_cast<uint8_t*>(p.cache.v_sf);
    a.stride[0] = p.k_stride; a.stride[1] = p.v_stride;
    a.slot_count = p.cache.num_pages * p.cache.page_size;
    a.H = (int)p.cache.H;
    a.page_shift = __builtin_ctzll((unsigned long long)p.cache.page_size);
    switch (p.cache.D) {
    case 64: return launch<64>(a, p.T, p.f32, write, stream);
    case 128: return launch<128>(a, p.T, p.f32, write, stream);
    case 256: return launch<256>(a, p.T, p.f32, write, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_kv4_cache_write(const KvCopy& p, hipStream_t stream) { return launch(p, true, stream); }
hipError_t launch_kv4_cache_read(const KvCopy& p, hipStream_t stream) { return launch(p, false, stream); }

}  // namespace dg
