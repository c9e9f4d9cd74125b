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
// Bound: memory, one pass with 16-byte accesses to the rows: a lane holds 8 values
// (4 of an fp32 row that is read), four lanes a block, D / 8 a row.  The scale bytes of 128
// values meet in one lane, which stores them as a word.  Keys and values share a launch
// (gridDim.y = 2).  Read rows are stored past the caches; written codes are not, the
// attention that follows reads them.
// Measured: 40000 tokens of 8 heads of 128 in bf16, 208 MB: written in 45 us, 4.7 TB/s (46
// with a token's heads side by side in a workgroup), read in 33 us, 6.3 TB/s (39 with one
// row a lane); 16384 tokens, 85 MB, 20 and 15 us; 16384 of 4 heads in fp32, 16 and 14 us (17 with
// 8 values a lane, in two stores); 5 tokens, 2.7 us each.
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
    int64_t tokens, total;          // rows: tokens * H
    int64_t slot_count;             // num_pages * page_size
    int H, page_shift;
};

// The value of lane l + N of the same 16 lanes, in lane l.
template <int N>
__device__ __forceinline__ uint32_t from_right(uint32_t v) {
    return dpp<0x100 + N>(v);
}

// A workgroup has one head of tokens that follow one another, whose codes are neighbours in
// a page: rows of 32 to 128 bytes make whole cache lines in one XCD's cache.
template <typename In, int D>
__global__ __launch_bounds__(kThreads) void kv4_cache_write_kernel(CopyArgs a) {
    constexpr int LPR = D / 8;
    const int kv = blockIdx.y, part = threadIdx.x % LPR;
    const uint32_t group = blockIdx.x / (uint32_t)a.H;
    const int h = (int)(blockIdx.x - group * (uint32_t)a.H);
    const int64_t t = (int64_t)group * (kThreads / LPR) + threadIdx.x / LPR;
    if (t >= a.tokens) return;                 // whole rows: LPR divides a wave
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

// The values of a lane's codes as 16 bytes, stored past the caches.
__device__ __forceinline__ void store_values(uint16_t* p, uint32_t w, float scale) {
    const u32x4_t v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
}

__device__ __forceinline__ void store_values(float* p, uint32_t w, float scale) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    __builtin_nontemporal_store(f32x4_t{a.x, a.y, b.x, b.y}, reinterpret_cast<f32x4_t*>(p));
}

// A lane makes 16 bytes of R rows: 8 values of bf16, 4 of fp32.
template <typename Out, int D, int R>
__global__ __launch_bounds__(kThreads) void kv4_cache_read_kernel(CopyArgs a) {
    constexpr int EPL = 16 / sizeof(Out), LPR = D / EPL, RPB = kThreads / LPR;
    const int kv = blockIdx.y, part = threadIdx.x % LPR;
    const int64_t first = (int64_t)blockIdx.x * (R * RPB) + threadIdx.x / LPR;
    if (first >= a.total) return;
    uint32_t w[R], s[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t r = first + k * RPB, t = r / a.H;
        const int slot = r < a.total ? a.slots[t] : -1;
        w[k] = 0;
        s[k] = 127;
        if (slot >= 0 && slot < a.slot_count) {
            const int64_t row = pool_row(slot, (int)(r - t * a.H), a.H, a.page_shift);
            const uint8_t* codes = a.codes[kv] + row * (D / 2) + part * (EPL / 2);
            if constexpr (EPL == 8) w[k] = *reinterpret_cast<const uint32_t*>(codes);
            else w[k] = *reinterpret_cast<const uint16_t*>(codes);
            s[k] = a.sf[kv][row * (D / 32) + part * EPL / 32];
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t r = first + k * RPB;     // rows are dense
        if (r < a.total) store_values(static_cast<Out*>(a.rows[kv]) + r * D + part * EPL, w[k], __uint_as_float(s[k] << 23));
    }
}

template <typename Out, int D>
hipError_t launch_read(const CopyArgs& a, hipStream_t stream) {
    constexpr int64_t rows = kThreads / (D * sizeof(Out) / 16);
    // four rows a lane where that leaves more workgroups than are resident
    if (a.total > 4096 * rows) {
        hipLaunchKernelGGL((kv4_cache_read_kernel<Out, D, 4>), dim3((unsigned)((a.total + 4 * rows - 1) / (4 * rows)), 2), dim3(kThreads), 0,
                           stream, a);
    } else {
        hipLaunchKernelGGL((kv4_cache_read_kernel<Out, D, 1>), dim3((unsigned)((a.total + rows - 1) / rows), 2), dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

template <int D>
hipError_t launch_piece(const CopyArgs& a, bool f32, bool write, hipStream_t stream) {
    if (!write) return f32 ? launch_read<float, D>(a, stream) : launch_read<uint16_t, D>(a, stream);
    constexpr int64_t rows = kThreads / (D / 8);
    const dim3 grid((unsigned)((a.tokens + rows - 1) / rows * a.H), 2), block(kThreads);
    if (f32) hipLaunchKernelGGL((kv4_cache_write_kernel<float, D>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((kv4_cache_write_kernel<uint16_t, D>), grid, block, 0, stream, a);
    return hipGetLastError();
}

// A grid has fewer than 2^32 threads a side, so tokens beyond 2^31 threads' take further
// launches (many fp32 reads have four rows a lane, half as many threads as the others).
template <int D>
hipError_t launch(const CopyArgs& a, int64_t T, bool f32, bool write, hipStream_t stream) {
    const int64_t piece = (1ll << 31) / (a.H * (D / 8));         // H is at most 65535
    for (int64_t t = 0; t < T; t += piece) {
        CopyArgs b = a;
        b.slots = a.slots + t;
        for (int i = 0; i < 2; ++i) b.rows[i] = static_cast<char*>(a.rows[i]) + t * a.stride[i] * (f32 ? 4 : 2);
        b.tokens = T - t < piece ? T - t : piece;
        b.total = b.tokens * a.H;
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
