// The FP8 key/value cache on gfx950: rows quantised as they are written to
// their slots, and read back.
//
// A row is the D values of one token and head.  Written:
//   s    = max |x| / 448 (fp32, correctly rounded; 1 where that is 0)
//   code = the e4m3 value nearest to clamp(x / s, -448, 448), x / s the
//          correctly rounded fp32 quotient, ties to the even mantissa;
// a row that holds a NaN or an infinity gets s = NaN and codes 0, so that it
// reads as NaN wherever it is used and nowhere else.  Read back: code * s in
// fp32 (one rounding), rounded once more for bf16.
//
// Bound: memory.  A value is read and written once, so the kernels are one
// pass with 16-byte accesses: a lane holds 8 values of a row, D / 8 lanes a
// row, and the row's maximum is log2(D / 8) exchanges between lanes.  Keys and
// values share a launch (gridDim.y = 2), which halves the launches of a decode
// step.  Read rows are stored past the caches (40000 tokens of 8 heads of 128
// values as bf16, 249 MB: 47 us, 5.2 TB/s, against 64 us with plain stores);
// written codes are not, the attention that follows reads them.  16384 tokens of
// that shape are written in 23 us, 4.4 TB/s of the 101 MB that pass.
#include "fp8_values.h"
#include "row_access.h"
#include "serve_internal.h"

namespace dg {
namespace {

constexpr float kMaxE4m3 = 448.0f;
constexpr int kThreads = 256;
constexpr int kEpl = 8;             // values a lane

struct CopyArgs {
    const int32_t* slots;
    void* rows[2];
    uint8_t* codes[2];
    float* sf[2];
    int64_t stride[2];
    int64_t total;                  // rows: tokens * H
    int64_t slot_count;             // num_pages * page_size
    int H, page_shift;
};

// x / s, correctly rounded, given y = 1 / s correctly rounded: each correction adds
// the exact remainder x - q s times y, the first leaves q within a unit in the
// last place, and from such a q a correction with a correctly rounded reciprocal
// gives the rounded quotient (Markstein).  The remainder is a multiple of the last
// places of q and s multiplied, and exact where that is a number of fp32: from
// s = 2^-92 on for q >= 2^-11.  (Less than that is below half the smallest code, with
// an exact remainder or not.)
constexpr float kLeastScale = 0x1p-92f;

__device__ __forceinline__ float quotient(float x, float s, float y) {
#pragma clang fp contract(off)
    float q = x * y;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x), y, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x), y, q);
    return __builtin_copysignf(q, x);         // the corrections lose the sign of a zero
}

template <typename In, int D>
__global__ __launch_bounds__(kThreads) void kv_cache_write_kernel(CopyArgs a) {
    constexpr int LPR = D / kEpl;
    const int kv = blockIdx.y;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const int part = threadIdx.x % LPR;
    if (r >= a.total) return;                  // whole rows: LPR divides a wave
    const int64_t t = r / a.H;
    const int h = (int)(r - t * a.H);
    const int slot = a.slots[t];
    float x[8];
    load8(static_cast<const In*>(a.rows[kv]) + t * a.stride[kv] + (int64_t)h * D + part * kEpl, x);
    // the maximum of the bit patterns of |x|: NaN and infinity come out on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    const bool finite = m < 0x7F800000u;
    float s = __uint_as_float(m) / kMaxE4m3;
    if (s == 0.0f) s = 1.0f;
    const float y = 1.0f / s;
    const bool exact = s >= kLeastScale;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = exact ? quotient(x[i], s, y) : x[i] / s;
        q[i] = finite ? __builtin_fminf(__builtin_fmaxf(q[i], -kMaxE4m3), kMaxE4m3) : 0.0f;
    }
    if (slot < 0 || slot >= a.slot_count) return;
    const int64_t row = pool_row(slot, h, a.H, a.page_shift);
    u32x2_t w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], c, true);
        w[i] = (uint32_t)c;
    }
    *reinterpret_cast<u32x2_t*>(a.codes[kv] + row * D + part * kEpl) = w;
    if (part == 0) a.sf[kv][row] = finite ? s : __builtin_nanf("");
}

template <typename Out, int D>
__global__ __launch_bounds__(kThreads) void kv_cache_read_kernel(CopyArgs a) {
    constexpr int LPR = D / kEpl;
    const int kv = blockIdx.y;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const int part = threadIdx.x % LPR;
    if (r >= a.total) return;
    const int64_t t = r / a.H;
    const int h = (int)(r - t * a.H);
    const int slot = a.slots[t];
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0 && slot < a.slot_count) {
        const int64_t row = pool_row(slot, h, a.H, a.page_shift);
        const float s = a.sf[kv][row];
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(a.codes[kv] + row * D + part * kEpl);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            x[4 * i] = lo.x * s;
            x[4 * i + 1] = lo.y * s;
            x[4 * i + 2] = hi.x * s;
            x[4 * i + 3] = hi.y * s;
        }
    }
    store8(static_cast<Out*>(a.rows[kv]) + t * a.stride[kv] + (int64_t)h * D + part * kEpl, x);
}

template <int D>
hipError_t launch_piece(const CopyArgs& a, bool f32, bool write, hipStream_t stream) {
    constexpr int64_t rows = kThreads / (D / kEpl);
    const dim3 grid((unsigned)((a.total + rows - 1) / rows), 2), block(kThreads);
    if (write) {
        if (f32) hipLaunchKernelGGL((kv_cache_write_kernel<float, D>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((kv_cache_write_kernel<uint16_t, D>), grid, block, 0, stream, a);
    } else {
        if (f32) hipLaunchKernelGGL((kv_cache_read_kernel<float, D>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((kv_cache_read_kernel<uint16_t, D>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

// A grid has fewer than 2^32 threads, so tokens beyond 2^31 threads' take further launches.
template <int D>
hipError_t launch(const CopyArgs& a, int64_t T, bool f32, bool write, hipStream_t stream) {
    const int64_t piece = (1ll << 31) / (a.H * (D / kEpl));      // H is at most 65535
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
    a.sf[0] = static_cast<float*>(p.cache.k_sf); a.sf[1] = static_cast<float*>(p.cache.v_sf);
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

hipError_t launch_kv_cache_write(const KvCopy& p, hipStream_t stream) { return launch(p, true, stream); }
hipError_t launch_kv_cache_read(const KvCopy& p, hipStream_t stream) { return launch(p, false, stream); }

}  // namespace dg
