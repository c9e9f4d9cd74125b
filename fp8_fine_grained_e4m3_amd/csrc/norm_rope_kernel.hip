// Norms of query and key heads with the rotation by position in the same pass, and
// their gradients, gfx950.
//
// A row is the D values of one token and head, w the tensor's weights.
//   n = x r,  r = (mean x^2 + eps)^-1/2,  y = n w,
//   z = y turned: of a pair (y1, y2) with the angle t = position * inv_freq[i],
//       z1 = y1 cos t - y2 sin t,  z2 = y2 cos t + y1 sin t;
// the pairs are values i and i + R / 2 of the first R, or neighbours 2 i, 2 i + 1;
// values from R on are not turned.  Backward, from dz:
//   dy = dz turned by -t,  dw = sum of dy n over all rows,  g = dy w,
//   dx = r (g - n mean(g n)).
//
// Bound: memory; a row is read once and written once.  A lane has 8 values of a row
// (16 bytes of bf16), D / 8 lanes a row, whose sums are exchanges between lanes.
// What a lane needs of a pair's other half comes from the lane that loaded it, as
// loaded (bf16 in halves of words).  Angles are shared by a token's heads: a
// workgroup takes rows that follow one another, and computes the cosines and sines
// of their tokens once, into LDS, while its first rows are on their way.  The angle
// is taken in 64 bits, in turns, and reduced to an eighth of a turn before it is
// rounded to fp32, so far positions lose nothing.
//
// Measured: 16384 tokens of 32 + 8 heads of 128 in bf16, 336 MB, 63 us, 5.3 TB/s (a 2 GiB
// copy: 4.9 to 5.3); their gradients, 503 MB, 104 us, 4.8 TB/s, of which the sums of dw take
// 5.  8192 tokens in fp32, the same bytes: 67 and 107 us.  5 tokens: 3.6 us.  When these took
// 66 and 107 us: plain stores 71; two rows a lane and step instead of four (gradients: of two)
// 71; gradients, whose grid is kBackwardGroups workgroups, each with a sum of dw, in 512 of
// them 118, in 2048 112.
#include "fp8_values.h"
#include "row_access.h"
#include "serve_internal.h"

#include <algorithm>

namespace dg {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
    const void* x[2];                     // queries, keys
    const void* dz[2];
    void* out[2];                         // z, or dx
    int64_t x_stride[2], dz_stride[2], out_stride[2];
    const void* w[2];                     // NULL: ones
    float* dw[2];
    float* parts;                         // sums of dy n of each workgroup, [workgroups, D]
    const int32_t* positions;
    const float* inv_freq;
    float eps;
    uint32_t rows[2], heads[2];
    uint64_t magic[2];                    // row / heads = row * magic >> shift
    int shift[2];
    int groups[2], group_rows;            // workgroups, rows of a step of one
    int half;                             // R / 2
    bool w_f32;
};

template <typename T>
struct Raw;                               // 8 values as they are stored
template <>
struct Raw<uint16_t> { uint32_t w[4]; };
template <>
struct Raw<float> { uint32_t w[8]; };

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(r) / 16; ++i) {
        const u32x4_t v = reinterpret_cast<const u32x4_t*>(p)[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[4 * i + k] = v[k];
    }
    return r;
}

__device__ __forceinline__ void values_of(const Raw<uint16_t>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r.w[i] << 16);
        x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void values_of(const Raw<float>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
}

// Rows of a large problem are stored past the caches, which they would pass through
// before they are read; those of a small one are read from there.
template <int PASSES, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&x)[8]) {
    if constexpr (PASSES > 1) store8(p, x);
    else put8(p, x);
}

template <typename T>
__device__ __forceinline__ Raw<T> from_lane(const Raw<T>& r, int lane) {
    Raw<T> o;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r) / 4); ++i) o.w[i] = (uint32_t)__shfl((int)r.w[i], lane);
    return o;
}

__device__ __forceinline__ void load_weights(const RopeArgs& a, int kind, int at, float (&w)[8]) {
    if (a.w[kind] == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    } else if (a.w_f32) {
        load8(static_cast<const float*>(a.w[kind]) + at, w);
    } else {
        load8(static_cast<const uint16_t*>(a.w[kind]) + at, w);
    }
}

// cos and sin of position * freq.
__device__ __forceinline__ f32x2_t cos_sin(int position, float freq) {
    const double turns = (double)position * (double)freq * 0.15915494309189533577;
    const double quarter = __builtin_rint(4.0 * turns);
    const float f = (float)(2.0 * (turns - 0.25 * quarter));       // half turns, from -1/4 to 1/4
    float s, c;
    sincospif(f, &s, &c);
    const int q = (int)(quarter - 4.0 * __builtin_floor(0.25 * quarter));
    const float x = q & 1 ? s : c, y = q & 1 ? c : s;
    return f32x2_t{q == 1 || q == 2 ? -x : x, q >= 2 ? -y : y};
}

// r of a row: 1 / sqrt(mean x^2 + eps).  Squares that pass fp32's largest number are
// taken again 2^-140 as large.
template <int D>
__device__ __forceinline__ float scale_of_row(const float (&x)[8], float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(x[i], x[i], ss);
    ss = sum_of_row<D / 8>(ss);
    const float a = ss * (1.0f / D) + eps;
    float r = __builtin_amdgcn_rsqf(a);
    r = __builtin_fmaf(0.5f * r, __builtin_fmaf(-a * r, r, 1.0f), r);
    if (__any(ss == __builtin_inff())) {
        float small = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = x[i] * 0x1p-70f;
            small = __builtin_fmaf(y, y, small);
        }
        small = sum_of_row<D / 8>(small);
        if (ss == __builtin_inff()) r = __builtin_amdgcn_rsqf(small * (1.0f / D)) * 0x1p-70f;
    }
    return r;
}

// Where the lane's 8 values stand in the rotation.
struct Turn {
    bool on;                              // they are turned
    int partner;                          // lane with the other halves (the same for neighbours)
    int angle;                            // first of their angles (of values not turned: any)
    float sign;                           // -1: first halves, 1: second ones
};

template <int D, bool NEIGHBOURS>
__device__ __forceinline__ Turn turn_of(int half, int part, int lane) {
    Turn t;
    t.on = part * 8 < 2 * half;
    if (NEIGHBOURS) {
        t.partner = lane;
        t.angle = t.on ? part * 4 : 0;
        t.sign = 0.0f;
    } else {
        const bool second = part * 8 >= half;
        t.partner = t.on ? (second ? lane - half / 8 : lane + half / 8) : lane;
        t.angle = !t.on ? 0 : second ? part * 8 - half : part * 8;
        t.sign = second ? 1.0f : -1.0f;
    }
    return t;
}

// The lane's 8 values turned: own and, where pairs are halves, the partner's ones.
// sign 1 turns by the angle, -1 back.  Values that are not turned pass as they are: a
// product with a sine of 0 would make NaN of an infinity beside or at them.
template <bool NEIGHBOURS>
__device__ __forceinline__ void turn(const Turn& t, const f32x2_t* angles, float sign, const float (&own)[8],
                                     const float (&other)[8], float (&z)[8]) {
    if (NEIGHBOURS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2_t cs = angles[t.angle + i];
            const float s = sign * cs.y;
            const float a = own[2 * i] * cs.x - own[2 * i + 1] * s, b = own[2 * i + 1] * cs.x + own[2 * i] * s;
            z[2 * i] = t.on ? a : own[2 * i];
            z[2 * i + 1] = t.on ? b : own[2 * i + 1];
        }
    } else {
        const float way = sign * t.sign;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const f32x2_t cs = angles[t.angle + i];
            const float a = own[i] * cs.x + other[i] * (way * cs.y);
            z[i] = t.on ? a : own[i];
        }
    }
}

// Cosines and sines of tokens first to last into LDS.
__device__ __forceinline__ void fill_angles(const RopeArgs& a, uint32_t first, uint32_t last, f32x2_t* angles) {
    const uint32_t n = (last - first + 1) * (uint32_t)a.half;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t t = i / (uint32_t)a.half;
        angles[i] = cos_sin(a.positions[first + t], a.inv_freq[i - t * (uint32_t)a.half]);
    }
}

__device__ __forceinline__ uint32_t token_of(const RopeArgs& a, int kind, uint32_t row) {
    return (uint32_t)((uint64_t)row * a.magic[kind] >> a.shift[kind]);
}

// A workgroup's step is PASSES times the rows that its lanes hold at once.
template <typename T, int D, bool NEIGHBOURS, int PASSES>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(RopeArgs a) {
    constexpr int LPR = D / 8, RPP = kThreads / LPR;
    extern __shared__ f32x2_t sm_angles[];
    const int kind = (int)blockIdx.x >= a.groups[0], group = (int)blockIdx.x - (kind ? a.groups[0] : 0);
    const int lane = threadIdx.x & 63, part = threadIdx.x % LPR;
    const uint32_t rows = a.rows[kind];
    float w[8], wo[8];
    load_weights(a, kind, part * 8, w);
    const Turn t = turn_of<D, NEIGHBOURS>(a.half, part, lane);
    if (!NEIGHBOURS) load_weights(a, kind, (part + t.partner - lane) * 8, wo);
    for (uint32_t row0 = (uint32_t)group * (PASSES * RPP); row0 < rows; row0 += (uint32_t)a.groups[kind] * (PASSES * RPP)) {
        Raw<T> raw[PASSES];
        uint32_t token[PASSES], head[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const uint32_t row = min(row0 + p * RPP + threadIdx.x / LPR, rows - 1);
            token[p] = token_of(a, kind, row);
            head[p] = row - token[p] * a.heads[kind];
            raw[p] = load_raw(static_cast<const T*>(a.x[kind]) + token[p] * a.x_stride[kind] + head[p] * D + part * 8);
        }
        const uint32_t first = token_of(a, kind, row0), last = token_of(a, kind, min(row0 + PASSES * RPP, rows) - 1);
        fill_angles(a, first, last, sm_angles);
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            float x[8], other[8], z[8];
            values_of(raw[p], x);
            const float r = scale_of_row<D>(x, a.eps);
            if (!NEIGHBOURS) {
                values_of(from_lane(raw[p], t.partner), other);
#pragma unroll
                for (int i = 0; i < 8; ++i) other[i] = other[i] * r * wo[i];
            }
            // the row's factor first: r * w may leave fp32's range where n * w does not
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
            turn<NEIGHBOURS>(t, sm_angles + (token[p] - first) * a.half, 1.0f, x, other, z);
            if (row0 + p * RPP + threadIdx.x / LPR < rows)
                store_row<PASSES>(static_cast<T*>(a.out[kind]) + token[p] * a.out_stride[kind] + head[p] * D + part * 8, z);
        }
        __syncthreads();
    }
}

template <typename T, int D, bool NEIGHBOURS, int PASSES>
__global__ __launch_bounds__(kThreads) void norm_rope_backward_kernel(RopeArgs a) {
    constexpr int LPR = D / 8, RPP = kThreads / LPR;
    extern __shared__ f32x2_t sm_angles[];
    __shared__ float sm_sum[RPP][D + 4];
    const int kind = (int)blockIdx.x >= a.groups[0], group = (int)blockIdx.x - (kind ? a.groups[0] : 0);
    const int lane = threadIdx.x & 63, part = threadIdx.x % LPR;
    const uint32_t rows = a.rows[kind];
    float w[8], dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    load_weights(a, kind, part * 8, w);
    const Turn t = turn_of<D, NEIGHBOURS>(a.half, part, lane);
    for (uint32_t row0 = (uint32_t)group * (PASSES * RPP); row0 < rows; row0 += (uint32_t)a.groups[kind] * (PASSES * RPP)) {
        Raw<T> raw[PASSES], draw[PASSES];
        uint32_t token[PASSES], head[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const uint32_t row = min(row0 + p * RPP + threadIdx.x / LPR, rows - 1);
            token[p] = token_of(a, kind, row);
            head[p] = row - token[p] * a.heads[kind];
            raw[p] = load_raw(static_cast<const T*>(a.x[kind]) + token[p] * a.x_stride[kind] + head[p] * D + part * 8);
            draw[p] = load_raw(static_cast<const T*>(a.dz[kind]) + token[p] * a.dz_stride[kind] + head[p] * D + part * 8);
        }
        const uint32_t first = token_of(a, kind, row0), last = token_of(a, kind, min(row0 + PASSES * RPP, rows) - 1);
        fill_angles(a, first, last, sm_angles);
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const bool live = row0 + p * RPP + threadIdx.x / LPR < rows;
            float x[8], dz[8], other[8], dy[8];
            values_of(raw[p], x);
            values_of(draw[p], dz);
            const float r = scale_of_row<D>(x, a.eps);
            if (!NEIGHBOURS) values_of(from_lane(draw[p], t.partner), other);
            turn<NEIGHBOURS>(t, sm_angles + (token[p] - first) * a.half, -1.0f, dz, other, dy);
            float gn = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= r;                                 // n
                if (live) dw[i] = __builtin_fmaf(dy[i], x[i], dw[i]);
                dy[i] *= w[i];                             // g
                gn = __builtin_fmaf(dy[i], x[i], gn);
            }
            gn = sum_of_row<LPR>(gn) * (1.0f / D);
#pragma unroll
            for (int i = 0; i < 8; ++i) dy[i] = r * __builtin_fmaf(-x[i], gn, dy[i]);
            if (live) store_row<PASSES>(static_cast<T*>(a.out[kind]) + token[p] * a.out_stride[kind] + head[p] * D + part * 8, dy);
        }
        __syncthreads();
    }
    if (a.dw[kind] == nullptr) return;
    // the workgroup's sum, row by row
#pragma unroll
    for (int i = 0; i < 8; ++i) sm_sum[threadIdx.x / LPR][part * 8 + i] = dw[i];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < RPP; ++r) s += sm_sum[r][d];
        a.parts[(int64_t)blockIdx.x * D + d] = s;
    }
}

// dw: the workgroups' sums, 32 of them side by side for each value, always in the same order.
__global__ __launch_bounds__(1024) void norm_rope_weights_kernel(RopeArgs a, int D) {
    __shared__ float sm_sum[32][33];
    const int kind = blockIdx.y, d = blockIdx.x * 32 + threadIdx.x % 32, side = threadIdx.x / 32;
    if (a.dw[kind] == nullptr) return;
    const float* parts = a.parts + (int64_t)(kind ? a.groups[0] : 0) * D + d;
    float s = 0.0f;
#pragma unroll 4
    for (int g = side; g < a.groups[kind]; g += 32) s += parts[(int64_t)g * D];
    sm_sum[side][threadIdx.x % 32] = s;
    __syncthreads();
    if (side > 0) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += sm_sum[k][threadIdx.x];
    a.dw[kind][d] = s;
}

// Passes of a step and workgroups of a problem.
struct Plan {
    int passes;
    int groups[2];
};

constexpr int kBackwardGroups = 1024;     // at most this many sums of dw

Plan plan_of(int64_t T, int64_t Hq, int64_t H, int64_t D, bool backward) {
    const int64_t rpp = kThreads / (D / 8), rows[2] = {T * Hq, T * H};
    Plan p;
    p.passes = (rows[0] + rows[1]) / rpp > 2048 ? (backward ? 2 : 4) : 1;
    int64_t n[2];
    for (int i = 0; i < 2; ++i) n[i] = (rows[i] + rpp * p.passes - 1) / (rpp * p.passes);
    const int64_t most = backward ? kBackwardGroups : 1 << 20;
    for (int i = 0; i < 2; ++i) {
        const int64_t share = n[0] + n[1] <= most ? n[i] : std::max<int64_t>(1, most * n[i] / (n[0] + n[1]));
        p.groups[i] = (int)std::min(n[i], share);
    }
    return p;
}

template <typename T, int D, bool NEIGHBOURS, int PASSES, bool BACKWARD>
hipError_t launch_passes(const RopeArgs& a, hipStream_t stream) {
    // tokens that the rows of a step may touch
    const uint32_t rows = PASSES * (kThreads / (D / 8));
    uint32_t tokens = 0;
    for (int i = 0; i < 2; ++i)
        if (a.groups[i] > 0) tokens = std::max(tokens, std::min(a.rows[i] / a.heads[i], (rows + a.heads[i] - 2) / a.heads[i] + 1));
    const dim3 grid((unsigned)(a.groups[0] + a.groups[1]));
    const uint32_t lds = std::max(tokens * (uint32_t)a.half * 8, 64u);   // eight angles are read where none are turned
    if constexpr (BACKWARD)
        hipLaunchKernelGGL((norm_rope_backward_kernel<T, D, NEIGHBOURS, PASSES>), grid, dim3(kThreads), lds, stream, a);
    else
        hipLaunchKernelGGL((norm_rope_kernel<T, D, NEIGHBOURS, PASSES>), grid, dim3(kThreads), lds, stream, a);
    return hipGetLastError();
}

template <typename T, int D, bool NEIGHBOURS>
hipError_t launch_rows(const RopeArgs& a, int passes, bool backward, hipStream_t stream) {
    if (backward) return passes == 1 ? launch_passes<T, D, NEIGHBOURS, 1, true>(a, stream) : launch_passes<T, D, NEIGHBOURS, 2, true>(a, stream);
    return passes == 1 ? launch_passes<T, D, NEIGHBOURS, 1, false>(a, stream) : launch_passes<T, D, NEIGHBOURS, 4, false>(a, stream);
}

template <typename T, int D>
hipError_t launch_pairs(const RopeArgs& a, bool neighbours, int passes, bool backward, hipStream_t stream) {
    return neighbours ? launch_rows<T, D, true>(a, passes, backward, stream) : launch_rows<T, D, false>(a, passes, backward, stream);
}

template <typename T>
hipError_t launch_dim(const RopeArgs& a, int64_t D, bool neighbours, int passes, bool backward, hipStream_t stream) {
    switch (D) {
    case 64: return launch_pairs<T, 64>(a, neighbours, passes, backward, stream);
    case 128: return launch_pairs<T, 128>(a, neighbours, passes, backward, stream);
    case 256: return launch_pairs<T, 256>(a, neighbours, passes, backward, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

int64_t norm_rope_workspace_bytes(int64_t T, int64_t Hq, int64_t H, int64_t D) {
    const Plan p = plan_of(T, Hq, H, D, true);
    return (int64_t)(p.groups[0] + p.groups[1]) * D * 4;
}

hipError_t launch_norm_rope(const NormRope& p, hipStream_t stream) {
    const bool backward = p.backward;
    const Plan plan = plan_of(p.T, p.Hq, p.H, p.D, backward);
    RopeArgs a;
    for (int i = 0; i < 2; ++i) {
        a.x[i] = p.x[i]; a.dz[i] = p.dz[i]; a.out[i] = p.out[i];
        a.x_stride[i] = p.x_stride[i]; a.dz_stride[i] = p.dz_stride[i]; a.out_stride[i] = p.out_stride[i];
        a.w[i] = p.w[i]; a.dw[i] = p.dw[i];
        a.heads[i] = (uint32_t)(i ? p.H : p.Hq);
        a.rows[i] = (uint32_t)(p.T * a.heads[i]);
        a.groups[i] = plan.groups[i];
        // row / heads for rows below 2^31: 2^(31 + l) / heads rounded up, l = ceil(log2 heads)
        int l = 0;
        while ((1u << l) < a.heads[i]) ++l;
        a.shift[i] = 31 + l;
        a.magic[i] = a.heads[i] > 0 ? (1ull << a.shift[i]) / a.heads[i] + 1 : 0;
    }
    a.parts = static_cast<float*>(p.workspace);
    a.positions = p.positions; a.inv_freq = p.inv_freq;
    a.eps = p.eps; a.half = (int)(p.R / 2); a.w_f32 = p.w_f32;
    if (a.groups[0] + a.groups[1] > 0) {
        const hipError_t e = p.f32 ? launch_dim<float>(a, p.D, p.neighbours, plan.passes, backward, stream)
                                   : launch_dim<uint16_t>(a, p.D, p.neighbours, plan.passes, backward, stream);
        if (e != hipSuccess) return e;
    }
    if (backward && (a.dw[0] || a.dw[1]))
        hipLaunchKernelGGL(norm_rope_weights_kernel, dim3((unsigned)(p.D / 32), 2), dim3(1024), 0, stream, a, (int)p.D);
    return hipGetLastError();
}

}  // namespace dg
