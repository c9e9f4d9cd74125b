// What the tree attention kernels of the FP8 and the FP4 cache share: their
// arguments, how a call's work is cut into runs, and the join of what was cut.
//
// The rows of one key head are a request's n tokens times the G query heads that
// share it (row = token * G + head); a row block is 16 or 32 of them.  Steps of 32
// keys of all requests, end to end, are cut into equal runs, and a workgroup goes
// through the requests that its run touches.  Where a run ends inside a request, its
// O, maximum and sum go to the workspace, and a second kernel joins a request's
// parts in order, a thread for four values of a row.
#pragma once

#include "fp8_values.h"
#include "serve_internal.h"

#include <algorithm>

namespace dg {
namespace {

constexpr int kStep = 32;                 // keys of a wave's step
// O is put down 2^kSpare too small: waves and parts (at most 8 x 768 over the FP8 cache, 16 x
// 256 over the FP4 one), each with a sum below 1, then add up without passing fp32's largest
// number, whatever the values.
constexpr int kSpare = 13;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    const uint8_t* kc;
    const void* ks;                       // scales, of the cache's type
    const uint8_t* vc;
    const void* vs;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* tree;
    const uint64_t* mask;
    uint16_t* o;
    float* lse;
    int2* split;                          // [B, H, row blocks]: first and last run of a request; last < first: one
    float* parts;                         // [runs * H, row blocks, 2]: O [ROWS, D], then maxima and sums [ROWS, 2]
    float scale;
    int B, N, H, G, num_pages, page_shift, max_pages, mask_words;
    int runs, row_blocks;
    bool whole;                           // a run is a request
};

// A request's context, tree and the steps of row block rb over them.
struct Request {
    int ctx, n, L, steps;
};

__device__ __forceinline__ Request request_of(const AttnArgs& a, int ctx, int n, int first_row) {
    const int most = a.max_pages << a.page_shift;
    Request r;
    r.ctx = min(max(ctx, 0), most);
    r.n = min(max(n, 0), a.N);
    r.L = min(r.ctx + r.n, most);
    r.steps = first_row < r.n * a.G ? (r.L + kStep - 1) / kStep : 0;
    return r;
}

__device__ __forceinline__ Request request(const AttnArgs& a, int b, int first_row) {   // b uniform
    return request_of(a, uniform_input(a.ctx + b), a.tree ? uniform_input(a.tree + b) : a.N, first_row);
}

__device__ __forceinline__ int steps_of_lane(const AttnArgs& a, int b, int first_row) {
    return b < a.B ? request_of(a, a.ctx[b], a.tree ? a.tree[b] : a.N, first_row).steps : 0;
}

// Joins the parts of requests that were split: D / 4 threads a row and SIDE of
// them side by side, which go through the parts with a running maximum, four at
// a time, and meet in LDS.
template <int D, int SIDE>
__global__ __launch_bounds__(256) void tree_attn_join_kernel(AttnArgs a, int rows_of_block, int64_t first_row) {
    constexpr int TPR = D / 4, RPB = 256 / (TPR * SIDE);
    static_assert(SIDE == 1 || RPB == 1, "threads that meet return together");
    __shared__ f32x4_t sm_v[SIDE > 1 ? 256 : 1];
    __shared__ float sm_ml[SIDE > 1 ? 256 : 1][2];
    const int all_rows = a.N * a.G;
    const int side = threadIdx.x / TPR % SIDE, d = threadIdx.x % TPR * 4;
    const int64_t id = first_row + (int64_t)blockIdx.x * RPB + threadIdx.x / (TPR * SIDE);   // (b, h, row)
    if (id >= (int64_t)a.B * a.H * all_rows) return;
    const int64_t bh = id / all_rows;
    const int r = (int)(id - bh * all_rows), b = (int)(bh / a.H), h = (int)(bh - (int64_t)b * a.H);
    const int rb = r / rows_of_block, in_block = r - rb * rows_of_block;
    const int2 split = a.split[bh * a.row_blocks + rb];
    const int n = a.tree ? min(max(a.tree[b], 0), a.N) : a.N;
    if (split.y < split.x) return;        // one run, or nothing: written
    const int64_t part = (int64_t)rows_of_block * (D + 2), next = (int64_t)a.H * a.row_blocks * 2 * part;
    const float* at = a.parts + ((int64_t)split.x * a.H + h) * a.row_blocks * 2 * part + rb * 2 * part;
    const int parts = split.y - split.x + 1;
    const int ml = rows_of_block * D + 2 * in_block, o = in_block * D + d;
    float top = -__builtin_inff(), sum = 0.0f;
    f32x4_t v = {0, 0, 0, 0};
    // adds a partial sum with its maximum; a part that saw nothing has the sum 0 (one
    // that saw nothing but NaN has the maximum -inf too, but the sum NaN)
    auto add = [&](float m, float l, f32x4_t w) {
        if (l == 0.0f) return;
        const float t = __builtin_fmaxf(top, m);
        const float f = __builtin_amdgcn_exp2f(top - t), g = __builtin_amdgcn_exp2f(m - t);
        top = t;
        sum = sum * f + l * g;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = v[i] * f + w[i] * g;
    };
    for (int u0 = side; u0 < parts; u0 += 4 * SIDE) {
        f32x2_t x[4];
        f32x4_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // part u: the second place of the first run, then the first places
            const int u = min(u0 + k * SIDE, parts - 1);
            const float* from = at + u * next + (u == 0 ? part : 0);
            x[k] = *reinterpret_cast<const f32x2_t*>(from + ml);
            w[k] = *reinterpret_cast<const f32x4_t*>(from + o);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (u0 + k * SIDE < parts) add(x[k].x, x[k].y, w[k]);
    }
    if constexpr (SIDE > 1) {
        sm_v[threadIdx.x] = v;
        sm_ml[threadIdx.x][0] = top;
        sm_ml[threadIdx.x][1] = sum;
        __syncthreads();
        if (side > 0) return;
        for (int k = 1; k < SIDE; ++k) {
            const int from = threadIdx.x + k * TPR;
            add(sm_ml[from][0], sm_ml[from][1], sm_v[from]);
        }
    }
    const bool none = r >= n * a.G || sum == 0.0f;
    const float inv = none ? 0.0f : (1 << kSpare) / sum;
    const int64_t to = ((int64_t)b * a.N + r / a.G) * a.H * a.G + h * a.G + r % a.G;
    u32x2_t w = {0, 0};
    if (!none) w = u32x2_t{f32x2_to_bf16x2(v.x * inv, v.y * inv), f32x2_to_bf16x2(v.z * inv, v.w * inv)};
    *reinterpret_cast<u32x2_t*>(a.o + to * D + d) = w;
    if (d == 0) a.lse[to] = none ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Launches the join; few rows have many parts each: a workgroup a row, else a thread for each four values.
template <int D>
hipError_t launch_join(const AttnArgs& a, int rows_of_block, hipStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.H * a.N * a.G, per = 256 / (D / 4);
    if (rows <= 4096) {
        hipLaunchKernelGGL((tree_attn_join_kernel<D, 1024 / D>), dim3((unsigned)rows), dim3(256), 0, stream, a, rows_of_block,
                           (int64_t)0);
        return hipGetLastError();
    }
    // a grid has fewer than 2^32 threads: rows beyond 2^31 threads' take further launches
    const int64_t piece = (1ll << 31) / 256 * per;
    for (int64_t row = 0; row < rows; row += piece) {
        const int64_t n = std::min(piece, rows - row);
        hipLaunchKernelGGL((tree_attn_join_kernel<D, 1>), dim3((unsigned)((n + per - 1) / per)), dim3(256), 0, stream, a,
                           rows_of_block, row);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// What a call of these sizes launches.
struct Shape {
    int row_tiles, row_blocks, runs, waves;
    bool whole;

    int rows() const { return 16 * row_tiles; }
};

// The workspace: a split request's runs, then the parts.
int64_t split_bytes(int64_t B, int64_t H, const Shape& s) { return (B * H * s.row_blocks * 8 + 15) / 16 * 16; }

int64_t shape_workspace_bytes(int64_t B, int64_t H, int64_t D, const Shape& s) {
    if (s.whole || s.runs == 1) return 0;      // no request is split
    return split_bytes(B, H, s) + 2ll * s.runs * H * s.row_blocks * s.rows() * (D + 2) * 4;
}

// The arguments that do not depend on the cache's format.
AttnArgs args_of(const TreeAttnProblem& p, const Shape& s) {
    AttnArgs a;
    a.q = p.q; a.q_stride = p.q_stride;
    a.table = p.page_table; a.ctx = p.context_lens; a.tree = p.tree_lens; a.mask = p.tree_mask;
    a.o = p.o; a.lse = p.lse; a.scale = p.scale;
    a.B = (int)p.B; a.N = (int)p.N; a.H = (int)p.cache.H; a.G = (int)(p.Hq / p.cache.H);
    a.num_pages = (int)p.cache.num_pages; a.max_pages = (int)p.max_pages;
    a.page_shift = __builtin_ctzll((unsigned long long)p.cache.page_size);
    a.mask_words = (int)((p.N + 63) / 64);
    a.runs = s.runs; a.row_blocks = s.row_blocks; a.whole = s.whole;
    a.kc = p.cache.k_codes; a.ks = p.cache.k_sf; a.vc = p.cache.v_codes; a.vs = p.cache.v_sf;
    a.split = static_cast<int2*>(p.workspace);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + split_bytes(p.B, p.cache.H, s));
    return a;
}

}  // namespace
}  // namespace dg
