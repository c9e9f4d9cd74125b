// Attention for a tree of drafted tokens over the FP8 cache, gfx950.
//
// Token i of request b (N at most, tree_lens[b] of them) sees the request's
// context, positions [0, c), and of its own tree the tokens j whose bit its
// mask has, at positions c + j.  With one token this is decode attention.
//   S_j = scale * ks_j * (q . kc_j)      kc, vc e4m3 codes, ks, vs their scales
//   o   = sum_j p_j vs_j vc_j,  p = softmax(S),  lse = ln sum_j exp S_j
// A row that sees nothing has o = 0 and lse = -inf.
//
// The rows of one key head are its n tokens times the G query heads that share
// it (row = token * G + head), so a key or value is fetched once for all.
//
// Bound: a few rows per key head leave the cache's bytes as the floor, so the
// cache goes from HBM straight to registers, no LDS and no barrier on the way:
// a wave takes 32 keys a step, holds its own running maximum and sum, fetches
// the next step's keys as soon as this step's are in the product and its
// values after the second product.
//  * S^T = K q^T by 16x16x32 bf16 MFMA (e4m3 and the query are exact in bf16):
//    lane l converts the 16-byte pieces of key l & 15 that it loaded itself;
//    the query has the same order of D in its fragments.
//  * S^T leaves lane l with keys 4 (l >> 4) + i of both 16-key tiles for row
//    l & 15, which is the operand layout of O^T = V^T P^T when the 32 keys are
//    summed in that order: P never leaves its lane.  V's operand needs 8 keys
//    of one D value in a lane; a lane loads D / 16 consecutive values of those
//    8 keys and exchanges halves of words in registers (v_perm), so the cache
//    keeps its row order.
//  * P is rounded to bf16 for the second product with the value's scale in it
//    (one rounding, relative 2^-9, of terms whose sum is rounded to bf16 at
//    the end); maximum, sum and O are fp32.
// The keys are split over workgroups where (request, key head) pairs are few;
// partial O, maximum and sum meet in the workspace and a second kernel joins
// them in the order of the splits.
#include "fp8_values.h"
#include "serve_internal.h"

#include <algorithm>

namespace dg {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;                 // keys a wave's step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    const uint8_t* kc;
    const float* ks;
    const uint8_t* vc;
    const float* vs;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* tree;
    const uint64_t* mask;
    uint16_t* o;
    float* lse;
    float* part_o;                        // [B, H, N * G, splits, D]
    float* part_ml;                       // [B, H, N * G, splits, 2]
    float scale;
    int B, N, H, G, num_pages, page_shift, max_pages, splits, mask_words;
};

template <int D>
struct VWord;
template <>
struct VWord<64> { typedef uint32_t type __attribute__((ext_vector_type(1))); };
template <>
struct VWord<128> { typedef u32x2_t type; };
template <>
struct VWord<256> { typedef u32x4_t type; };

// One step's share of the cache in a lane.
template <int D>
struct Keys {
    u32x4_t k[2][D / 64];
    typename VWord<D>::type v[2][4];
    f32x4_t ks[2], vs[2];
};

// Where a step's two 16-key tiles lie (rows of the pool), uniform.
struct Place {
    int64_t row[2];
    bool live[2];                         // the tile has keys and a valid page
};

__device__ __forceinline__ int request_len(const AttnArgs& a, int b, int& ctx, int& n) {
    const int most = a.max_pages << a.page_shift;
    ctx = min(max(a.ctx[b], 0), most);
    n = a.tree ? min(max(a.tree[b], 0), a.N) : a.N;
    return min((int64_t)ctx + n, (int64_t)most);
}

template <int D, int RT>
__global__ __launch_bounds__(kWaves * 64, 2) void tree_attn_kernel(AttnArgs a) {
    constexpr int DT = D / 16;            // 16-row tiles of O^T
    constexpr int ROWS = 16 * RT;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.x % a.splits, bh = blockIdx.x / a.splits;
    const int b = bh / a.H, h = bh - b * a.H;
    const int row0 = blockIdx.y * ROWS;
    const int all_rows = a.N * a.G, Hq = a.H * a.G;
    int ctx, n;
    const int L = request_len(a, b, ctx, n);
    const int rows = n * a.G;
    const bool whole = a.splits == 1;

    if (row0 >= rows) {                   // nothing but rows past the tree's end
        if (whole) {
            for (int i = threadIdx.x; i < ROWS * D; i += blockDim.x) {
                const int r = row0 + i / D;
                if (r < all_rows)
                    a.o[((int64_t)(b * (int64_t)a.N + r / a.G) * Hq + h * a.G + r % a.G) * D + i % D] = 0;
            }
            for (int r = row0 + threadIdx.x; r < min(row0 + ROWS, all_rows); r += blockDim.x)
                a.lse[(int64_t)(b * (int64_t)a.N + r / a.G) * Hq + h * a.G + r % a.G] = -__builtin_inff();
        }
        return;
    }

    // this workgroup's steps, dealt to its waves in turn
    const int steps = (L + kStep - 1) / kStep;
    const int chunk = (steps + a.splits - 1) / a.splits;
    const int s_end = min(steps, (split + 1) * chunk);
    int s = split * chunk + wave;

    // the lane's query row of each row tile, its D values in the keys' order
    bf16x8_t qf[RT][D / 32];
    int tok[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = row0 + 16 * t + r16;
        tok[t] = r / a.G;
        const int hq = h * a.G + r - tok[t] * a.G;
        const uint16_t* src = a.q + (int64_t)(b * (int64_t)a.N + tok[t]) * a.q_stride + (int64_t)hq * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            u32x4_t w = {0, 0, 0, 0};
            if (r < rows) w = *reinterpret_cast<const u32x4_t*>(src + (c / 2) * 64 + g * 16 + (c % 2) * 8);
            qf[t][c] = __builtin_bit_cast(bf16x8_t, w);
        }
        tok[t] = min(tok[t], a.N - 1);
    }

    const int32_t* table = a.table + (int64_t)b * a.max_pages;
    auto place = [&](int step) {
        Place w;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int j0 = step * kStep + 16 * t;
            w.row[t] = 0;
            w.live[t] = j0 < L;
            if (w.live[t]) {
                const int page = table[j0 >> a.page_shift];
                w.live[t] = page >= 0 && page < a.num_pages;
                if (w.live[t])
                    w.row[t] = (((int64_t)page * a.H + h) << a.page_shift) + (j0 & ((1 << a.page_shift) - 1));
            }
        }
        return w;
    };
    Keys<D> x;
    auto fetch_k = [&](const Place& w) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* kp = a.kc + (w.row[t] + r16) * D + g * 16;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) x.k[t][c] = *reinterpret_cast<const u32x4_t*>(kp + 64 * c);
            x.ks[t] = *reinterpret_cast<const f32x4_t*>(a.ks + w.row[t] + 4 * g);
        }
    };
    auto fetch_v = [&](const Place& w) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* vp = a.vc + (w.row[t] + 4 * g) * D + r16 * DT;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x.v[t][i] = *reinterpret_cast<const typename VWord<D>::type*>(vp + i * D);
            x.vs[t] = *reinterpret_cast<const f32x4_t*>(a.vs + w.row[t] + 4 * g);
        }
    };

    f32x4_t acc[RT][DT];
    float m[RT], l[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = -__builtin_inff();
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[t][i] = f32x4_t{0, 0, 0, 0};
    }
    const float c2 = a.scale * kLog2e;

    Place at{}, next{};
    if (s < s_end) {
        at = place(s);
        fetch_k(at);
        fetch_v(at);
    }
    for (; s < s_end; s += kWaves) {
        const int j0 = s * kStep;
        const bool more = s + kWaves < s_end;
        if (more) next = place(s + kWaves);
        const bool all = j0 + kStep <= ctx && at.live[0] && at.live[1];   // uniform: no mask here
        f32x4_t sc[RT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bf16x8_t kf[D / 32];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                kf[2 * c] = e4m3x8_to_bf16x8(x.k[u][c].x, x.k[u][c].y);
                kf[2 * c + 1] = e4m3x8_to_bf16x8(x.k[u][c].z, x.k[u][c].w);
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                f32x4_t p = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < D / 32; ++c) p = mfma_bf16(kf[c], qf[t][c], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[t][u][i] = p[i] * (x.ks[u][i] * c2);
            }
        }
        if (more) fetch_k(next);
        if (!all) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + 16 * u + 4 * g + i;      // position
                    const int d = j - ctx;                      // number in the tree
                    const bool there = at.live[u] && j < L;
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        bool seen = there;
                        if (there && d >= 0)
                            seen = a.mask ? (a.mask[((int64_t)b * a.N + tok[t]) * a.mask_words + (d >> 6)] >> (d & 63)) & 1
                                          : d <= tok[t];
                        if (!seen) sc[t][u][i] = -__builtin_inff();
                    }
                    // values past the end may hold anything: 0 * NaN must not reach O
                    if (!there) x.v[u][i] = typename VWord<D>::type(0);
                }
        }
        bf16x8_t pf[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float mx = m[t];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) mx = __builtin_fmaxf(mx, sc[t][u][i]);
            mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16));
            mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
            const float base = mx == -__builtin_inff() ? 0.0f : mx;   // nothing seen yet: exp2 stays 0
            if (__any(mx != m[t])) {
                const float f = __builtin_amdgcn_exp2f(m[t] - base);
                l[t] *= f;
#pragma unroll
                for (int i = 0; i < DT; ++i) acc[t][i] *= f;
                m[t] = mx;
            }
            u32x4_t w;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(sc[t][u][i] - base);
                    l[t] += e;
                    p[i] = e * x.vs[u][i];
                    if (!all) p[i] = sc[t][u][i] == -__builtin_inff() ? 0.0f : p[i];   // scales of unseen keys
                }
                w[2 * u] = f32x2_to_bf16x2(p[0], p[1]);
                w[2 * u + 1] = f32x2_to_bf16x2(p[2], p[3]);
            }
            pf[t] = __builtin_bit_cast(bf16x8_t, w);
        }
        // V^T: tile i takes D value r16 * DT + i of the lane's 8 keys
#pragma unroll
        for (int w = 0; w < DT / 4; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                u32x4_t even, odd;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t ka = x.v[u][2 * i][w], kb = x.v[u][2 * i + 1][w];
                        const uint32_t va = half ? e4m3x2_to_bf16x2<true>(ka) : e4m3x2_to_bf16x2<false>(ka);
                        const uint32_t vb = half ? e4m3x2_to_bf16x2<true>(kb) : e4m3x2_to_bf16x2<false>(kb);
                        even[2 * u + i] = __builtin_amdgcn_perm(vb, va, 0x05040100u);
                        odd[2 * u + i] = __builtin_amdgcn_perm(vb, va, 0x07060302u);
                    }
                const int i = 4 * w + 2 * half;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    acc[t][i] = mfma_bf16(__builtin_bit_cast(bf16x8_t, even), pf[t], acc[t][i]);
                    acc[t][i + 1] = mfma_bf16(__builtin_bit_cast(bf16x8_t, odd), pf[t], acc[t][i + 1]);
                }
            }
        if (more) fetch_v(next);
        at = next;
    }

    // join the waves
    constexpr int PITCH = D + 4;
    __shared__ __attribute__((aligned(16))) float sm_o[ROWS * PITCH];
    __shared__ float sm_m[kWaves][ROWS], sm_l[kWaves][ROWS];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        if (g == 0) {
            sm_m[wave][16 * t + r16] = m[t];
            sm_l[wave][16 * t + r16] = l[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        float top = sm_m[0][16 * t + r16];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][16 * t + r16]);
        const float f = m[t] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[t] - top);
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[t][i] *= f;
    }
#pragma unroll 1
    for (int w = 0; w < kWaves; ++w) {
        if (wave == w) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < DT / 4; ++c) {
                        float* at = sm_o + (16 * t + r16) * PITCH + (4 * g + i) * DT + 4 * c;
                        f32x4_t v = {acc[t][4 * c][i], acc[t][4 * c + 1][i], acc[t][4 * c + 2][i],
                                     acc[t][4 * c + 3][i]};
                        if (w > 0) v += *reinterpret_cast<const f32x4_t*>(at);
                        *reinterpret_cast<f32x4_t*>(at) = v;
                    }
        }
        __syncthreads();
    }
    // each thread takes 4 values of a row at a time
    for (int i = threadIdx.x; i < ROWS * D / 4; i += kWaves * 64) {
        const int rr = i / (D / 4), d = (i % (D / 4)) * 4, r = row0 + rr;
        if (r >= all_rows) continue;
        float top = sm_m[0][rr], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][rr]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (sm_m[w][rr] != -__builtin_inff()) sum += sm_l[w][rr] * __builtin_amdgcn_exp2f(sm_m[w][rr] - top);
        f32x4_t v = *reinterpret_cast<const f32x4_t*>(sm_o + rr * PITCH + d);
        if (whole) {
            const bool none = r >= rows || top == -__builtin_inff();
            const float inv = none ? 0.0f : 1.0f / sum;
            const int64_t at = (int64_t)(b * (int64_t)a.N + r / a.G) * Hq + h * a.G + r % a.G;
            u32x2_t w = {0, 0};
            if (!none) w = u32x2_t{f32x2_to_bf16x2(v.x * inv, v.y * inv), f32x2_to_bf16x2(v.z * inv, v.w * inv)};
            *reinterpret_cast<u32x2_t*>(a.o + at * D + d) = w;
            if (d == 0) a.lse[at] = none ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
        } else if (r < rows) {
            const int64_t at = ((int64_t)bh * all_rows + r) * a.splits + split;
            *reinterpret_cast<f32x4_t*>(a.part_o + at * D + d) = v;
            if (d == 0) {
                a.part_ml[2 * at] = top;
                a.part_ml[2 * at + 1] = sum;
            }
        }
    }
}

// Joins the splits of a row: D / 4 threads a row, splits in order.
template <int D>
__global__ __launch_bounds__(256) void tree_attn_join_kernel(AttnArgs a) {
    constexpr int TPR = D / 4;
    const int64_t all_rows = (int64_t)a.N * a.G;
    const int64_t id = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;   // (b, h, row)
    const int d = threadIdx.x % TPR * 4;
    if (id >= (int64_t)a.B * a.H * all_rows) return;
    const int bh = (int)(id / all_rows), r = (int)(id - bh * all_rows);
    const int b = bh / a.H, h = bh - b * a.H;
    int ctx, n;
    request_len(a, b, ctx, n);
    const float* ml = a.part_ml + 2 * id * a.splits;
    const bool row = r < n * a.G;
    float top = -__builtin_inff();
    if (row)
        for (int s = 0; s < a.splits; ++s) top = __builtin_fmaxf(top, ml[2 * s]);
    const bool none = top == -__builtin_inff();
    float sum = 0.0f;
    f32x4_t v = {0, 0, 0, 0};
    if (!none)
        for (int s = 0; s < a.splits; ++s) {
            if (ml[2 * s] == -__builtin_inff()) continue;       // saw nothing
            const float f = __builtin_amdgcn_exp2f(ml[2 * s] - top);
            sum += ml[2 * s + 1] * f;
            v += *reinterpret_cast<const f32x4_t*>(a.part_o + (id * a.splits + s) * D + d) * f;
        }
    const float inv = none ? 0.0f : 1.0f / sum;
    const int64_t at = ((int64_t)b * a.N + r / a.G) * a.H * a.G + h * a.G + r % a.G;
    u32x2_t w = {0, 0};
    if (!none) w = u32x2_t{f32x2_to_bf16x2(v.x * inv, v.y * inv), f32x2_to_bf16x2(v.z * inv, v.w * inv)};
    *reinterpret_cast<u32x2_t*>(a.o + at * D + d) = w;
    if (d == 0) a.lse[at] = none ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Row tiles a wave holds: up to 256 O values a lane's registers can keep.
int row_tiles(int64_t N, int64_t G, int64_t D) {
    const int64_t rows = N * G;
    const int t = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    return std::min<int64_t>(t, 256 / D);
}

// Splits of the keys: enough workgroups for two a CU of 256, none of fewer
// than four steps a wave.  From the sizes alone, so that a size has one order
// of sums; the lengths themselves are on the device.
int64_t split_count(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D, int64_t max_pages,
                    int64_t page_size) {
    const int64_t G = Hq / H, block = 16 * row_tiles(N, G, D);
    const int64_t groups = B * H * ((N * G + block - 1) / block);
    const int64_t steps = (max_pages * page_size + kStep - 1) / kStep;
    return std::max<int64_t>(1, std::min((512 + groups - 1) / groups, steps / (4 * kWaves)));
}

template <int D>
hipError_t launch(const AttnArgs& a, int rt, hipStream_t stream) {
    const int all_rows = a.N * a.G;
    const dim3 grid((unsigned)(a.B * a.H * a.splits), (unsigned)((all_rows + 16 * rt - 1) / (16 * rt)));
    const dim3 block(kWaves * 64);
    if constexpr (D == 64)
        if (rt == 4) hipLaunchKernelGGL((tree_attn_kernel<D, 4>), grid, block, 0, stream, a);
    if constexpr (D <= 128)
        if (rt == 2) hipLaunchKernelGGL((tree_attn_kernel<D, 2>), grid, block, 0, stream, a);
    if (rt == 1) hipLaunchKernelGGL((tree_attn_kernel<D, 1>), grid, block, 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = (int64_t)a.B * a.H * all_rows, per = 256 / (D / 4);
    hipLaunchKernelGGL((tree_attn_join_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0,
                       stream, a);
    return hipGetLastError();
}

}  // namespace

int64_t tree_attn_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D,
                                  int64_t max_pages, int64_t page_size) {
    const int64_t splits = split_count(B, N, Hq, H, D, max_pages, page_size);
    return splits == 1 ? 0 : B * N * Hq * splits * (D + 2) * 4;
}

hipError_t launch_tree_attn(const TreeAttnProblem& p, hipStream_t stream) {
    AttnArgs a;
    a.q = p.q; a.q_stride = p.q_stride;
    a.kc = p.cache.k_codes; a.ks = p.cache.k_sf; a.vc = p.cache.v_codes; a.vs = p.cache.v_sf;
    a.table = p.page_table; a.ctx = p.context_lens; a.tree = p.tree_lens; a.mask = p.tree_mask;
    a.o = p.o; a.lse = p.lse; a.scale = p.scale;
    a.B = (int)p.B; a.N = (int)p.N; a.H = (int)p.cache.H; a.G = (int)(p.Hq / p.cache.H);
    a.num_pages = (int)p.cache.num_pages; a.max_pages = (int)p.max_pages;
    a.page_shift = __builtin_ctzll((unsigned long long)p.cache.page_size);
    a.mask_words = (int)((p.N + 63) / 64);
    a.splits = (int)split_count(p.B, p.N, p.Hq, p.cache.H, p.cache.D, p.max_pages, p.cache.page_size);
    a.part_o = static_cast<float*>(p.workspace);
    a.part_ml = a.part_o + p.B * p.N * p.Hq * a.splits * p.cache.D;
    const int rt = row_tiles(p.N, a.G, p.cache.D);
    switch (p.cache.D) {
    case 64: return launch<64>(a, rt, stream);
    case 128: return launch<128>(a, rt, stream);
    case 256: return launch<256>(a, rt, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dg
