// Attention for a tree of drafted tokens over the FP8 cache, gfx950.
//
// Token i of request b (N at most, tree_lens[b] of them) sees the request's
// context, positions [0, c), and of its own tree the tokens j whose bit its
// mask has, at positions c + j.  With one token this is decode attention.
//   S_j = scale * ks_j * (q . kc_j)      kc, vc e4m3 codes, ks, vs their scales
//   o   = sum_j p_j vs_j vc_j,  p = softmax(S),  lse = ln sum_j exp S_j
// A row that sees nothing has o = 0 and lse = -inf: its sum is 0, where what is seen
// leaves 1 or more, or NaN.  (The maximum does not tell: it passes over NaN.)
//
// The rows of one key head are its n tokens times the G query heads that share
// it (row = token * G + head), so a key or value is fetched once for all.
//
// Bound: a few rows per key head leave the cache's bytes as the floor, so the
// cache goes from HBM straight to registers, no LDS and no barrier on the way:
// a wave takes 32 keys a step, holds its own running maximum and sum, and asks
// for the next step's keys and values while it computes.
//  * S^T = K q^T by 16x16x32 bf16 MFMA (e4m3 and the query are exact in bf16):
//    lane l converts the 16-byte pieces of key l & 15 that it loaded itself; the
//    query has the same order of D in its fragments.
//  * S^T leaves lane l with keys 4 (l >> 4) + i of both 16-key tiles for row
//    l & 15, which is the operand layout of O^T = V^T P^T when the 32 keys are
//    summed in that order: P never leaves its lane.  V's operand needs 8 keys
//    of one D value in a lane; a lane loads D / 16 consecutive values of those
//    8 keys and exchanges halves of words in registers (v_perm), so the cache
//    keeps its row order.
//  * P, times the values' scales, is rounded to fp16 for the second product (e4m3
//    is exact in fp16 too): 11 bits, against bf16's 8, keep its rounding below
//    the output's.  fp16 has few exponents, so P vs 2^(11 - x) is what is
//    rounded, x the exponent of the largest scale that the row has seen in its wave:
//    terms down to 2^-35 of the largest possible one count.  Maximum, sum and O are
//    fp32.
//  * Scores are checked against the running maximum in their own lanes, and the
//    maximum follows, with the exchange and the scaling of O that this takes, only
//    where one passes it by 2^4 or more: in nearly every step it does not.  P's
//    range leaves those 4 powers of two free.
// A workgroup has 16 or 32 rows, and its waves share their steps and add up in
// LDS.  More rows than that are further workgroups beside it, which find the
// keys in the XCD's cache: all of 128 rows' waves in one workgroup, each with 32
// of them and all steps, leave less to join within it but four times the parts
// to join through memory (one request of 40 tokens over 20000: 55 us against 40).
// With many rows the VALU (widening keys and values, exponentials) is the bound.
//
// Short requests have a workgroup each, for a key head and a row block, as the
// table's size or, in a long table, their lengths tell.  Long ones differ in
// length, so the steps of all of them, end to end, are cut into equal runs, and the
// workgroup of a run goes through the requests that it touches.  Where a run ends
// inside a request, its O, maximum and sum go to the workspace, and a second kernel
// joins a request's parts in order, a thread for four values of a row.
// (Joined by the last workgroup to arrive instead, a long request's
// parts pass through one CU: 344 us against 174 for two trees of 16 over 100001
// tokens, both as they were then.)
// Measured (a batch "of n over c" goes from n tokens and c positions down to half of
// them): 32 single tokens over 8192, 32 / 8 heads of 128, 417 MB, 90 us, 4.6 TB/s;
// two trees of 16 over 100001, 64 / 8 heads of 128, 317 MB and 66 GFLOP, 141 us,
// 2.2 TB/s and 0.46 PFLOP/s with the VALU 47% and the matrix unit 20% busy; 7 trees
// of 24 over 3001, the last of them idle, 21 us.
#include "fp8_values.h"
#include "serve_internal.h"

#include <algorithm>
#include <type_traits>

namespace dg {
namespace {

constexpr int kWaves = 4;                 // of a workgroup where requests are split
constexpr int kStep = 32;                 // keys of a wave's step
// Several requests that turn out to be short, though their table is long, stay
// whole and are dealt to the runs in turn: where none has more than kBrief steps,
// or kFew and there are as many requests as runs.  Borders between requests in a
// run, and parts to join, cost more than equal runs gain (64 requests of 20 to 700
// tokens: 16.5 us against 25.8; 7 trees of 24 over 500 to 760, 12.7 against 18.6;
// 128 of 500 to 2000, 70 against 79; alone, 760: 11.3 against 10.0).
constexpr int kBrief = 24, kFew = 64;
constexpr int kTop = 11;                  // P of a value with the largest scale is below 2^(kTop + kLazy)
constexpr float kLazy = 4.0f;             // how far, in powers of two, scores pass m before m follows
// O is put down 2^kSpare too small: waves and parts, 8 x 768 at most, each with a sum
// below 1, then add up without passing fp32's largest number, whatever the values.
constexpr int kSpare = 13;
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
    int2* split;                          // [B, H, row blocks]: first and last run of a request; last < first: one
    float* parts;                         // [runs * H, row blocks, 2]: O [ROWS, D], then maxima and sums [ROWS, 2]
    float scale;
    int B, N, H, G, num_pages, page_shift, max_pages, mask_words;
    int runs, row_blocks;
    bool whole;                           // a run is a request
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
    float ks[2], vs[2];                   // of keys 4 g + lane % 4 of each tile
};

// Where a step's two 16-key tiles lie (rows of the pool), uniform.
struct Place {
    int64_t row[2];
    bool live[2];                         // the tile has keys and a valid page
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

// RT: row tiles, of each of a workgroup's W waves the same.
template <int D, int RT, int W>
__global__ __launch_bounds__(W * 64, D == 256 ? 1 : D == 128 || W == 8 ? 2 : 3) void tree_attn_kernel(AttnArgs a) {
    constexpr int DT = D / 16;            // 16-row tiles of O^T
    constexpr int ROWS = 16 * RT;
    constexpr int PITCH = D + 4;          // of a row of O in LDS
    constexpr int PART = ROWS * (D + 2);  // floats of a part
    __shared__ __attribute__((aligned(16))) float sm_o[W][ROWS * PITCH];
    __shared__ f32x2_t sm_ml[W][ROWS];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The row blocks of a run follow one another on one XCD (workgroups go to the
    // eight in turn), whose cache then has their keys.
    const int in_xcd = blockIdx.x >> 3, rb = in_xcd % a.row_blocks;
    const int run_head = (in_xcd / a.row_blocks) * 8 + (blockIdx.x & 7);
    if (run_head >= a.runs * a.H) return;
    const int run = run_head / a.H, h = run_head - run * a.H;
    const int row0 = rb * ROWS;
    const int all_rows = a.N * a.G, Hq = a.H * a.G;

    int b = run, stride = 1, end = a.B;
    int64_t s0 = 0, s1 = 1ll << 62, start = 0, total = 0, runs = 1;     // start: of request b
    if (a.whole) {
        end = run + 1;
    } else {
        // this run's steps of all requests', and the request that they start in
        uint32_t upto = 0;                // of the lane's request and those before it of its 64, 2^31 at most
        bool brief = a.B > 1, few = a.B >= a.runs;
        for (int base = 0; base < a.B; base += 64) {
            const int own = steps_of_lane(a, base + lane, row0);
            brief = brief && !__any(own > kBrief);
            few = few && !__any(own > kFew);
            upto = sum_up_to_lane(own);
            total += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
        }
        if (brief || few) {
            stride = a.runs;
        } else {
            runs = max((int64_t)1, min((int64_t)a.runs, total / W));
            if (run >= runs) return;
            s0 = total * run / runs;
            s1 = total * (run + 1) / runs;
            b = a.B;
            for (int base = 0; base < a.B; base += 64) {
                if (a.B > 64) upto = sum_up_to_lane(steps_of_lane(a, base + lane, row0));
                const uint32_t before = __shfl_up(upto, 1);
                const int64_t from = start + (lane > 0 ? before : 0u);
                const uint64_t hit = __ballot(base + lane < a.B && (start + upto > s0 || from >= s0));
                if (hit != 0) {
                    const int at = __builtin_ctzll(hit);
                    b = base + at;
                    if (at > 0) start += (uint32_t)__builtin_amdgcn_readlane(upto, at - 1);
                    break;
                }
                start += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
            }
        }
    }

    for (; b < end && (start < s1 || (run == runs - 1 && start == total)); b += stride) {
    const Request rq = request(a, b, row0);
    const int ctx = rq.ctx, rows = rq.n * a.G;
    // a token alone that does not see itself is as good as past the end
    const bool blind = a.N == 1 && a.mask && !(uniform_input(reinterpret_cast<const int32_t*>(a.mask + b)) & 1);
    const int L = blind ? min(ctx, rq.L) : rq.L;
    const int lo = (int)max(s0 - start, (int64_t)0), hi = (int)min(s1 - start, (int64_t)rq.steps);
    start += rq.steps;
    auto out_row = [&](int r) { return ((int64_t)b * a.N + r / a.G) * Hq + h * a.G + r % a.G; };
    const bool whole = lo == 0 && hi == rq.steps;
    if (lo == 0 && threadIdx.x == 0 && !a.whole && a.runs > 1) {
        // the last run that starts at or before the request's last step
        const int64_t last = whole ? run - 1 : (start * runs + total - 1) / total - 1;
        a.split[((int64_t)b * a.H + h) * a.row_blocks + rb] = make_int2(run, (int)last);
    }
    if (rq.steps == 0) {                  // no row of the block sees anything
        for (int i = threadIdx.x; i < ROWS * D / 8; i += W * 64) {
            const int r = row0 + i / (D / 8);
            if (r >= all_rows) break;
            const int64_t at = out_row(r);
            *reinterpret_cast<u32x4_t*>(a.o + at * D + i % (D / 8) * 8) = u32x4_t{0, 0, 0, 0};
            if (i % (D / 8) == 0) a.lse[at] = -__builtin_inff();
        }
        continue;
    }

    const int qlane = fresh(lane), qr16 = qlane & 15, qg = qlane >> 4;
    // the lane's query row of each row tile, its D values in the keys' order
    bf16x8_t qf[RT][D / 32];
    int tok[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = row0 + 16 * t + qr16;
        tok[t] = r / a.G;
        const int hq = h * a.G + r - tok[t] * a.G;
        const uint16_t* src = a.q + ((int64_t)b * a.N + tok[t]) * a.q_stride + (int64_t)hq * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            u32x4_t w = {0, 0, 0, 0};
            if (r < rows) w = *reinterpret_cast<const u32x4_t*>(src + (c / 2) * 64 + qg * 16 + (c % 2) * 8);
            qf[t][c] = __builtin_bit_cast(bf16x8_t, w);
        }
        tok[t] = min(tok[t], a.N - 1);
    }

    const int32_t* table = a.table + (int64_t)b * a.max_pages;
    // Lanes 2 n and 2 n + 1 ask for the pages of a step's two tiles: vector loads,
    // in the order of the others, two steps ahead.  (Scalar loads are waited for
    // where the page is first looked at, twice a step.)
    auto ask = [&](int step) {
        return table[min((step * kStep + 16 * (lane & 1)) >> a.page_shift, a.max_pages - 1)];
    };
    auto place = [&](int step, int pages) {
        Place w;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int j0 = step * kStep + 16 * t, page = __builtin_amdgcn_readlane(pages, t);
            w.live[t] = j0 < L && page >= 0 && page < a.num_pages;
            w.row[t] = w.live[t] ? (((int64_t)page * a.H + h) << a.page_shift) + (j0 & ((1 << a.page_shift) - 1)) : 0;
        }
        return w;
    };
    f32x4_t acc[RT][DT];                  // in units of 2^(unit + more - kTop)
    float m[RT], base[RT], l[RT];         // base: m, or 0 while nothing was seen, so that exp2 stays 0
    // The exponent of the largest value scale that a row has seen is unit + more.  Rows
    // have the same, and no more, until a masked step has one that not all of them see.
    int unit = -1000, more[RT];
    bool differ = false;
    float largest = 0.0f;                 // 2^unit
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = -__builtin_inff();
        base[t] = l[t] = 0.0f;
        more[t] = 0;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[t][i] = f32x4_t{0, 0, 0, 0};
    }
    const float c2 = a.scale * kLog2e;
    const bool apart = a.N > 1;           // rows of several tokens: they may see different keys
    // The next step's keys are asked for when this step's are in the first
    // product, its values when they are in the second.  Neither is conditional
    // (past the last step the last one again), and they stay where they are
    // written: the compiler then waits for this step's loads alone.
    if (lo + wave < hi) {
    // uniform bases, a lane's place in 32 bits
    const uint32_t k_off = r16 * D + g * 16, v_off = 4 * g * D + r16 * DT, s_off = 4 * (4 * g + (lane & 3));
    Keys<D> x;
    auto fetch_k = [&](const Place& w, int t) {
        const uint8_t* base = a.kc + w.row[t] * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) x.k[t][c] = *reinterpret_cast<const u32x4_t*>(base + 64 * c + k_off);
        x.ks[t] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.ks + w.row[t]) + s_off);
    };
    auto fetch_v = [&](const Place& w) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t* base = a.vc + w.row[t] * D;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x.v[t][i] = *reinterpret_cast<const typename VWord<D>::type*>(base + i * D + v_off);
            x.vs[t] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.vs + w.row[t]) + s_off);
        }
    };
    const int s_last = hi - 1;
    int pages = ask(min(lo + wave, s_last)), pages_next = ask(min(lo + wave + W, s_last));
    Place at = place(min(lo + wave, s_last), pages);
    pages = ask(min(lo + wave + 2 * W, s_last));
    fetch_k(at, 0);
    fetch_k(at, 1);
    __builtin_amdgcn_sched_barrier(0);
    fetch_v(at);
    __builtin_amdgcn_sched_barrier(0);
    // A query row with an infinity becomes one of NaN, which its softmax is: scores that
    // are all -infinity would look like those of hidden keys.  0 * q sums to 0 or to NaN.
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        f32x4_t zero = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) zero = mfma_bf16(bf16x8_t(0.0f), qf[t][c], zero);
        const bool finite = zero.x == 0.0f;
        if (!__all(finite)) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                if (!finite) qf[t][c] = bf16x8_t(__builtin_nanf(""));
        }
    }
    for (int s = lo + wave; s < hi; s += W) {
        const int j0 = s * kStep;
        const Place next = place(min(s + W, s_last), pages_next);
        pages_next = pages;
        pages = ask(min(s + 3 * W, s_last));
        __builtin_amdgcn_sched_barrier(0);
        const bool all = j0 + kStep <= ctx && at.live[0] && at.live[1] && !differ;   // uniform: no mask here
        float sc[RT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bf16x8_t kf[D / 32];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                kf[2 * c] = e4m3x8_to_bf16x8(x.k[u][c].x, x.k[u][c].y);
                kf[2 * c + 1] = e4m3x8_to_bf16x8(x.k[u][c].z, x.k[u][c].w);
            }
            const float own = x.ks[u] * c2;
            const float kscale[4] = {of_quad<0>(own), of_quad<1>(own), of_quad<2>(own), of_quad<3>(own)};
            __builtin_amdgcn_sched_barrier(0);
            fetch_k(next, u);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                f32x4_t p = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < D / 32; ++c) p = mfma_bf16(kf[c], qf[t][c], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[t][u][i] = p[i] * kscale[i];
            }
        }
        if (!all) {
            const int mlane = fresh(lane), g = mlane >> 4;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + 16 * u + 4 * g + i;      // position
                        const int d = j - ctx;                      // number in the tree
                        bool seen = at.live[u] && j < L;
                        if (seen && d >= 0 && apart)
                            seen = a.mask ? (a.mask[((int64_t)b * a.N + tok[t]) * a.mask_words + (d >> 6)] >> (d & 63)) & 1
                                          : d <= tok[t];
                        if (!seen) sc[t][u][i] = -__builtin_inff();
                    }
            // values past the end may hold anything: 0 * NaN must not reach O
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (!at.live[u] || j0 + 16 * u + 4 * g + (mlane & 3) >= L) x.vs[u] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!at.live[u] || j0 + 16 * u + 4 * g + i >= L) x.v[u][i] = typename VWord<D>::type(0);
            }
            // A row's scales are those of the keys that it sees: a large one that is hidden
            // from it must not take the bits of its own.
            if (apart) {
                differ = false;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    float far = 0.0f;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float v = __builtin_fabsf(x.vs[u]);
                        const float vs[4] = {of_quad<0>(v), of_quad<1>(v), of_quad<2>(v), of_quad<3>(v)};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (sc[t][u][i] != -__builtin_inff()) far = __builtin_fmaxf(far, vs[i]);
                    }
                    const float now = __builtin_amdgcn_ldexpf(1.0f, unit + more[t]);
                    if (__any(far > now)) {
                        far = max_of_groups(far);
                        const int add = far > now ? max(__builtin_amdgcn_frexp_expf(far) - unit - more[t], 0) : 0;
                        const float shrink = __builtin_amdgcn_ldexpf(1.0f, max(-add, -1000));
#pragma unroll
                        for (int i = 0; i < DT; ++i) acc[t][i] *= shrink;
                        more[t] += add;
                    }
                    differ |= __any(more[t] != __builtin_amdgcn_readfirstlane(more[0]));
                }
                if (!differ) {
                    unit += __builtin_amdgcn_readfirstlane(more[0]);
                    largest = __builtin_amdgcn_ldexpf(1.0f, unit);
#pragma unroll
                    for (int t = 0; t < RT; ++t) more[t] = 0;
                }
            }
        }
        // A wave in its softmax goes before one in its products, which the matrix unit
        // holds up anyway (1 to 2%).
        __builtin_amdgcn_s_setprio(1);
        // Whether a score or a value's scale outgrows what O is relative to.  The
        // lanes look at their own; only then is the row's maximum exchanged.
        float mx[RT];
        const float top = all || !apart ? __builtin_fmaxf(__builtin_fabsf(x.vs[0]), __builtin_fabsf(x.vs[1])) : 0.0f;
        bool over = top > largest;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            mx[t] = sc[t][0][0];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[t] = __builtin_fmaxf(mx[t], sc[t][u][i]);
            over |= mx[t] > m[t] + kLazy;
        }
        if (__any(over)) {
            float far = __builtin_fmaxf(__builtin_fmaxf(of_quad<0>(top), of_quad<1>(top)),
                                        __builtin_fmaxf(of_quad<2>(top), of_quad<3>(top)));
            far = max_of_groups(__builtin_fmaxf(far, largest));
            const int now = __builtin_amdgcn_readfirstlane(far > largest ? __builtin_amdgcn_frexp_expf(far) : unit);
            const float shrink = __builtin_amdgcn_ldexpf(1.0f, max(unit - now, -1000));
            unit = now;
            largest = __builtin_amdgcn_ldexpf(1.0f, now);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                mx[t] = __builtin_fmaxf(max_of_groups(mx[t]), m[t]);
                if (mx[t] != -__builtin_inff()) base[t] = mx[t];
                const float f = __builtin_amdgcn_exp2f(m[t] - base[t]);
                l[t] *= f;
#pragma unroll
                for (int i = 0; i < DT; ++i) acc[t][i] *= f * shrink;
                m[t] = mx[t];
            }
        }
        float vs[2][4];                   // without a mask in units of the largest so far
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float v = __builtin_amdgcn_ldexpf(x.vs[u], all ? kTop - unit : 0);
            vs[u][0] = of_quad<0>(v);
            vs[u][1] = of_quad<1>(v);
            vs[u][2] = of_quad<2>(v);
            vs[u][3] = of_quad<3>(v);
        }
        f16x8_t pf[RT];
        auto weigh = [&](auto some_hidden) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                float p[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = __builtin_amdgcn_exp2f(sc[t][u][i] - base[t]);
                        l[t] += e;
                        if (!decltype(some_hidden)::value) p[u][i] = e * vs[u][i];
                        // a hidden key's weight is 0 whatever its value's scale
                        else if (sc[t][u][i] == -__builtin_inff()) p[u][i] = 0.0f;
                        else p[u][i] = e * __builtin_amdgcn_ldexpf(vs[u][i], kTop - unit - more[t]);
                    }
                u32x4_t w;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    w[2 * u] = f32x2_to_f16x2(p[u][0], p[u][1]);
                    w[2 * u + 1] = f32x2_to_f16x2(p[u][2], p[u][3]);
                }
                pf[t] = __builtin_bit_cast(f16x8_t, w);
            }
        };
        if (all) weigh(std::false_type());
        else weigh(std::true_type());
        __builtin_amdgcn_s_setprio(0);
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
                        const uint32_t both = __builtin_amdgcn_perm(kb, ka, half ? 0x07030602u : 0x05010400u);
                        even[2 * u + i] = e4m3x2_to_f16x2<false>(both);
                        odd[2 * u + i] = e4m3x2_to_f16x2<true>(both);
                    }
                const int i = 4 * w + 2 * half;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    acc[t][i] = mfma_f16(__builtin_bit_cast(f16x8_t, even), pf[t], acc[t][i]);
                    acc[t][i + 1] = mfma_f16(__builtin_bit_cast(f16x8_t, odd), pf[t], acc[t][i + 1]);
                }
            }
        __builtin_amdgcn_sched_barrier(0);
        fetch_v(next);
        __builtin_amdgcn_sched_barrier(0);
        at = next;
    }
    }

    // The waves put down their O and meet: a thread then adds up four values of a
    // row, wave by wave, relative to the largest of their maxima.
    const int elane = fresh(lane), er16 = elane & 15, eg = elane >> 4;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] = sum_of_groups(l[t]);
        // the sum's power of two goes to the maximum
        const int k = __builtin_amdgcn_frexp_expf(l[t]), shift = unit + more[t] - kTop - k - kSpare;
        if (eg == 0) sm_ml[wave][16 * t + er16] = f32x2_t{m[t] + (float)k, __builtin_amdgcn_ldexpf(l[t], -k)};
        float* mine = sm_o[wave] + (16 * t + er16) * PITCH + 4 * eg * DT;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < DT / 4; ++c)
                *reinterpret_cast<f32x4_t*>(mine + i * DT + 4 * c) =
                    f32x4_t{__builtin_amdgcn_ldexpf(acc[t][4 * c][i], shift), __builtin_amdgcn_ldexpf(acc[t][4 * c + 1][i], shift),
                            __builtin_amdgcn_ldexpf(acc[t][4 * c + 2][i], shift),
                            __builtin_amdgcn_ldexpf(acc[t][4 * c + 3][i], shift)};
    }
    __syncthreads();
    // A run has one part of a request that goes on from the run before (the first
    // of its two places) and one of a request that begins in it (the second).
    float* part = a.parts + (((int64_t)run_head * a.row_blocks + rb) * 2 + (lo > 0 ? 0 : 1)) * PART;
    for (int i = fresh(threadIdx.x); i < ROWS * D / 4; i += W * 64) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) top = __builtin_fmaxf(top, sm_ml[w][r].x);
        f32x4_t v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const f32x2_t ml = sm_ml[w][r];
            const float f = ml.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(ml.x - top);
            sum += f * ml.y;
            v += f * *reinterpret_cast<const f32x4_t*>(sm_o[w] + r * PITCH + d);
        }
        if (!whole) {
            *reinterpret_cast<f32x4_t*>(part + r * D + d) = v;
            if (d == 0) *reinterpret_cast<f32x2_t*>(part + ROWS * D + 2 * r) = f32x2_t{top, sum};
        } else if (row0 + r < all_rows) {
            const bool none = row0 + r >= rows || sum == 0.0f;      // a sum of NaN is none of it
            const float inv = none ? 0.0f : (1 << kSpare) / sum;
            const int64_t at = out_row(row0 + r);
            u32x2_t w = {0, 0};
            if (!none) w = u32x2_t{f32x2_to_bf16x2(v.x * inv, v.y * inv), f32x2_to_bf16x2(v.z * inv, v.w * inv)};
            *reinterpret_cast<u32x2_t*>(a.o + at * D + d) = w;
            if (d == 0) a.lse[at] = none ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
        }
    }
    __syncthreads();                      // before the next request's
    }
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

// What a call of these sizes launches.
struct Shape {
    int row_tiles, row_blocks, runs, waves;
    bool whole;

    int rows() const { return 16 * row_tiles; }
};

// Rows of a workgroup: 16 where there are no more (and for D = 256, whose O fills
// the registers), else 32.
// Whole requests, a workgroup each and no second kernel, where that is soon done
// whatever the lengths turn out to be: up to 1024 positions, or up to 2048 where
// requests and heads make 128 workgroups, up to 4096 where they make 256 or have
// two row tiles.  Their waves are as many as are resident with all the others, up
// to eight for two row tiles and four else, and halved only where that leaves a wave
// 16 steps at most (with all four, up to 32 fall to a wave of one row tile) (60
// trees of 24 over 221: 45 us with one wave, 60 with four, 100 with eight; 16 of 64
// over 300: 22 with two, 28 with four, 43 with eight; 8 of 16 over 1000: 17 with
// eight, 19 with four, 27 with two).  In graphs, whole against split: 16
// requests of 60, 5.5 us against 16.4; 64 of 1000, 20.9 against 28.8; 64 of 4000,
// 76 against 87; one of 500, 8.0 against 10.1; 7 trees of 24 over 3001, 20.9
// against 24.0; but one of 2000, 17.1 against 11.3, and of 1000 with D = 256, 15.5
// against 11.9.  (One of 1000, D = 128: 11.0 against 10.6, and a launch of 2.4 us
// less for the host.)
// Runs: two workgroups a CU of 256, one for D = 256 (its registers; two that
// follow one another cost 4 to 18%); no run is shorter than one step a wave.
// Three fit for D = 64, but more runs are more parts to join and more places
// read at once: the third is taken where 32 rows compute long, 16 steps a wave
// (16 requests of 20 tokens over 8000: 56 us against 63; with 5 steps a wave, 7 of
// 24 over 3001: 25.9 against 24.4).  Runs in excess of what is resident would
// follow the others: one request of 40 tokens over 20000, D = 128, takes 40 us in
// 480 workgroups, 52 in 560.  From the sizes alone: lengths are on the device.
Shape shape_of(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D, int64_t max_pages, int64_t page_size) {
    const int64_t rows = N * (Hq / H);
    Shape s;
    s.row_tiles = rows <= 16 || D == 256 ? 1 : 2;
    s.row_blocks = (int)((rows + s.rows() - 1) / s.rows());
    const int64_t groups = H * s.row_blocks, most = (max_pages * page_size + kStep - 1) / kStep, steps = B * most;
    const int64_t workgroups = B * groups;
    s.whole = most <= (D == 256 ? 16 : 32) || (most <= (s.row_tiles == 2 ? 128 : 64) && workgroups >= 128) ||
              (most <= 128 && workgroups >= 256);
    if (workgroups > (1 << 20)) s.whole = false;       // a grid has fewer than 2^32 threads
    s.waves = kWaves;
    if (s.whole) {
        const int64_t resident = 1024 * (D == 256 ? 1 : D == 128 ? 2 : 3);
        s.waves = s.row_tiles == 2 ? 8 : 4;
        while (s.waves > 1 && workgroups * s.waves > resident && 2 * most <= 16 * s.waves) s.waves /= 2;
    }
    s.runs = (int)B;
    if (s.whole) return s;
    const bool third = D == 64 && s.row_tiles == 2 && steps * groups >= 768 * 16 * kWaves;
    const int64_t wanted = D == 256 ? 256 : third ? 768 : 512;
    s.runs = (int)std::max<int64_t>(1, std::min(wanted / groups, steps / kWaves));
    return s;
}

template <int D, int RT>
void launch_waves(const AttnArgs& a, int waves, dim3 grid, hipStream_t stream) {
    if (waves == 1) hipLaunchKernelGGL((tree_attn_kernel<D, RT, 1>), grid, dim3(64), 0, stream, a);
    else if (waves == 2) hipLaunchKernelGGL((tree_attn_kernel<D, RT, 2>), grid, dim3(128), 0, stream, a);
    else if (waves == 4) hipLaunchKernelGGL((tree_attn_kernel<D, RT, 4>), grid, dim3(256), 0, stream, a);
    else if constexpr (RT == 2) hipLaunchKernelGGL((tree_attn_kernel<D, RT, 8>), grid, dim3(512), 0, stream, a);
}

template <int D>
hipError_t launch(const AttnArgs& a, const Shape& s, hipStream_t stream) {
    const int64_t groups = ((int64_t)a.runs * a.H + 7) / 8 * 8;
    const dim3 grid((unsigned)(groups * a.row_blocks));
    if (s.row_tiles == 1) {
        launch_waves<D, 1>(a, s.waves, grid, stream);
    } else if constexpr (D <= 128) {
        launch_waves<D, 2>(a, s.waves, grid, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole || a.runs == 1) return e;
    // few rows have many parts each: a workgroup a row, else a thread for each four values
    const int64_t rows = (int64_t)a.B * a.H * a.N * a.G, per = 256 / (D / 4);
    if (rows <= 4096) {
        hipLaunchKernelGGL((tree_attn_join_kernel<D, 1024 / D>), dim3((unsigned)rows), dim3(256), 0, stream, a, s.rows(),
                           (int64_t)0);
        return hipGetLastError();
    }
    // a grid has fewer than 2^32 threads: rows beyond 2^31 threads' take further launches
    const int64_t piece = (1ll << 31) / 256 * per;
    for (int64_t row = 0; row < rows; row += piece) {
        const int64_t n = std::min(piece, rows - row);
        hipLaunchKernelGGL((tree_attn_join_kernel<D, 1>), dim3((unsigned)((n + per - 1) / per)), dim3(256), 0, stream, a,
                           s.rows(), row);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t split_bytes(int64_t B, int64_t H, const Shape& s) { return (B * H * s.row_blocks * 8 + 15) / 16 * 16; }

}  // namespace

int64_t tree_attn_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D,
                                  int64_t max_pages, int64_t page_size) {
    const Shape s = shape_of(B, N, Hq, H, D, max_pages, page_size);
    if (s.whole || s.runs == 1) return 0;      // no request is split
    return split_bytes(B, H, s) + 2ll * s.runs * H * s.row_blocks * s.rows() * (D + 2) * 4;
}

hipError_t launch_tree_attn(const TreeAttnProblem& p, hipStream_t stream) {
    const Shape s = shape_of(p.B, p.N, p.Hq, p.cache.H, p.cache.D, p.max_pages, p.cache.page_size);
    AttnArgs a;
    a.q = p.q; a.q_stride = p.q_stride;
    a.kc = p.cache.k_codes; a.ks = p.cache.k_sf; a.vc = p.cache.v_codes; a.vs = p.cache.v_sf;
    a.table = p.page_table; a.ctx = p.context_lens; a.tree = p.tree_lens; a.mask = p.tree_mask;
    a.o = p.o; a.lse = p.lse; a.scale = p.scale;
    a.B = (int)p.B; a.N = (int)p.N; a.H = (int)p.cache.H; a.G = (int)(p.Hq / p.cache.H);
    a.num_pages = (int)p.cache.num_pages; a.max_pages = (int)p.max_pages;
    a.page_shift = __builtin_ctzll((unsigned long long)p.cache.page_size);
    a.mask_words = (int)((p.N + 63) / 64);
    a.runs = s.runs; a.row_blocks = s.row_blocks; a.whole = s.whole;
    a.split = static_cast<int2*>(p.workspace);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + split_bytes(p.B, p.cache.H, s));
    switch (p.cache.D) {
    case 64: return launch<64>(a, s, stream);
    case 128: return launch<128>(a, s, stream);
    case 256: return launch<256>(a, s, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dg
