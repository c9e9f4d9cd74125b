// Attention for a tree of drafted tokens, or one token, over the FP4 cache, gfx950.
//
// What is seen, o and lse are as over the FP8 cache (tree_attn_kernel.hip):
//   S_j = scale * (q . k_j),  o = sum_j softmax(S)_j v_j,  lse = ln sum_j exp S_j
// with k and v in e2m1 codes, a power-of-two scale (E8M0) for 32 values of a row.
//
// A value, code times scale, is a number of bf16, and one instruction makes two of
// them of a byte and a scale: both products run on the matrix unit in bf16, with keys
// and values exact.
//  * S^T = K q^T: lane l converts the D / 8 bytes of key l & 15 that it loaded itself,
//    values of one block of 32 (two for D = 256; half of one for D = 64); the query has
//    the same order of D in its fragments.
//  * S^T leaves lane l with keys 4 (l >> 4) + i of both 16-key tiles for row l & 15,
//    the operand layout of O^T = V^T P^T when the 32 keys are summed in that order: P
//    never leaves its lane.  V's operand needs 8 keys of one D value in a lane; a lane
//    loads D / 16 consecutive values of those 8 keys, all of one block, and exchanges
//    halves of words (v_perm) once they are bf16.  A key's scale of the block is a
//    rotation of the word of its scales: the conversion looks at the eight bits of the
//    exponent alone.
//  * P is rounded to fp16 for the second product: 11 bits, which bf16's 8 would make as
//    large an error as the output's own rounding, and fp16 holds the values exactly while
//    their scales are from 2^-18 to 2^13 (weights, 2^kTop as large, are kept to 2^-36 of the
//    largest).  Each step's scales are looked at, a word a lane; where one is out of that
//    range, or NaN, the wave takes its steps again for the rows that see it, in bf16, which
//    has fp32's exponents and holds every value, with P in two parts, the first 8 bits and
//    the next 8.  Rows that do not see it keep what they have, and their bits.  Where a row's
//    O passes fp32's largest number even so (values beyond 2^90), once more with that row's
//    weights 2^-kDown as large, which 2^30 weights of 2^kLazy do not outgrow; always so, the
//    exponentials' arguments would lose their last five bits.  (Always two bf16 parts: 145 us
//    against 124 for two trees of 16 over 100001.  Where all scales are out of fp16's range:
//    248 us against 127 for these, 91 against 52 for 32 single tokens over 8192.)
//  * Maximum, sum and O are fp32; the maximum follows where a score of the row passes it by
//    2^4, whatever other rows do, so that a row's bits are its own (all rows together: 124 us
//    against 126 for two trees of 16 over 100001).
// Codes hold neither NaN nor infinity and a hidden key's weight is 0, so what a row
// does not see reaches it only through a scale that is NaN.  Past the end of a request
// scales are replaced; where rows of one request see different keys, a NaN of a value
// is counted by a product of its own for the rows that see it.
//
// Bound: a few rows per key head leave the cache's bytes as the floor, half of the FP8
// cache's; with many rows each wave's chain of widening, product, exponentials and product
// is it, which two waves a SIMD overlap in part (two trees of 16 over 100001: VALU 47% and
// matrix unit 21% busy; the row blocks of a run widen the same keys, each for itself).  The
// cache goes from HBM straight to registers; a wave asks for its next step's keys and
// values when it is done with the ones it has, and the other waves of its SIMD cover the
// wait.  (Asked for during the step, or two steps ahead: the same times, and 10 to 40
// registers more.)  Work is cut into runs and joined as over the FP8 cache.
// Measured, in graphs, in tables as wide as the longest request (a batch "of n over c" goes
// from n tokens and c positions down to half of them): 32 single tokens over 8192, 32 / 8 heads of 128, 215 MB, 52 us, 4.1 TB/s,
// of which the first keys take 5 us to come (a loop over the same bytes alone: 38 us); one
// over 1000, 9.3 us; two trees of 16 over 100001, 64 / 8 heads of 128, 164 MB and 66 GFLOP,
// 126 us and 0.52 PFLOP/s; 7 trees of 24 over 3001, the last of them idle, 16 us.
#include "tree_attn_common.h"

#include <type_traits>

namespace dg {
namespace {

constexpr int kBrief = 24, kFew = 64;     // steps of requests that stay whole in a long table
constexpr float kLazy = 4.0f;             // how far, in powers of two, scores pass m before m follows
constexpr float kTop = 11.0f;             // weights are 2^kTop as large: up to 2^(kTop + kLazy), in fp16's range
constexpr uint32_t kLeast = 0x6D6D6D6Du;   // E8M0 of 2^-18 in each byte: from there on 32 scales are in fp16's range
constexpr float kDown = 45.0f;            // and 2^(kTop - kDown) where O would overflow

// One step's share of the cache in a lane.
template <int D>
struct Keys4 {
    static constexpr int VW = D == 256 ? 2 : 1;
    uint32_t k[2][D / 32];
    uint32_t v[2][4][VW];
    uint32_t ks[2];
    uint32_t vs[2];                       // of key 4 g + lane % 4 of each tile
};

// Where a step's two 16-key tiles lie (rows of the pool), uniform.
struct Place {
    int64_t row[2];
    bool live[2];                         // the tile has keys and a valid page
};

// floor(x / y) of whole numbers below 2^50.
__device__ __forceinline__ int64_t floor_div(int64_t x, int64_t y) {
    const int64_t q = (int64_t)((double)x / (double)y);
    return q * y > x ? q - 1 : q;         // a quotient that was rounded up to the next whole number
}

// The requests and steps of a run.
struct Span {
    int b, stride, end;                   // first request, from one to the next, past the last
    int ctx, n;                           // lengths of the first request, as given, where known
    bool known;
    int64_t s0, s1, start;                // the run's steps of all requests'; where request b starts
    int64_t total, runs, per, more;       // all steps; runs in use, of which `more` have per + 1 steps, the others per
    bool none;                            // the run has nothing to do

    __device__ __forceinline__ int64_t first_step(int64_t run) const { return per * run + min(run, more); }
    __device__ __forceinline__ int64_t run_of(int64_t step) const {
        const int64_t longer = more * (per + 1);
        return step < longer ? floor_div(step, per + 1) : more + floor_div(step - longer, per);
    }
};

// Several requests with no more than kBrief steps, or kFew where there are as many of
// them as runs, stay whole and are dealt to the runs in turn.
template <int W>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int run, int row0, int lane) {
    Span s = {run, 1, a.B, 0, 0, false, 0, 1ll << 62, 0, 0, 1, 1ll << 62, 0, false};
    if (a.whole) {
        s.end = run + 1;
        return s;
    }
    // this run's steps of all requests', and the request that they start in
    uint32_t upto = 0;                    // of the lane's request and those before it of its 64, 2^31 at most
    int ctx = 0, n = a.N;
    auto steps = [&](int b) {
        if (b >= a.B) return 0;
        ctx = a.ctx[b];
        n = a.tree ? a.tree[b] : a.N;
        return request_of(a, ctx, n, row0).steps;
    };
    bool brief = a.B > 1, few = a.B >= a.runs;
    for (int base = 0; base < a.B; base += 64) {
        const int own = steps(base + lane);
        brief = brief && !__any(own > kBrief);
        few = few && !__any(own > kFew);
        upto = sum_up_to_lane(own);
        s.total += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
    }
    if (brief || few) {
        s.stride = a.runs;
        return s;
    }
    s.runs = max((int64_t)1, min((int64_t)a.runs, s.total / W));
    if (run >= s.runs) {
        s.none = true;
        return s;
    }
    s.per = floor_div(s.total, s.runs);
    s.more = s.total - s.per * s.runs;
    s.s0 = s.first_step(run);
    s.s1 = s.first_step(run + 1);
    s.b = a.B;
    for (int base = 0; base < a.B; base += 64) {
        if (a.B > 64) upto = sum_up_to_lane(steps(base + lane));
        const uint32_t before = __shfl_up(upto, 1);
        const int64_t from = s.start + (lane > 0 ? before : 0u);
        const uint64_t hit = __ballot(base + lane < a.B && (s.start + upto > s.s0 || from >= s.s0));
        if (hit != 0) {
            const int at = __builtin_ctzll(hit);
            s.b = base + at;
            s.ctx = __builtin_amdgcn_readlane(ctx, at);
            s.n = __builtin_amdgcn_readlane(n, at);
            s.known = true;
            if (at > 0) s.start += (uint32_t)__builtin_amdgcn_readlane(upto, at - 1);
            break;
        }
        s.start += (uint32_t)__builtin_amdgcn_readlane(upto, 63);
    }
    return s;
}

// Two values of byte B of a word of codes as two bf16.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_to_bf16x2(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}

// The same as two fp16: exact for scales from 2^-23 to 2^13.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, B));
}

// The bits that any lane of l's group of 16 has.
__device__ __forceinline__ uint32_t any_of_group(uint32_t v) {
    v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);     // lane ^ 1
    v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);     // lane ^ 2
    v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);    // the other four of eight
    v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);    // the other eight of sixteen
    return v;
}

// The bits that any of lanes l, l ^ 16, l ^ 32 and l ^ 48 has.
__device__ __forceinline__ uint32_t any_of_groups(uint32_t v) {
    u32x2_t s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = s.x | s.y;
    s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return s.x | s.y;
}

// Eight values of a word as an MFMA fragment.
__device__ __forceinline__ bf16x8_t e2m1x8_to_bf16x8(uint32_t w, float scale) {
    const u32x4_t r = {e2m1x2_to_bf16x2<0>(w, scale), e2m1x2_to_bf16x2<1>(w, scale), e2m1x2_to_bf16x2<2>(w, scale),
                       e2m1x2_to_bf16x2<3>(w, scale)};
    return __builtin_bit_cast(bf16x8_t, r);
}

// A uniform place in memory, kept in scalar registers: what a lane adds to it (in 32 bits)
// stays an offset of the load, and takes no 64-bit sums in vector registers.
typedef const __attribute__((address_space(1))) uint8_t* Uniform;

__device__ __forceinline__ Uniform uniform(const uint8_t* p) {
    uint64_t u = reinterpret_cast<uintptr_t>(p);
    asm("" : "+s"(u));                    // the compiler cannot take the sum apart again
    return reinterpret_cast<Uniform>(u);
}

template <typename T>
__device__ __forceinline__ T load_at(Uniform base, uint32_t place, int more = 0) {
    return *reinterpret_cast<const __attribute__((address_space(1))) T*>(base + place + more);
}

// f(0), .., f(N - 1), each a constant.
template <int N, typename F>
__device__ __forceinline__ void for_bytes(F f) {
    if constexpr (N > 1) for_bytes<N - 1>(f);
    f(std::integral_constant<int, N - 1>());
}

// V's operands of D values 2 B and 2 B + 1 of a lane's D / 16: pairs of its 8 keys.
template <int B, int D, typename F>
__device__ __forceinline__ void pairs(const Keys4<D>& x, const uint32_t (&scale)[2][4], u32x4_t& even, u32x4_t& odd, F convert) {
    constexpr std::integral_constant<int, B % 4> byte{};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a = convert(byte, x.v[u][2 * i][B / 4], scale[u][2 * i]);
            const uint32_t b = convert(byte, x.v[u][2 * i + 1][B / 4], scale[u][2 * i + 1]);
            even[2 * u + i] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            odd[2 * u + i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        }
}

// RT: row tiles, of each of a workgroup's W waves the same.
template <int D, int RT, int W>
__global__ __launch_bounds__(W * 64, W == 16 ? 4 : D == 256 ? 1 : D == 128 || W == 8 ? 2 : 3) void tree_attn4_kernel(AttnArgs a) {
    constexpr int DT = D / 16;            // 16-row tiles of O^T
    constexpr int ROWS = 16 * RT;
    constexpr int PITCH = D + 4;          // of a row of O in LDS
    constexpr int PART = ROWS * (D + 2);  // floats of a part
    typedef Keys4<D> Keys;
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

    const Span span = span_of<W>(a, run, row0, lane);
    if (span.none) return;
    int64_t start = span.start;           // of request b
    // r / G of rows below 2^20: what the product is off by is less than half of 1 / G
    const float one_of_g = 1.0f / (float)a.G;
    auto token_of = [&](int r) { return (int)(((float)r + 0.5f) * one_of_g); };
    for (int b = span.b; b < span.end && (start < span.s1 || (run == span.runs - 1 && start == span.total)); b += span.stride) {
    // What does not depend on the request's lengths is asked for before they are known:
    // its first pages and queries.
    const int lo = (int)max(span.s0 - start, (int64_t)0);
    const Uniform pages_of = uniform(reinterpret_cast<const uint8_t*>(a.table + (int64_t)b * a.max_pages));
    // Lanes 2 n and 2 n + 1 ask for the pages of a step's two tiles: vector loads,
    // in the order of the others, two steps ahead.
    auto ask = [&](int step) {
        const int page = min((step * kStep + 16 * (lane & 1)) >> a.page_shift, a.max_pages - 1);
        return load_at<int32_t>(pages_of, 4 * page);
    };
    int pages = ask(lo + wave), pages_next = ask(lo + wave + W), pages_after = ask(lo + wave + 2 * W);
    // the lane's query row of each row tile, its D values in the keys' order
    const int qlane = fresh(lane), qr16 = qlane & 15, qg = qlane >> 4;
    u32x4_t query[RT][D / 32];
    int tok[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = min(row0 + 16 * t + qr16, all_rows - 1);
        tok[t] = token_of(r);
        const int hq = h * a.G + r - tok[t] * a.G;
        const uint16_t* src = a.q + ((int64_t)b * a.N + tok[t]) * a.q_stride + (int64_t)hq * D + qg * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) query[t][c] = *reinterpret_cast<const u32x4_t*>(src + c * 8);
    }
    // a token alone that does not see itself is as good as past the end
    const bool blind = a.N == 1 && a.mask && !(uniform_input(reinterpret_cast<const int32_t*>(a.mask + b)) & 1);
    const Request rq = span.known && b == span.b ? request_of(a, span.ctx, span.n, row0) : request(a, b, row0);
    const int ctx = rq.ctx, rows = rq.n * a.G;
    const int L = blind ? min(ctx, rq.L) : rq.L;
    const int hi = (int)min(span.s1 - start, (int64_t)rq.steps);
    start += rq.steps;
    auto out_row = [&](int r) {
        const int token = token_of(r);
        return ((int64_t)b * a.N + token) * Hq + h * a.G + r - token * a.G;
    };
    const bool whole = lo == 0 && hi == rq.steps;
    if (lo == 0 && threadIdx.x == 0 && !a.whole && a.runs > 1) {
        // the run of the request's last step
        const int64_t last = whole ? run - 1 : span.run_of(start - 1);
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
    bf16x8_t qf[RT][D / 32];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            qf[t][c] = __builtin_bit_cast(bf16x8_t, row0 + 16 * t + qr16 < rows ? query[t][c] ^ (a.scale < 0.0f ? 0x80008000u : 0u)
                                                                                : u32x4_t{0, 0, 0, 0});
    f32x4_t acc[RT][DT];
    float m[RT], base[RT], l[RT];         // base: m + down, or 0 while nothing was seen, so that exp2 stays 0
    float down[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) down[t] = -kTop;
    // Whether a scale of a value was out of fp16's range: in a step that all rows see, and, bit
    // t, one that the lane's row of tile t sees.
    uint32_t out = 0, out_seen = 0;
    auto pass = [&](auto is_wide) {
    constexpr bool WIDE = decltype(is_wide)::value;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = -__builtin_inff();
        base[t] = 0.0f;
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[t][i] = f32x4_t{0, 0, 0, 0};
    }
    // Scores stay products until the exponential: with a scale that is not negative (the
    // query's sign takes that) they are in the same order.  Above 0, so that -infinity stays, and
    // so little that no product brings a score with the scale 0 to 2^-20.
    const float c2 = __builtin_fmaxf(__builtin_fabsf(a.scale) * kLog2e, 0x1p-149f);
    const bool apart = a.N > 1;           // rows of several tokens: they may see different keys
    if (lo + wave < hi) {
    // uniform bases, a lane's place in 32 bits
    uint32_t k_off = r16 * (D / 2) + g * (D / 8), ks_off = r16 * (D / 32) + (D == 64 ? g / 2 : g * (D / 128));
    uint32_t v_off = 4 * g * (D / 2) + r16 * (D / 32), vs_off = (4 * g + (r16 & 3)) * (D / 32) + (D == 256 ? r16 / 8 * 4 : 0);
    // rotation that brings the block's byte of a word of scales to the exponent's place
    const uint32_t turn = (8 * (D == 64 ? r16 / 8 : D == 128 ? r16 / 4 : r16 / 2 % 4) - 23) & 31;
    Keys x;
    const uint8_t* const k_sf = static_cast<const uint8_t*>(a.ks);
    const uint8_t* const v_sf = static_cast<const uint8_t*>(a.vs);
    auto fetch_k = [&](const Place& w, int t) {
        asm volatile("" : "+v"(k_off), "+v"(ks_off));
        const Uniform from = uniform(a.kc + w.row[t] * (D / 2));
        if constexpr (D == 64) {
            const u32x2_t v = load_at<u32x2_t>(from, k_off);
            x.k[t][0] = v.x;
            x.k[t][1] = v.y;
        } else {
#pragma unroll
            for (int c = 0; c < D / 128; ++c) {
                const u32x4_t v = load_at<u32x4_t>(from, k_off, 16 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) x.k[t][4 * c + i] = v[i];
            }
        }
        const Uniform sf = uniform(k_sf + w.row[t] * (D / 32));
        if constexpr (D == 256) x.ks[t] = load_at<uint16_t>(sf, ks_off);
        else x.ks[t] = load_at<uint8_t>(sf, ks_off);
    };
    auto fetch_v = [&](const Place& w) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            asm volatile("" : "+v"(v_off), "+v"(vs_off));
            const Uniform from = uniform(a.vc + w.row[t] * (D / 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 64) {
                    x.v[t][i][0] = load_at<uint16_t>(from, v_off, i * (D / 2));
                } else if constexpr (D == 128) {
                    x.v[t][i][0] = load_at<uint32_t>(from, v_off, i * (D / 2));
                } else {
                    const u32x2_t v = load_at<u32x2_t>(from, v_off, i * (D / 2));
                    x.v[t][i][0] = v.x;
                    x.v[t][i][1] = v.y;
                }
            }
            const Uniform sf = uniform(v_sf + w.row[t] * (D / 32));
            if constexpr (D == 64) x.vs[t] = load_at<uint16_t>(sf, vs_off);
            else x.vs[t] = load_at<uint32_t>(sf, vs_off);
        }
    };
    int ahead[2] = {pages_next, pages_after};     // pages of the two steps after this one
    Place at = place(lo + wave, pages);
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
        const Place next = place(s + W, ahead[0]);
        ahead[0] = ahead[1];
        ahead[1] = ask(s + 3 * W);
        __builtin_amdgcn_sched_barrier(0);
        const bool all = j0 + kStep <= ctx && at.live[0] && at.live[1];      // uniform: no mask here
        float sc[RT][2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bf16x8_t kf[D / 32];
            const float s0 = __uint_as_float(x.ks[u] << 23), s1 = D == 256 ? __uint_as_float(x.ks[u] << 15) : s0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) kf[c] = e2m1x8_to_bf16x8(x.k[u][c], c < 4 ? s0 : s1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                f32x4_t p = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < D / 32; ++c) p = mfma_bf16(kf[c], qf[t][c], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[t][u][i] = p[i];
            }
        }
        // whether fp16 holds the step's values
        if (!WIDE && all) {
            constexpr uint32_t least = D == 64 ? kLeast & 0xFFFF : kLeast;
            out |= ((x.vs[0] - least) | (x.vs[1] - least)) & 0xE0E0E0E0u;
        }
        // Scales of the lane's block of its 8 keys' values, from the lanes of its quad.  These
        // have the same block (for D = 256 two, of the word that they all have).
        uint32_t vscale[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t own = x.vs[u];
            if constexpr (D < 256) own = __builtin_amdgcn_alignbit(own, own, turn);
            vscale[u][0] = __float_as_uint(of_quad<0>(__uint_as_float(own)));
            vscale[u][1] = __float_as_uint(of_quad<1>(__uint_as_float(own)));
            vscale[u][2] = __float_as_uint(of_quad<2>(__uint_as_float(own)));
            vscale[u][3] = __float_as_uint(of_quad<3>(__uint_as_float(own)));
            if constexpr (D == 256)
#pragma unroll
                for (int i = 0; i < 4; ++i) vscale[u][i] = __builtin_amdgcn_alignbit(vscale[u][i], vscale[u][i], turn);
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
            // scales past the end may be NaN: 0 * NaN must not reach O
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!at.live[u] || j0 + 16 * u + 4 * g + i >= L) vscale[u][i] = 0x3F800000u;
            if (!WIDE) {
                auto far = [&](int u, int i) { return ((vscale[u][i] & 0x7F800000u) - (kLeast << 24 >> 1)) & 0xF0000000u; };
                uint32_t any = 0;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) any |= far(u, i);
                if (__any(any != 0)) {
                    // One out of the range, or NaN, counts for the rows that see its key alone: those take
                    // their steps again, and to the others it must not be more than 0 times a number.
                    uint32_t off = 0;     // bit 4 u + i
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (far(u, i)) {
                                off |= 1u << (4 * u + i);
                                vscale[u][i] = 0x3F800000u;
                            }
                    off = any_of_group(off);       // of all blocks: the 16 lanes have different ones
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if ((off >> (4 * u + i) & 1) && sc[t][u][i] != -__builtin_inff()) out_seen |= 1u << t;
                }
            }
            if (WIDE && apart) {
                bool bad = false;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) bad |= (vscale[u][i] & 0x7F800000u) == 0x7F800000u;
                if (__any(bad)) {
                    // ones where a value is NaN, times ones where a row sees its key: rows that see any
                    u32x4_t ind;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const bool first = (vscale[u][2 * i] & 0x7F800000u) == 0x7F800000u;
                            const bool second = (vscale[u][2 * i + 1] & 0x7F800000u) == 0x7F800000u;
                            ind[2 * u + i] = (first ? 0x3F80u : 0) | (second ? 0x3F800000u : 0);
                            if (first) vscale[u][2 * i] = 0x3F800000u;
                            if (second) vscale[u][2 * i + 1] = 0x3F800000u;
                        }
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        u32x4_t see;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                see[2 * u + i] = (sc[t][u][2 * i] != -__builtin_inff() ? 0x3F80u : 0) |
                                                 (sc[t][u][2 * i + 1] != -__builtin_inff() ? 0x3F800000u : 0);
                        const f32x4_t count = mfma_bf16(__builtin_bit_cast(bf16x8_t, ind), __builtin_bit_cast(bf16x8_t, see),
                                                        f32x4_t{0, 0, 0, 0});
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (count[k] > 0.0f)
#pragma unroll
                                for (int i = 0; i < DT; ++i) acc[t][i][k] = __builtin_nanf("");
                    }
                }
            }
        }
        // A wave in its softmax goes before one in its products.
        __builtin_amdgcn_s_setprio(1);
        // Whether a score outgrows what O is relative to.  The lanes look at their own;
        // only then is the row's maximum exchanged.
        float mx[RT];
        bool over = false;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            mx[t] = sc[t][0][0];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[t] = __builtin_fmaxf(mx[t], sc[t][u][i]);
            mx[t] *= c2;
            over |= mx[t] > m[t] + kLazy;
        }
        if (__any(over)) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                // each row by its own scores: what the others have takes no bits of it
                mx[t] = max_of_groups(mx[t]);
                float f = 1.0f;
                if (mx[t] > m[t] + kLazy) {
                    const float from = base[t];
                    base[t] = mx[t] + down[t];
                    f = m[t] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(from - base[t]);
                    m[t] = mx[t];
                }
                l[t] *= f;
#pragma unroll
                for (int i = 0; i < DT; ++i) acc[t][i] *= f;
            }
        }
        float e[RT][2][4];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[t][u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][u][i], c2, -base[t]));
                    l[t] += e[t][u][i];
                }
        if constexpr (!WIDE) {
            f16x8_t pf[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                u32x4_t w;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) w[2 * u + i] = f32x2_to_f16x2(e[t][u][2 * i], e[t][u][2 * i + 1]);
                pf[t] = __builtin_bit_cast(f16x8_t, w);
            }
            __builtin_amdgcn_s_setprio(0);
            for_bytes<D / 32>([&](auto byte) {
                constexpr int B = decltype(byte)::value;
                u32x4_t even, odd;
                pairs<B>(x, vscale, even, odd, [](auto b, uint32_t w, uint32_t sf) {
                    return e2m1x2_to_f16x2<decltype(b)::value>(w, __uint_as_float(sf));
                });
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    acc[t][2 * B] = mfma_f16(__builtin_bit_cast(f16x8_t, even), pf[t], acc[t][2 * B]);
                    acc[t][2 * B + 1] = mfma_f16(__builtin_bit_cast(f16x8_t, odd), pf[t], acc[t][2 * B + 1]);
                }
            });
        } else {
            bf16x8_t p_hi[RT], p_lo[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                u32x4_t top, rest;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e0 = e[t][u][2 * i], e1 = e[t][u][2 * i + 1];
                        const uint32_t b0 = __float_as_uint(e0), b1 = __float_as_uint(e1);
                        top[2 * u + i] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
                        rest[2 * u + i] = f32x2_to_bf16x2(e0 - __uint_as_float(b0 & 0xFFFF0000u), e1 - __uint_as_float(b1 & 0xFFFF0000u));
                    }
                p_hi[t] = __builtin_bit_cast(bf16x8_t, top);
                p_lo[t] = __builtin_bit_cast(bf16x8_t, rest);
            }
            __builtin_amdgcn_s_setprio(0);
            for_bytes<D / 32>([&](auto byte) {
                constexpr int B = decltype(byte)::value;
                u32x4_t even, odd;
                pairs<B>(x, vscale, even, odd, [](auto b, uint32_t w, uint32_t sf) {
                    return e2m1x2_to_bf16x2<decltype(b)::value>(w, __uint_as_float(sf));
                });
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    acc[t][2 * B] = mfma_bf16(__builtin_bit_cast(bf16x8_t, even), p_lo[t], acc[t][2 * B]);
                    acc[t][2 * B + 1] = mfma_bf16(__builtin_bit_cast(bf16x8_t, odd), p_lo[t], acc[t][2 * B + 1]);
                    acc[t][2 * B] = mfma_bf16(__builtin_bit_cast(bf16x8_t, even), p_hi[t], acc[t][2 * B]);
                    acc[t][2 * B + 1] = mfma_bf16(__builtin_bit_cast(bf16x8_t, odd), p_hi[t], acc[t][2 * B + 1]);
                }
            });
        }
        __builtin_amdgcn_sched_barrier(0);
        fetch_k(next, 0);
        fetch_k(next, 1);
        fetch_v(next);
        __builtin_amdgcn_sched_barrier(0);
        at = next;
    }
    }
    };
    pass(std::false_type());
    // the lane's values of O of its row of tile t, in the wave's LDS
    auto o_of = [&](int t, int l) { return sm_o[wave] + (16 * t + (l & 15)) * PITCH + 4 * (l >> 4) * DT; };
    if (__any(out | out_seen)) {
        // The rows that saw such a scale take the steps again in bf16, and once more where O passed fp32's
        // largest number; the others keep what they have, so that it hangs on what they see alone.
        const uint32_t again = __any(out) ? ~0u : any_of_groups(out_seen);
        float m16[RT], base16[RT], l16[RT];
        const int put = fresh(lane);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            m16[t] = m[t], base16[t] = base[t], l16[t] = l[t];
#pragma unroll
            for (int i = 0; i < DT; ++i) *reinterpret_cast<f32x4_t*>(o_of(t, put) + 4 * i) = acc[t][i];
        }
        for (int n = 0; n < 2; ++n) {
            pass(std::true_type());
            bool off = false;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                float sum = 0.0f;         // 0, or NaN
#pragma unroll
                for (int i = 0; i < DT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum = __builtin_fmaf(acc[t][i][k], 0.0f, sum);
                down[t] = max_of_groups(sum == 0.0f ? -kTop : kDown - kTop);
                off |= down[t] > 0.0f;
            }
            if (!__any(off)) break;
        }
        const int get = fresh(lane);      // another copy: what was put down is not kept in registers
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (again >> t & 1) continue;
            m[t] = m16[t], base[t] = base16[t], l[t] = l16[t];
#pragma unroll
            for (int i = 0; i < DT; ++i) acc[t][i] = *reinterpret_cast<const f32x4_t*>(o_of(t, get) + 4 * i);
        }
    }

    // The waves put down their O and meet: a thread then adds up four values of a
    // row, wave by wave, relative to the largest of their maxima.
    const int elane = fresh(lane), er16 = elane & 15, eg = elane >> 4;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] = sum_of_groups(l[t]);
        // the sum's power of two goes to the maximum
        const int k = __builtin_amdgcn_frexp_expf(l[t]), shift = -k - kSpare;
        const float top = m[t] == -__builtin_inff() ? m[t] : base[t] + (float)k;
        if (eg == 0) sm_ml[wave][16 * t + er16] = f32x2_t{top, __builtin_amdgcn_ldexpf(l[t], -k)};
        float* mine = o_of(t, elane);
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

// Rows of a workgroup: 16 where there are no more (and for D = 256, whose O fills
// the registers), and where 32 would leave CUs without a workgroup and keys are few
// enough to be widened twice; else 32.  16 against 32 rows, in graphs, D = 128: 8 trees
// of 16 over 1000, 32 / 8 heads, 11.7 us against 16.4; over 8000, 39 against 43; but over
// 14000, 63 against 57; 16 of 16 over 1000, 14.7 against 16.6; but over 3000, 30 against 28.
// D = 64: 7 trees of 24 over 3001, 32 / 4 heads, 16 against 21.  (64, with the query in
// LDS: 33 us for these when 32 took 20; D = 128 does not fit the registers, 182 us against 123.)
// Whole requests, a workgroup each and no second kernel, where that is soon done
// whatever the lengths turn out to be: up to 1024 positions (D = 256: 512), up to 2048
// where requests and heads make 32 workgroups (D = 256: 128), up to 4096 where they make
// 128 (not D = 256), up to 12288 where they make 256 of 16 rows.  Split against whole: 8 of
// 2000, 16.8 us against 13.4; 16 of 3000, 20.6 against 17.9; 24 of 4000, 25.5 against 22.0; 4
// trees of 16 over 3000, 21.8 against 17.8; 32 of 8192, 57.4 against 51.9; 128 of 8192, 189
// against 177; but 8 of 4000, 18.6 against 21.2, 16 of 8192, 33 against 43, and one of 1000
// with D = 256, 11.3 against 13.3.
// A whole request has eight waves, four where 16 steps are all (one of 1000: 9.3 us with
// eight, 10.6 with four; 32 of 4000, 28 and 39), and as many fewer as are resident with all
// the others, halved only where that leaves a wave 16 steps at most.
// Runs: two workgroups of four waves a CU of 256, or one of eight where requests may be
// long (fewer parts to join: one of 20000, 14.2 us against 16.1; 16 of 8192, 33 against
// 35; 4 of 2000, 14.7 against 14.4).  D = 64 with two row tiles has room for a third wave a
// SIMD only in workgroups of four (16 trees of 20 over 8000: 38 us against 44).  D = 256:
// one workgroup a CU, of eight waves where each has 8 steps (16 of 8192, 55 us against 57;
// one tree of 33 over 8192, 61 against 69; but 8 trees of 2 over 8000, 26 against 24).
// D = 64 with one row tile has registers for four waves a SIMD: sixteen a workgroup where
// requests may be long and a CU has one of them (32 of 8192, 34 us against 42; 40 of
// 8192, 45 against 47; split, 32 of 20000, 76 against 85; but 32 of 1000 in either table
// 1 us more, and with fewer or more requests, 16 of 8192, 25.3 against 24.7, 8 of 1000 in a
// table of 60000, 16 against 14, 256 of 300 in one of 20000, 38.6 against 36.2).
// From the sizes alone: lengths are on the device.  All these figures are of tables as wide
// as the longest request; short requests in a wider one are cut as if they were long (the
// 7 trees of 24 in a table of 32768: 26 us against 16; 8 trees of 16 over 1000: 26 against 11.5).
Shape shape_of(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D, int64_t max_pages, int64_t page_size) {
    const int64_t rows = N * (Hq / H), most = (max_pages * page_size + kStep - 1) / kStep;
    const int64_t pairs = (rows + 31) / 32 * B * H;     // workgroups of two row tiles
    Shape s;
    s.row_tiles = rows <= 16 || D == 256 || (pairs < 256 && most <= 256) || (pairs < 512 && most <= 32) ? 1 : 2;
    s.row_blocks = (int)((rows + s.rows() - 1) / s.rows());
    const int64_t groups = H * s.row_blocks, steps = B * most;
    const int64_t workgroups = B * groups;
    s.whole = most <= (D == 256 ? 16 : 32) || (D <= 128 && most <= 64 && workgroups >= 32) ||
              (most <= (D == 256 ? 64 : 128) && workgroups >= 128) ||
              (s.row_tiles == 1 && most <= 384 && workgroups >= 256);
    if (workgroups > (1 << 20)) s.whole = false;       // a grid has fewer than 2^32 threads
    const bool sixteen = D * s.row_tiles == 64 && most > 64 && workgroups >= 256 && workgroups < 512;
    if (s.whole) {
        const int64_t resident = 1024 * (D == 64 ? 3 : 2);
        s.waves = s.row_tiles == 2 || most > 16 ? 8 : 4;
        if (sixteen) s.waves = 16;
        while (s.waves > 1 && workgroups * s.waves > resident && 2 * most <= 16 * s.waves) s.waves /= 2;
        s.runs = (int)B;
        return s;
    }
    if (D == 256) s.waves = steps * groups >= 256 * 64 ? 8 : 4;
    else s.waves = most > 128 && (D == 128 || s.row_tiles == 1) ? 8 : 4;
    if (sixteen) s.waves = 16;
    const int64_t wanted = D == 256 || s.waves >= 8 ? 256 : 512;
    s.runs = (int)std::max<int64_t>(1, std::min(wanted / groups, steps / s.waves));
    return s;
}

template <int D, int RT>
void launch_waves(const AttnArgs& a, int waves, dim3 grid, hipStream_t stream) {
    if (waves == 1) hipLaunchKernelGGL((tree_attn4_kernel<D, RT, 1>), grid, dim3(64), 0, stream, a);
    else if (waves == 2) hipLaunchKernelGGL((tree_attn4_kernel<D, RT, 2>), grid, dim3(128), 0, stream, a);
    else if (waves == 4) hipLaunchKernelGGL((tree_attn4_kernel<D, RT, 4>), grid, dim3(256), 0, stream, a);
    else if (waves == 8) hipLaunchKernelGGL((tree_attn4_kernel<D, RT, 8>), grid, dim3(512), 0, stream, a);
    else if constexpr (D * RT == 64) hipLaunchKernelGGL((tree_attn4_kernel<D, RT, 16>), grid, dim3(1024), 0, stream, a);
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
    return launch_join<D>(a, s.rows(), stream);
}

}  // namespace

int64_t tree_attn4_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D,
                                   int64_t max_pages, int64_t page_size) {
    return shape_workspace_bytes(B, H, D, shape_of(B, N, Hq, H, D, max_pages, page_size));
}

hipError_t launch_tree_attn4(const TreeAttnProblem& p, hipStream_t stream) {
    const Shape s = shape_of(p.B, p.N, p.Hq, p.cache.H, p.cache.D, p.max_pages, p.cache.page_size);
    const AttnArgs a = args_of(p, s);
    switch (p.cache.D) {
    case 64: return launch<64>(a, s, stream);
    case 128: return launch<128>(a, s, stream);
    case 256: return launch<256>(a, s, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dg
