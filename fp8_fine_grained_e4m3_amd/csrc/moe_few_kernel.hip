// A mixture-of-experts layer for a few tokens, gfx950, in two kernels.
//
//   h(t, e) = silu(W1_e[:I] x_t) * (W1_e[I:] x_t)
//   y_t     = sum_j w_tj W2_{e_tj} h(t, e_tj)
// with e4m3 weights of one fp32 scale per 128 x 128 block (the GEMMs' B
// operand), bf16 x, and ids outside [0, E) taking no part.
//
// Bound: the weights of the experts that are reached are read once from HBM;
// everything else is small beside them.  So the weights go from HBM straight
// into registers in the layout of the MFMA's row operand (lane l: 16 bytes of
// row l & 15), are widened to bf16 there (exact) and multiplied by the tokens
// as columns, and no barrier stands between a weight's load and its use.  The
// product of a 128-K block is scaled and added to the fp32 accumulator, as in
// the GEMMs.
//  * Up: a workgroup takes 16 gate rows and the 16 up rows beside them of one
//    reached expert; its waves deal the K blocks among themselves and meet in
//    LDS, where silu and the product are taken in fp32.  h is stored as the
//    sum of bf16 parts, each the truncated rest of the one before: two parts
//    (2^-16 of h) where y is bf16, three (all of fp32's bits) where it is
//    fp32, so that the second product can use the matrix unit without
//    rounding h.
//  * Down: a workgroup takes 16 rows of y for up to 64 tokens over all reached
//    experts, so the sum over experts needs no atomics: its waves take equal
//    runs of (expert, K block), add each expert's weighted product to their
//    own fp32 slab in LDS, and the slabs are summed in order.
// The first kernel's workgroups find the reached experts from the ids by
// themselves (a bitmap in LDS) and leave each expert's tokens and weights in
// the workspace for the second.
#include "fp8_values.h"
#include "serve_internal.h"

#include <algorithm>

namespace dg {
namespace {

constexpr int kBlk = 128;
constexpr int kUpWaves = 4, kDownWaves = 8;
constexpr int kTile = 16;               // rows and tokens of a matrix tile
constexpr int kGroup = 64;              // tokens of a pass

// Workspace: per reached expert its number, its token count and its list.
struct Reached {
    int32_t expert, count;
};
struct Entry {
    int32_t pair;                       // t * topk + j: the row of h
    float weight;
};

struct MoeArgs {
    const uint16_t* x;
    const uint8_t* w1;
    const float* s1;
    const uint8_t* w2;
    const float* s2;
    const int32_t* ids;
    const float* weights;
    void* y;
    uint16_t* h;                        // [parts][T * topk][I]
    int32_t* reached_count;
    Reached* reached;                   // [min(E, T * topk)]
    Entry* entries;                     // [min(E, T * topk)][T]
    int T, topk, E, H, I;
};

// The MFMA fragments of a 128-byte K block of a weight row: lane l loads bytes
// [64 j + 16 g, + 16) of row l & 15, j = 0, 1; fragment 2 j + half takes eight
// of them, so K value (j, half, g, i) is 64 j + 16 g + 8 half + i.
struct WBlock {
    u32x4_t w[2];
};

__device__ __forceinline__ WBlock load_w(const uint8_t* p) {      // p: row + K block + 16 g
    WBlock b;
    b.w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
    b.w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 64));
    return b;
}

__device__ __forceinline__ bf16x8_t w_frag(const WBlock& b, int c) {
    const u32x4_t& w = b.w[c / 2];
    return c % 2 ? e4m3x8_to_bf16x8(w.z, w.w) : e4m3x8_to_bf16x8(w.x, w.y);
}

struct XBlock {
    u32x4_t x[4];
};

__device__ __forceinline__ XBlock load_x(const uint16_t* p, bool live) {   // p: row + K block + 16 g
    XBlock b;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        b.x[c] = u32x4_t{0, 0, 0, 0};
        if (live) b.x[c] = *reinterpret_cast<const u32x4_t*>(p + 64 * (c / 2) + 8 * (c % 2));
    }
    return b;
}

// The K blocks of a wave, gate and up rows by MT token tiles.
template <int MT>
__device__ __forceinline__ void up_products(const MoeArgs& a, const uint8_t* (&w)[2], const float* (&s)[2],
                                            const uint16_t* (&xr)[MT], const bool (&live)[MT], int wave,
                                            f32x4_t (&acc)[2][MT]) {
    const int KB = a.H / kBlk;
    for (int kb = wave; kb < KB; kb += kUpWaves) {
        WBlock wb[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) wb[r] = load_w(w[r] + (int64_t)kb * kBlk);
        XBlock xb[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) xb[t] = load_x(xr[t] + kb * kBlk, live[t]);
        f32x4_t p[2][MT];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) p[r][t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bf16x8_t f = w_frag(wb[r], c);
#pragma unroll
                for (int t = 0; t < MT; ++t) p[r][t] = mfma_bf16(f, __builtin_bit_cast(bf16x8_t, xb[t].x[c]), p[r][t]);
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float sc = s[r][kb];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(p[r][t][i], sc, acc[r][t][i]);
        }
    }
}

template <int PARTS, int MT>
__device__ __forceinline__ void up_pass(const MoeArgs& a, int e, int i0, int first, int count,
                                        const Entry* list, float* sm, int wave, int lane) {
    const int r16 = lane & 15, g = lane >> 4;
    const uint8_t* w[2];
    const float* s[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = i0 + r * a.I;
        w[r] = a.w1 + ((int64_t)e * 2 * a.I + row + r16) * a.H + 16 * g;
        s[r] = a.s1 + ((int64_t)e * (2 * a.I / kBlk) + row / kBlk) * (a.H / kBlk);
    }
    const uint16_t* xr[MT];
    bool live[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int at = first + 16 * t + r16;
        live[t] = at < count;
        const int token = live[t] ? list[at].pair / a.topk : 0;
        xr[t] = a.x + (int64_t)token * a.H + 16 * g;
    }
    f32x4_t acc[2][MT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
    up_products<MT>(a, w, s, xr, live, wave, acc);

    // [wave][gate, up][token][16 rows]
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t)
            *reinterpret_cast<f32x4_t*>(sm + (((wave * 2 + r) * MT + t) * 16 + r16) * 16 + 4 * g) = acc[r][t];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 256; i += kUpWaves * 64) {
        const int tok = i / 16, row = i % 16;
        if (first + tok < count) {
            float v[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                v[r] = 0.0f;
#pragma unroll
                for (int k = 0; k < kUpWaves; ++k) v[r] += sm[((k * 2 + r) * MT * 16 + tok) * 16 + row];
            }
            float rest = v[0] / (1.0f + __expf(-v[0])) * v[1];
            uint16_t* dst = a.h + (int64_t)list[first + tok].pair * a.I + i0 + row;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                uint32_t bits = __float_as_uint(rest) & 0xFFFF0000u;
                if (rest != rest) bits = 0x7FC00000u;
                dst[(int64_t)p * a.T * a.topk * a.I] = (uint16_t)(bits >> 16);
                // the rest of an infinity or a NaN is nothing
                rest = (bits & 0x7F800000u) == 0x7F800000u ? 0.0f : rest - __uint_as_float(bits);
            }
        }
    }
    __syncthreads();
}

template <int PARTS>
__global__ __launch_bounds__(kUpWaves * 64) void moe_up_kernel(MoeArgs a) {
    __shared__ uint32_t bitmap[kMoeMaxExperts / 32];
    __shared__ Entry list[kMoeMaxTokens];
    __shared__ float sm[kUpWaves * 2 * 4 * 256];
    __shared__ int found[2];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = a.I / kTile;
    const int tile = blockIdx.x % tiles, nth = blockIdx.x / tiles;
    const int pairs = a.T * a.topk;

    // the nth of the experts that are reached
    if (threadIdx.x < kMoeMaxExperts / 32) bitmap[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kUpWaves * 64) {
        const int id = a.ids[p];
        if (id >= 0 && id < a.E) atomicOr(&bitmap[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    if (wave == 0) {
        const uint32_t word = lane < kMoeMaxExperts / 32 ? bitmap[lane] : 0;
        const int c = __builtin_popcount(word);
        int before = c;                               // inclusive prefix over the words
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(before, o);
            if (lane >= o) before += v;
        }
        const int total = __builtin_amdgcn_readlane(before, 63);
        before -= c;
        if (lane == 0) found[0] = -1;
        if (nth >= before && nth < before + c) {
            uint32_t w = word;
            for (int i = before; i < nth; ++i) w &= w - 1;
            found[0] = lane * 32 + __builtin_ctz(w);
        }
        if (blockIdx.x == 0 && lane == 0) *a.reached_count = total;
    }
    __syncthreads();
    const int e = found[0];
    if (e < 0) return;                                // uniform

    // its tokens: a token's first slot with it carries the weights of all of them
    if (wave == 0) {
        int count = 0;
        for (int t0 = 0; t0 < a.T; t0 += 64) {
            const int t = t0 + lane;
            int first = -1;
            float weight = 0.0f;
            if (t < a.T)
                for (int j = 0; j < a.topk; ++j)
                    if (a.ids[t * a.topk + j] == e) {
                        if (first < 0) first = t * a.topk + j;
                        weight += a.weights[t * a.topk + j];
                    }
            const uint64_t have = __ballot(first >= 0);
            if (first >= 0) {
                const int at = count + __builtin_popcountll(have & ((1ull << lane) - 1));
                list[at] = Entry{first, weight};
                if (tile == 0) a.entries[(int64_t)nth * a.T + at] = Entry{first, weight};
            }
            count += __builtin_popcountll(have);
        }
        if (lane == 0) {
            found[1] = count;
            if (tile == 0) a.reached[nth] = Reached{e, count};
        }
    }
    __syncthreads();
    const int count = found[1];
    for (int first = 0; first < count; first += kGroup) {
        const int left = count - first;
        if (left <= 16) up_pass<PARTS, 1>(a, e, tile * kTile, first, count, list, sm, wave, lane);
        else if (left <= 32) up_pass<PARTS, 2>(a, e, tile * kTile, first, count, list, sm, wave, lane);
        else up_pass<PARTS, 4>(a, e, tile * kTile, first, count, list, sm, wave, lane);
    }
}

// One expert's K blocks [kb0, kb1) for 16 rows of y and MT tiles of its tokens
// from `first` on; the weighted product is added to the wave's slab.
template <int PARTS, int MT>
__device__ __forceinline__ void down_pass(const MoeArgs& a, int e, int n0, int kb0, int kb1, int first, int last,
                                          const Entry* list, int token0, float* slab, int lane) {
    const int r16 = lane & 15, g = lane >> 4;
    const uint8_t* w = a.w2 + ((int64_t)e * a.H + n0 + r16) * a.I + 16 * g;
    const float* s = a.s2 + ((int64_t)e * (a.H / kBlk) + n0 / kBlk) * (a.I / kBlk);
    const int64_t part = (int64_t)a.T * a.topk * a.I;
    const uint16_t* hr[MT];
    bool live[MT];
    int token[MT];
    float weight[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int at = first + 16 * t + r16;
        live[t] = at < last;
        Entry en{0, 0.0f};
        if (live[t]) en = list[at];
        hr[t] = a.h + (int64_t)en.pair * a.I + 16 * g;
        token[t] = en.pair / a.topk - token0;
        weight[t] = en.weight;
    }
    f32x4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4_t{0, 0, 0, 0};
    for (int kb = kb0; kb < kb1; ++kb) {
        const WBlock wb = load_w(w + (int64_t)kb * kBlk);
        XBlock hb[PARTS][MT];
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int t = 0; t < MT; ++t) hb[p][t] = load_x(hr[t] + p * part + kb * kBlk, live[t]);
        f32x4_t q[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) q[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bf16x8_t f = w_frag(wb, c);
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < MT; ++t) q[t] = mfma_bf16(f, __builtin_bit_cast(bf16x8_t, hb[p][t].x[c]), q[t]);
        }
        const float sc = s[kb];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(q[t][i], sc, acc[t][i]);
    }
    // a token is in an expert's list once: no two lanes of a tile meet
#pragma unroll
    for (int t = 0; t < MT; ++t)
        if (live[t]) {
            f32x4_t* at = reinterpret_cast<f32x4_t*>(slab + token[t] * kTile + 4 * g);
            *at += acc[t] * weight[t];
        }
}

template <int PARTS>
__global__ __launch_bounds__(kDownWaves * 64) void moe_down_kernel(MoeArgs a) {
    __shared__ float slabs[kDownWaves][kGroup * kTile];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * kTile, token0 = blockIdx.y * kGroup;
    const int tokens = min(a.T - token0, kGroup);
    float* slab = slabs[wave];
    for (int i = lane; i < kGroup * kTile; i += 64) slab[i] = 0.0f;

    const int KB = a.I / kBlk;
    const int64_t blocks = (int64_t)*a.reached_count * KB;
    const int64_t u0 = blocks * wave / kDownWaves, u1 = blocks * (wave + 1) / kDownWaves;
    for (int64_t u = u0; u < u1;) {
        const int nth = (int)(u / KB), kb0 = (int)(u - (int64_t)nth * KB);
        const int kb1 = (int)min((int64_t)KB, kb0 + (u1 - u));
        const int e = a.reached[nth].expert, count = a.reached[nth].count;
        const Entry* list = a.entries + (int64_t)nth * a.T;
        // the list is in order of tokens: this workgroup's are a run of it
        int first = 0, last = count;
        if (gridDim.y > 1) {
            int before = 0, within = 0;
            for (int i = lane; i < count; i += 64) {
                const int t = list[i].pair / a.topk;
                before += t < token0;
                within += t < token0 + kGroup;
            }
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) {
                before += __shfl_xor(before, o);
                within += __shfl_xor(within, o);
            }
            first = __builtin_amdgcn_readfirstlane(before);
            last = __builtin_amdgcn_readfirstlane(within);
        }
        // three parts of four tiles would not fit the registers
        for (constexpr int MOST = PARTS == 3 ? 2 : 4; first < last; first += 16 * MOST) {
            const int n = last - first;
            if (MOST == 4 && n > 32) down_pass<PARTS, MOST>(a, e, n0, kb0, kb1, first, last, list, token0, slab, lane);
            else if (n > 16) down_pass<PARTS, 2>(a, e, n0, kb0, kb1, first, last, list, token0, slab, lane);
            else down_pass<PARTS, 1>(a, e, n0, kb0, kb1, first, last, list, token0, slab, lane);
        }
        u += kb1 - kb0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * kTile; i += kDownWaves * 64) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kDownWaves; ++k) v += slabs[k][i];
        const int64_t at = (int64_t)(token0 + i / kTile) * a.H + n0 + i % kTile;
        if constexpr (PARTS == 3) static_cast<float*>(a.y)[at] = v;
        else static_cast<__bf16*>(a.y)[at] = (__bf16)v;
    }
}

template <int PARTS>
hipError_t launch(const MoeArgs& a, int slots, hipStream_t stream) {
    hipLaunchKernelGGL((moe_up_kernel<PARTS>), dim3((unsigned)((int64_t)slots * (a.I / kTile))),
                       dim3(kUpWaves * 64), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_down_kernel<PARTS>),
                       dim3((unsigned)(a.H / kTile), (unsigned)((a.T + kGroup - 1) / kGroup)),
                       dim3(kDownWaves * 64), 0, stream, a);
    return hipGetLastError();
}

constexpr int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

int64_t moe_few_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t I) {
    const int64_t slots = std::min(E, T * topk);
    return 16 + align16(slots * (int64_t)sizeof(Reached)) + align16(slots * T * (int64_t)sizeof(Entry)) +
           3 * T * topk * I * 2;
}

hipError_t launch_moe_few(const MoeFewProblem& p, hipStream_t stream) {
    MoeArgs a;
    a.x = p.x; a.w1 = p.w1; a.s1 = p.s1; a.w2 = p.w2; a.s2 = p.s2;
    a.ids = p.ids; a.weights = p.weights; a.y = p.y;
    a.T = (int)p.T; a.topk = (int)p.topk; a.E = (int)p.E; a.H = (int)p.H; a.I = (int)p.I;
    const int slots = std::min(a.E, a.T * a.topk);
    char* at = static_cast<char*>(p.workspace);
    a.reached_count = reinterpret_cast<int32_t*>(at);
    at += 16;
    a.reached = reinterpret_cast<Reached*>(at);
    at += align16(slots * (int64_t)sizeof(Reached));
    a.entries = reinterpret_cast<Entry*>(at);
    at += align16((int64_t)slots * a.T * (int64_t)sizeof(Entry));
    a.h = reinterpret_cast<uint16_t*>(at);
    return p.out_f32 ? launch<3>(a, slots, stream) : launch<2>(a, slots, stream);
}

}  // namespace dg
