// A mixture-of-experts layer for a few tokens, gfx950, in two kernels.
//
//   h(t, e) = silu(W1_e[:I] x_t) * (W1_e[I:] x_t)
//   y_t     = sum_j w_tj W2_{e_tj} h(t, e_tj)
// with e4m3 weights of one fp32 scale per 128 x 128 block (the GEMMs' B
// operand), bf16 x, and ids outside [0, E) taking no part.
//
// Bound: the weights of the experts that are reached are read once from HBM;
// everything else is small beside them.  So a wave fetches them in whole cache
// lines into registers, a block ahead, and passes them through its own piece of
// LDS, without a barrier, into the layout of the MFMA's row operand; they are
// widened to bf16 there (exact) and multiplied by the tokens as columns.  The
// product of a 128-K block is scaled and added to the fp32 accumulator, as in
// the GEMMs.
//  * Up: a workgroup takes 16 or 32 gate rows and the up rows beside them of one
//    reached expert; its waves deal the K blocks among themselves and meet in
//    LDS, where silu and the product are taken in fp32.  h is stored as the
//    sum of bf16 parts, each the truncated rest of the one before: two parts
//    (2^-16 of h) where y is bf16, three (all of fp32's bits) where it is
//    fp32, so that the second product can use the matrix unit without
//    rounding h.
//  * Down: a workgroup takes some rows of y for up to 64 tokens over the reached
//    experts, or a share of them; each expert's weighted product is added to an
//    fp32 slab in LDS.  The sums over experts need no atomics: slabs and shares
//    are added in order, the shares by the one that arrives last.
// The first kernel's workgroups find the reached experts from the ids by
// themselves (a bitmap in LDS) and leave each expert's tokens and weights in
// the workspace for the second.
//
// Measured, times of a whole layer with the weights' bytes over them: 1 token of
// 6 in 32 experts, 4096 x 2048: 37 us, 4.1 TB/s (each kernel's start and end are
// a third of it); 13 tokens: 134 to 140 us, 5.2 to 5.5 TB/s; 64 of 8 in 64 experts, 7168 x
// 2048, fp32: 536 us, 5.3 TB/s.  A plain read of as many bytes reaches 6.2.
#include "fp8_values.h"
#include "serve_internal.h"

#include <algorithm>
#include <type_traits>

namespace dg {
namespace {

constexpr int kBlk = 128;
constexpr int kUpWaves = 4, kDownWaves = 4;
constexpr int kTile = 16;               // rows and tokens of a matrix tile
constexpr int kGroup = 64;              // tokens of a pass

// Workspace, for each group of kGroup tokens: the reached experts with the
// tokens that they have there, `count` entries from `first` on, in token order.
struct Reached {
    int32_t expert, first, count;
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
    Reached* reached;                   // [groups][slots]
    Entry* entries;                     // [T * topk]: a group's from group * kGroup * topk on
    float* parts;                       // the second kernel's shares of y
    int32_t* arrived;                   // [row tiles][groups]: shares done, zeroed by the first kernel
    int T, topk, E, H, I, slots;        // slots: min(E, T * topk)
    int shares, counters;
};

// A 128-K block of NW tiles of 16 weight rows and of MT tiles of 16 columns on
// its way from memory to the matrix unit.  A weight row's block is one cache
// line, a column's two (a half of 64 K values each).  Lane l fetches 16 bytes,
// number l & 7, of lines l >> 3 and 8 + (l >> 3) of a tile, so an instruction
// asks for 8 whole lines; the wave passes them through its own piece of LDS,
// chunk c of line k at place c ^ (k & 7), to get the matrix operands.  (Fetching
// operands straight from memory, 16 rows of 64 bytes an instruction, asks the
// L1 for a line a lane, of which it looks up about one a clock, and fetches a
// line's halves apart: 4.9 TB/s in a plain read, against 6.2.)
// Operand lane l: bytes [16 g, + 16) of half h of row l & 15, g = l >> 4; fragment
// c takes eight of them, so its K value (g, i) is 64 h + 16 g + 8 c + i.
template <int NW, int MT>
struct Block {
    static constexpr int STAGE = (NW + MT) * 128;      // 16-byte chunks of LDS a wave
    u32x4_t w[NW][2];
    u32x4_t x[2][MT][2];

    // at(r, i): the lane's place in lines i of weight tile r
    template <typename F>
    __device__ __forceinline__ void load_w(F at) {
#pragma unroll
        for (int r = 0; r < NW; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) w[r][i] = *reinterpret_cast<const u32x4_t*>(at(r, i));
    }

    // at(t, i): the lane's place in columns i of tile t, first half
    template <typename F>
    __device__ __forceinline__ void load_x(F at) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) x[h][t][i] = *reinterpret_cast<const u32x4_t*>(at(t, i) + 128 * h);
    }

    // p = weights . columns; next_w and next_x fetch the next block into this one
    // as soon as its registers are free.
    template <typename F, typename G>
    __device__ __forceinline__ void multiply(u32x4_t* stage, int lane, f32x4_t (&p)[NW][MT], F next_w, G next_x) {
        u32x4_t* xs = stage + NW * 128;
        const int put = lane ^ (lane >> 3);                                  // line l >> 3, chunk l & 7
        const int row = (lane & 15) * 8, g = lane >> 4, turn = lane & 7;     // line l & 15
#pragma unroll
        for (int r = 0; r < NW; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) stage[r * 128 + i * 64 + put] = w[r][i];
        __builtin_amdgcn_sched_barrier(0);
        next_w();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < NW; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) p[r][t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) xs[t * 128 + i * 64 + put] = x[h][t][i];
            if (h == 1) {
                __builtin_amdgcn_sched_barrier(0);
                next_x();
                __builtin_amdgcn_sched_barrier(0);
            }
            wave_lds_order();
            u32x4_t v[NW];
#pragma unroll
            for (int r = 0; r < NW; ++r) v[r] = stage[r * 128 + row + ((4 * h + g) ^ turn)];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                bf16x8_t f[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) f[t] = __builtin_bit_cast(bf16x8_t, xs[t * 128 + row + ((2 * g + c) ^ turn)]);
#pragma unroll
                for (int r = 0; r < NW; ++r) {
                    const bf16x8_t a = c ? e4m3x8_to_bf16x8(v[r].z, v[r].w) : e4m3x8_to_bf16x8(v[r].x, v[r].y);
#pragma unroll
                    for (int t = 0; t < MT; ++t) p[r][t] = mfma_bf16(a, f[t], p[r][t]);
                }
            }
            wave_lds_order();
        }
    }
};

template <int NW, int MT>
__device__ __forceinline__ void clear(f32x4_t (&v)[NW][MT]) {
#pragma unroll
    for (int r = 0; r < NW; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) v[r][t] = f32x4_t{0, 0, 0, 0};
}

// acc += scale * p
template <int MT>
__device__ __forceinline__ void promote(const f32x4_t (&p)[MT], float scale, f32x4_t (&acc)[MT]) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[t][k] = __builtin_fmaf(p[t][k], scale, acc[t][k]);
}

// Blocks in flight.  Loads retire in order, so weights and columns are fetched
// equally far ahead; none of the main loops' loads is conditional, since a load
// that some path skips makes the compiler wait for the ones behind it; and they
// stay where they are written, since the scheduler gathers them at the loop's
// end otherwise.
// One is in the stage and one on its way; two more on their way gain 6% of the
// whole layer where a workgroup's registers are few (one column tile), nothing
// or less elsewhere.
template <int MT>
constexpr int kUpDepth = MT == 1 ? 2 : 1;
constexpr int kDownDepth = 1;

// Runs step(slot, block, whether to fetch block + DEPTH into the slot) for
// blocks 0 ... count - 1.
template <int DEPTH, typename F>
__device__ __forceinline__ void in_flight(int count, F step) {
    int i = 0;
    if constexpr (DEPTH == 1) {
        for (; i + 1 < count; ++i) step(0, i, std::true_type{});
        if (i < count) step(0, i, std::false_type{});
        return;
    }
    for (; i + 2 * DEPTH <= count; i += DEPTH)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) step(d, i + d, std::true_type{});
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
        if (i + d + DEPTH < count) step(d, i + d, std::true_type{});
        else if (i + d < count) step(d, i + d, std::false_type{});
    }
    i += DEPTH;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (i + d < count) step(d, i + d, std::false_type{});
}

// acc += scale * (weight block . column block) over the n 128-K blocks kb0,
// kb0 + step, ...  w, s and cols are uniform; a lane's places in a weight tile are
// w_off and w_off + w_next bytes on, its two in column tile t col[t] bytes.
template <int NW, int NS, int MT, int DEPTH>
__device__ __forceinline__ void products(const uint8_t* (&w)[NW], uint32_t w_off, uint32_t w_next,
                                         const float* (&s)[NS], const uint16_t* cols, const uint32_t (&col)[MT][2],
                                         u32x4_t* stage, int kb0, int n, int step, int lane, f32x4_t (&acc)[NW][MT]) {
    for (int j0 = 0; j0 < n; j0 += 64) {
        const int blocks = min(64, n - j0);
        float sv[NS];                              // lane j: the scale of the jth block
#pragma unroll
        for (int r = 0; r < NS; ++r) sv[r] = s[r][kb0 + (int64_t)(j0 + min(lane, blocks - 1)) * step];
        Block<NW, MT> ring[DEPTH];
        auto load_w = [&](int d, int j) {
            const int64_t k = (kb0 + (int64_t)(j0 + j) * step) * kBlk;
            ring[d].load_w([&](int r, int i) { return w[r] + k + (w_off + i * w_next); });
        };
        auto load_x = [&](int d, int j) {
            const int64_t k = (kb0 + (int64_t)(j0 + j) * step) * kBlk;
            ring[d].load_x([&](int t, int i) { return reinterpret_cast<const char*>(cols + k) + col[t][i]; });
        };
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            load_w(d, min(d, blocks - 1));
            load_x(d, min(d, blocks - 1));
            __builtin_amdgcn_sched_barrier(0);
        }
        in_flight<DEPTH>(blocks, [&](int d, int j, auto more) {
            f32x4_t p[NW][MT];
            ring[d].multiply(stage, lane, p, [&]() { if constexpr (more) load_w(d, j + DEPTH); },
                             [&]() { if constexpr (more) load_x(d, j + DEPTH); });
#pragma unroll
            for (int r = 0; r < NW; ++r)
                promote(p[r], __uint_as_float((uint32_t)__builtin_amdgcn_readlane(
                                  (int)__float_as_uint(sv[r / (NW / NS)]), j)), acc[r]);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
}

// 16 * RT gate rows and the up rows beside them for the tokens list[first ...]
// of an expert, MT tiles of them at most.
template <int PARTS, int RT, int MT, int DEPTH>
__device__ __forceinline__ void up_pass(const MoeArgs& a, int e, int i0, int first, int count,
                                        const int* list, float* sm, int wave, int lane) {
    const int r16 = lane & 15, g = lane >> 4;
    const uint8_t* w[2 * RT];             // gate tiles, then up tiles
    const float* s[2];
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r) {
        const int row = i0 + (r % RT) * kTile + (r / RT) * a.I;
        w[r] = a.w1 + ((int64_t)e * 2 * a.I + row) * a.H;
        s[r / RT] = a.s1 + ((int64_t)e * (2 * a.I / kBlk) + row / kBlk) * (a.H / kBlk);
    }
    // columns past the last token repeat the first one; their sums are not used
    uint32_t xr[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int at = first + 16 * t + 8 * c + (lane >> 3);
            xr[t][c] = 2u * ((uint32_t)(list[at < count ? at : first] / a.topk) * a.H + 8 * (lane & 7));
        }
    f32x4_t acc[2 * RT][MT];
    clear(acc);
    const int KB = a.H / kBlk;
    u32x4_t* stage = reinterpret_cast<u32x4_t*>(sm) + wave * Block<2 * RT, MT>::STAGE;    // the sums come after
    products<2 * RT, 2, MT, DEPTH>(w, (lane >> 3) * a.H + 16 * (lane & 7), 8 * a.H, s, a.x, xr, stage, wave,
                                       (KB - wave + kUpWaves - 1) / kUpWaves, kUpWaves, lane, acc);

    __syncthreads();
    // [wave][gate tiles, up tiles][token][16 rows]
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t)
            *reinterpret_cast<f32x4_t*>(sm + (((wave * 2 * RT + r) * MT + t) * 16 + r16) * 16 + 4 * g) = acc[r][t];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * MT * 256; i += kUpWaves * 64) {
        const int tok = i / (16 * RT), row = i % (16 * RT);
        if (first + tok < count) {
            float v[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                v[r] = 0.0f;
#pragma unroll
                for (int k = 0; k < kUpWaves; ++k)
                    v[r] += sm[((k * 2 * RT + r * RT + row / 16) * MT * 16 + tok) * 16 + row % 16];
            }
            float rest = v[0] / (1.0f + __expf(-v[0])) * v[1];
            uint16_t* dst = a.h + (int64_t)list[first + tok] * a.I + i0 + row;
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

template <int PARTS, int MOST, int RT>
__global__ __launch_bounds__(kUpWaves * 64, 2) void moe_up_kernel(MoeArgs a) {
    constexpr int DEPTH = kUpDepth<MOST>;
    __shared__ uint32_t bitmap[kMoeMaxExperts / 32];
    __shared__ int list[kMoeMaxTokens];               // the rows of h of its tokens
    // the waves' stages, then their sums
    __shared__ __attribute__((aligned(16))) float sm[kUpWaves * (2 * RT * MOST > 2 * (2 * RT + MOST)
                                                                      ? 2 * RT * MOST : 2 * (2 * RT + MOST)) * 256];
    __shared__ int found[2];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = a.I / (kTile * RT);
    const int tile = blockIdx.x % tiles, nth = blockIdx.x / tiles;
    const int pairs = a.T * a.topk;

    for (int64_t i = (int64_t)blockIdx.x * (kUpWaves * 64) + threadIdx.x; i < a.counters;
         i += (int64_t)gridDim.x * (kUpWaves * 64))
        a.arrived[i] = 0;

    // the nth of the experts that are reached
    int* ids = reinterpret_cast<int*>(sm);            // until the sums need it
    static_assert(kGroup == 64, "a wave has a group's tokens in its lanes");
    static_assert(MOST == 1 || sizeof(sm) >= kMoeMaxTokens * kMoeMaxTopk * 4, "the ids fit");
    static_assert(sizeof(sm) >= 16 * kMoeMaxTopk * 4, "those of 16 tokens fit");
    if (threadIdx.x < kMoeMaxExperts / 32) bitmap[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kUpWaves * 64) {
        const int id = a.ids[p];
        ids[p] = id;
        if (id >= 0 && id < a.E) atomicOr(&bitmap[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    if (wave == 0) {
        const uint32_t word = lane < kMoeMaxExperts / 32 ? bitmap[lane] : 0;
        const int c = __builtin_popcount(word);
        int before = c;                               // inclusive prefix over the words
#pragma unroll
        for (int o = 1; o < kMoeMaxExperts / 32; o <<= 1) {
            const int v = __shfl_up(before, o);
            if (lane >= o) before += v;
        }
        const int total = __builtin_amdgcn_readlane(before, kMoeMaxExperts / 32 - 1);
        before -= c;
        const uint64_t holds = __ballot(nth >= before && nth < before + c);
        int e = -1, count = 0;
        if (holds != 0) {                             // uniform
            const int at = __builtin_ctzll(holds);
            uint32_t w = __builtin_amdgcn_readlane(word, at);
            for (int i = __builtin_amdgcn_readlane(before, at); i < nth; ++i) w &= w - 1;
            e = at * 32 + __builtin_ctz(w);
            // its tokens: a token's first slot with it carries the weights of all of them
            for (int t0 = 0; t0 < a.T; t0 += kGroup) {
                const int t = min(t0 + lane, a.T - 1);
                int first = -1, below = 0;
                for (int j = a.topk - 1; j >= 0; --j) {
                    const int id = ids[t * a.topk + j];
                    if (id == e) first = t * a.topk + j;
                    below += id >= 0 && id < e;
                }
                if (t0 + lane >= a.T) first = -1, below = 0;
                const uint64_t have = __ballot(first >= 0);
                const int n = __builtin_popcountll(have), i = __builtin_popcountll(have & ((1ull << lane) - 1));
                if (first >= 0) list[count + i] = first;
                if (tile == 0) {                      // for the second kernel
                    // the group's slots of lower experts: room for all of their entries
#pragma unroll
                    for (int o = 32; o >= 1; o >>= 1) below += __shfl_xor(below, o);
                    if (first >= 0) {
                        float weight = 0.0f;
                        for (int j = 0; j < a.topk; ++j)
                            if (ids[t * a.topk + j] == e) weight += a.weights[t * a.topk + j];
                        a.entries[t0 * a.topk + below + i] = Entry{first, weight};
                    }
                    if (lane == 0) a.reached[t0 / kGroup * a.slots + nth] = Reached{e, below, n};
                }
                count += n;
            }
        }
        if (lane == 0) {
            found[0] = e;
            found[1] = count;
            if (blockIdx.x == 0) *a.reached_count = total;
        }
    }
    __syncthreads();
    const int e = found[0];
    if (e < 0) return;                                // uniform
    const int count = found[1], i0 = tile * kTile * RT;
    for (int first = 0; first < count; first += 16 * MOST) {
        if (count - first <= 16) up_pass<PARTS, RT, 1, DEPTH>(a, e, i0, first, count, list, sm, wave, lane);
        else up_pass<PARTS, RT, MOST, DEPTH>(a, e, i0, first, count, list, sm, wave, lane);
    }
}

// Tokens whose parts fit MOST column tiles, and the tokens of a workgroup.
template <int PARTS, int MOST>
constexpr int kPass = 16 * MOST / PARTS;
constexpr int kWideTiles = 2, kWideColumns = 2;     // where the waves share the columns
template <int MOST>
constexpr int kDownTokens = MOST == 1 ? 16 : kGroup;

// y of a workgroup's TOKENS x ROWS tile from its sums, sum(i) the values 2 i and
// 2 i + 1 of them, and those of the other shares, in order.
template <int PARTS, int TOKENS, int ROWS, typename F>
__device__ __forceinline__ void finish(const MoeArgs& a, int z, int tile, int tokens, int token0, int n0,
                                       int* meet, F sum) {
    auto put_y = [&](int i, float v0, float v1) {
        const int64_t at = (int64_t)(token0 + 2 * i / ROWS) * a.H + n0 + 2 * i % ROWS;
        if constexpr (PARTS == 3) *reinterpret_cast<f32x2_t*>(static_cast<float*>(a.y) + at) = f32x2_t{v0, v1};
        else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.y) + at) = f32x2_to_bf16x2(v0, v1);
    };
    // [tile][group][share][token][rows]
    const int64_t home = ((int64_t)tile * gridDim.y + blockIdx.y) * a.shares;
    uint64_t* parts = reinterpret_cast<uint64_t*>(a.parts + home * (TOKENS * ROWS));
    for (int i = threadIdx.x; i < tokens * ROWS / 2; i += kDownWaves * 64) {
        const f32x2_t v = sum(i);
        if (a.shares == 1) put_y(i, v.x, v.y);
        else
            __hip_atomic_store(parts + z * (TOKENS * ROWS / 2) + i, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (a.shares == 1) return;
    // The share that arrives last adds them up.  Its count is taken after every
    // wave's device-coherent stores have completed, and the parts are read with
    // device-coherent loads after it (the GEMMs' split-K order).
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    int* arrived = a.arrived + tile * gridDim.y + blockIdx.y;
    if (threadIdx.x == 0) *meet = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*meet != a.shares - 1) return;
    for (int i = threadIdx.x; i < tokens * ROWS / 2; i += kDownWaves * 64) {
        f32x2_t v = {0.0f, 0.0f};
        for (int k0 = 0; k0 < a.shares; k0 += 8) {
            uint64_t part[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                part[k] = __hip_atomic_load(parts + min(k0 + k, a.shares - 1) * (TOKENS * ROWS / 2) + i,
                                            __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k0 + k < a.shares) v += __builtin_bit_cast(f32x2_t, part[k]);
        }
        put_y(i, v.x, v.y);
    }
}

// A workgroup's tokens of `entries` and its list of passes, a thread an expert, its
// place by a prefix sum; returns their number.
template <int PASS>
__device__ __forceinline__ int list_passes(const MoeArgs& a, int token0, int tokens, Entry* entries,
                                           uint32_t* passes, int* totals) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // all loads on their way together: a thread's experts before their number is there
    auto load = [&](int nth) { return a.reached[blockIdx.y * a.slots + min(nth, a.slots - 1)]; };
    Reached next = load(threadIdx.x);
    const int reached = *a.reached_count;
    for (int i = threadIdx.x; i < tokens * a.topk; i += kDownWaves * 64) entries[i] = a.entries[token0 * a.topk + i];
    int pass_count = 0;
    for (int base = 0; base < reached; base += kDownWaves * 64) {
        const int nth = base + (int)threadIdx.x;
        Reached r = next;
        if (nth >= reached) r.count = 0;
        next = load(nth + kDownWaves * 64);
        const int n = (r.count + PASS - 1) / PASS;
        int before = n;                                // inclusive prefix in the wave
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(before, o);
            if (lane >= o) before += v;
        }
        if (lane == 63) totals[wave] = before;
        __syncthreads();
        int at = pass_count + before - n;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) {
            if (w < wave) at += totals[w];
            pass_count += totals[w];
        }
        for (int i = 0; i < n; ++i)
            passes[at + i] = r.expert | (r.first + i * PASS) << 10 | min(PASS, r.count - i * PASS) << 20;
        __syncthreads();
    }
    return __builtin_amdgcn_readfirstlane(pass_count);
}

// 16 * RT rows of y for the workgroup's tokens.  The work is a list of passes,
// an expert and up to kPass of its tokens each, of I / 128 K blocks; the waves
// take equal runs of the list's blocks.  A pass's columns are its tokens' first
// parts, then their second ones, ...  A wave's loads run kDownDepth blocks ahead of
// its products and over the ends of passes, so HBM's latency is met once.
template <int PARTS, int MOST, int RT>
__global__ __launch_bounds__(kDownWaves * 64) void moe_down_kernel(MoeArgs a) {
    constexpr int ROWS = RT * kTile, MT = MOST;
    constexpr int TOKENS = kDownTokens<MOST>, PASS = kPass<PARTS, MOST>;
    // a pass: expert | first of `entries` << 10 | tokens << 20
    static_assert(kMoeMaxExperts <= 1024 && kGroup * kMoeMaxTopk <= 1024 && PASS < 2048, "a pass fits a word");
    __shared__ __attribute__((aligned(16))) float slabs[kDownWaves][TOKENS * ROWS];
    __shared__ u32x4_t stages[kDownWaves][Block<RT, MT>::STAGE];
    __shared__ Entry entries[TOKENS * kMoeMaxTopk];
    __shared__ uint32_t passes[TOKENS * kMoeMaxTopk];
    __shared__ int totals[kDownWaves];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int z = blockIdx.x % a.shares, tile = blockIdx.x / a.shares;
    const int n0 = tile * ROWS, token0 = blockIdx.y * TOKENS;
    const int tokens = min(a.T - token0, TOKENS);
    float* slab = slabs[wave];
    for (int i = lane; i < TOKENS * ROWS; i += 64) slab[i] = 0.0f;

    const int pass_count = list_passes<PASS>(a, token0, tokens, entries, passes, totals);
    const int KB = a.I / kBlk;
    const int64_t blocks = (int64_t)pass_count * KB;
    const int share = z * kDownWaves + wave, all = a.shares * kDownWaves;
    const int64_t u0 = blocks * share / all;
    const int count = (int)(blocks * (share + 1) / all - u0);
    const uint32_t w_off = (lane >> 3) * a.I + 16 * (lane & 7);
    u32x4_t* stage = stages[wave];
    if (count > 0) {
        // the loads' place
        int lp = (int)(u0 / KB), lk = (int)(u0 - (int64_t)lp * KB);
        const uint8_t* w;
        const float* s;
        uint32_t col[MT][2];
        auto aim = [&]() {
            const int pass = __builtin_amdgcn_readfirstlane(passes[lp]);
            const int e = pass & 1023, first = pass >> 10 & 1023, n = pass >> 20;
            w = a.w2 + ((int64_t)e * a.H + n0) * a.I;
            s = a.s2 + ((int64_t)e * (a.H / kBlk) + n0 / kBlk) * KB;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // columns past the last repeat the first one; their sums are not used
                    const int c = 16 * t + 8 * i + (lane >> 3), p = c / n;
                    const int pair = entries[first + (p < PARTS ? c - p * n : 0)].pair;
                    col[t][i] = 2u * (((uint32_t)(p < PARTS ? p : 0) * a.T * a.topk + pair) * (uint32_t)a.I +
                                      8 * (lane & 7));
                }
        };
        Block<RT, MT> ring[kDownDepth];
        float scale[kDownDepth];
        auto load_w = [&](int d) {
            ring[d].load_w([&](int r, int i) {
                return w + ((int64_t)(r * kTile + 8 * i) * a.I + lk * kBlk) + w_off;
            });
        };
        auto load_x = [&](int d) {
            ring[d].load_x([&](int t, int i) { return reinterpret_cast<const char*>(a.h + lk * kBlk) + col[t][i]; });
            scale[d] = s[lk];
        };
        auto advance = [&]() {
            if (lk + 1 < KB) ++lk;
            else if (lp + 1 < pass_count) {            // else there is nothing more to fetch
                ++lp;
                lk = 0;
                aim();
            }
        };
        // the products' place
        int up = lp, uk = lk;
        f32x4_t acc[RT][MT];
        // the weighted sums to the slab; a token is in an expert's list once, so no
        // two lanes of a part meet
        auto flush = [&]() {
            const int pass = __builtin_amdgcn_readfirstlane(passes[up]);
            const int first = pass >> 10 & 1023, n = pass >> 20;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int c = 16 * t + r16, part = c / n;
                const Entry en = entries[first + (part < PARTS ? c - part * n : 0)];
                float* at = slab + (en.pair / a.topk - token0) * ROWS + 4 * g;
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    if (part == q)
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            *reinterpret_cast<f32x4_t*>(at + r * kTile) += acc[r][t] * en.weight;
                    wave_lds_order();
                }
            }
        };
        aim();
#pragma unroll
        for (int d = 0; d < kDownDepth; ++d) {
            load_w(d);
            load_x(d);
            advance();
            __builtin_amdgcn_sched_barrier(0);
        }
        clear(acc);
        in_flight<kDownDepth>(count, [&](int d, int i, auto more) {
            f32x4_t p[RT][MT];
            const float sc = scale[d];
            ring[d].multiply(stage, lane, p, [&]() { if constexpr (more) load_w(d); }, [&]() {
                if constexpr (more) {
                    load_x(d);
                    advance();
                }
            });
#pragma unroll
            for (int r = 0; r < RT; ++r) promote(p[r], sc, acc[r]);
            if (++uk == KB || i + 1 == count) {
                flush();
                clear(acc);
                uk = 0;
                ++up;
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    __syncthreads();
    // the waves' slabs in order
    finish<PARTS, TOKENS, ROWS>(a, z, tile, tokens, token0, n0, &totals[0], [&](int i) {
        f32x2_t v = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kDownWaves; ++k) v += *reinterpret_cast<const f32x2_t*>(slabs[k] + 2 * i);
        return v;
    });
}

// The same where columns are many.  The workgroup's waves stand side by side over
// 4 x 16 x RT rows of y and go through the same blocks, so that a column is
// fetched once for all of them (each wave fetches a quarter) and meets them in
// LDS, in two places in turn: one barrier a block.  What a wave has on its way is
// then mostly weights.
template <int PARTS>
__global__ __launch_bounds__(kDownWaves * 64, 2) void moe_down_wide_kernel(MoeArgs a) {
    constexpr int RT = kWideTiles, MT = kWideColumns, WROWS = RT * kTile, ROWS = kDownWaves * WROWS, PITCH = ROWS + 4;
    constexpr int TOKENS = kGroup, PASS = kPass<PARTS, MT>, DEPTH = kDownDepth;
    static_assert(kMoeMaxExperts <= 1024 && kGroup * kMoeMaxTopk <= 1024 && PASS < 2048, "a pass fits a word");
    __shared__ __attribute__((aligned(16))) float slab[TOKENS * PITCH];
    __shared__ u32x4_t weights[kDownWaves][RT * 128], columns[2][MT * 256];
    __shared__ Entry entries[TOKENS * kMoeMaxTopk];
    __shared__ uint32_t passes[TOKENS * kMoeMaxTopk];
    __shared__ int totals[kDownWaves];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int z = blockIdx.x % a.shares, tile = blockIdx.x / a.shares;
    const int n0 = tile * ROWS, row0 = n0 + wave * WROWS, token0 = blockIdx.y * TOKENS;
    const int tokens = min(a.T - token0, TOKENS);
    for (int i = threadIdx.x; i < TOKENS * PITCH; i += kDownWaves * 64) slab[i] = 0.0f;
    const int pass_count = list_passes<PASS>(a, token0, tokens, entries, passes, totals);
    __syncthreads();

    const int KB = a.I / kBlk;
    const int64_t blocks = (int64_t)pass_count * KB;
    const int64_t u0 = blocks * z / a.shares;
    const int count = (int)(blocks * (z + 1) / a.shares - u0);
    const uint32_t w_off = (lane >> 3) * a.I + 16 * (lane & 7);
    u32x4_t* stage = weights[wave];
    const int put = lane ^ (lane >> 3);                                  // line l >> 3, chunk l & 7
    const int line = r16 * 8, turn = lane & 7;
    if (count > 0) {
        // the loads' place
        int lp = (int)(u0 / KB), lk = (int)(u0 - (int64_t)lp * KB);
        const uint8_t* w;
        const float* s;
        // The wave's MT of the block's 4 MT column fetches, of 8 lines each:
        // number q = wave * MT + i is lines 8 (q % 2) ... of tile q / 2 % MT, half q / 2 / MT.
        uint32_t col[MT];
        auto aim = [&]() {
            const int pass = __builtin_amdgcn_readfirstlane(passes[lp]);
            const int e = pass & 1023, first = pass >> 10 & 1023, n = pass >> 20;
            w = a.w2 + ((int64_t)e * a.H + row0) * a.I;
            s = a.s2 + ((int64_t)e * (a.H / kBlk) + row0 / kBlk) * KB;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int q = wave * MT + i;
                // columns past the last repeat the first one; their sums are not used
                const int c = 16 * (q / 2 % MT) + 8 * (q % 2) + (lane >> 3), p = c / n;
                const int pair = entries[first + (p < PARTS ? c - p * n : 0)].pair;
                col[i] = 2u * (((uint32_t)(p < PARTS ? p : 0) * a.T * a.topk + pair) * (uint32_t)a.I +
                               64 * (q / 2 / MT) + 8 * (lane & 7));
            }
        };
        u32x4_t rw[DEPTH][RT][2], rx[DEPTH][MT];
        float scale[DEPTH];
        auto load = [&](int d) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    rw[d][r][i] = *reinterpret_cast<const u32x4_t*>(
                        w + ((int64_t)(r * kTile + 8 * i) * a.I + lk * kBlk) + w_off);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                rx[d][i] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(a.h + lk * kBlk) + col[i]);
            scale[d] = s[lk];
            if (lk + 1 < KB) ++lk;
            else if (lp + 1 < pass_count) {            // else there is nothing more to fetch
                ++lp;
                lk = 0;
                aim();
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // the products' place
        int up = lp, uk = lk;
        f32x4_t acc[RT][MT];
        // the weighted sums to the slab; a token is in an expert's list once, so no
        // two lanes of a part meet
        auto flush = [&]() {
            const int pass = __builtin_amdgcn_readfirstlane(passes[up]);
            const int first = pass >> 10 & 1023, n = pass >> 20;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int c = 16 * t + r16, part = c / n;
                const Entry en = entries[first + (part < PARTS ? c - part * n : 0)];
                float* at = slab + (en.pair / a.topk - token0) * PITCH + wave * WROWS + 4 * g;
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    if (part == q)
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            *reinterpret_cast<f32x4_t*>(at + r * kTile) += acc[r][t] * en.weight;
                    wave_lds_order();
                }
            }
        };
        aim();
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(d);       // past the last block the last one again, or more
        clear(acc);
        in_flight<DEPTH>(count, [&](int d, int i, auto more) {
            u32x4_t* xs = columns[i & 1];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) stage[r * 128 + k * 64 + put] = rw[d][r][k];
#pragma unroll
            for (int k = 0; k < MT; ++k) xs[(wave * MT + k) * 64 + put] = rx[d][k];
            const float sc = scale[d];
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (more) load(d);
            // Every wave's columns are there; those of the other place, which the
            // next block's go to, were read before the barrier behind this one.
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            f32x4_t p[RT][MT];
            clear(p);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4_t v[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) v[r] = stage[r * 128 + line + ((4 * h + g) ^ turn)];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    bf16x8_t f[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        f[t] = __builtin_bit_cast(bf16x8_t, xs[(h * MT + t) * 128 + line + ((2 * g + c) ^ turn)]);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const bf16x8_t m = c ? e4m3x8_to_bf16x8(v[r].z, v[r].w) : e4m3x8_to_bf16x8(v[r].x, v[r].y);
#pragma unroll
                        for (int t = 0; t < MT; ++t) p[r][t] = mfma_bf16(m, f[t], p[r][t]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) promote(p[r], sc, acc[r]);
            if (++uk == KB || i + 1 == count) {
                flush();
                clear(acc);
                uk = 0;
                ++up;
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    __syncthreads();
    finish<PARTS, TOKENS, ROWS>(a, z, tile, tokens, token0, n0, &totals[0], [&](int i) {
        return *reinterpret_cast<const f32x2_t*>(slab + 2 * i / ROWS * PITCH + 2 * i % ROWS);
    });
}
// The second kernel of a call: `shares` workgroups for a tile of `rows` rows and
// `tokens` tokens.  One column tile where no expert can have more; its workgroups
// are small, and 1024 are wanted, else the 512 that are resident: a few more
// follow the others (13 tokens of 6 in 32 experts, 7168 x 2048: 275 us in 672,
// 252 in 448).  A share has 8 blocks of work to be worth its place in the join.
// 32 rows for two column tiles fetch a column half as often, but where that
// leaves half the chip idle 16 do better, in either kernel (64 of 2 in 8, 1024 x
// 512: 16.4 us against 20.0; 17 of 2 in 4, 512 x 512: 12.2 against 14.5).
// With waves that share the columns, a tile has four times the rows, and takes
// four times the shares to fill the chip, up to 16: from 40 tiles on, where 12
// do, that gains (64 of 8 in 64 experts, 7168 x 2048, fp32: 536 us against 612;
// 128 of 8 in 128, 4096 x 1536: 533 against 628), below it loses (48 of 4 in 32,
// 2048 x 1024: 65 against 54; 32 tiles: 0 to 2%).
struct Down {
    bool wide;
    int most, rows, tokens, shares;
};

Down down_of(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I, int parts) {
    const int64_t blocks = std::min(E, T * topk) * (I / kBlk);
    Down d;
    d.most = T * parts <= 16 ? 1 : 2;
    d.tokens = d.most == 1 ? kDownTokens<1> : kDownTokens<2>;
    const int64_t groups = (T + d.tokens - 1) / d.tokens, wide_rows = kDownWaves * kTile * kWideTiles;
    d.wide = d.most == 2 && H / wide_rows * groups >= 40;
    const bool narrow = H / kTile * groups * (blocks / 8) < 1024;
    d.rows = (int)(d.wide ? wide_rows : kTile * (d.most == 1 || narrow ? 1 : 2));
    const int64_t wanted = (d.most == 1 ? 1024 : 512) / (H / d.rows * groups);
    d.shares = (int)std::max<int64_t>(1, std::min({(int64_t)(d.wide ? 16 : 8), wanted, blocks / 8}));
    return d;
}

constexpr int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

// The workspace's pieces, laid out at `base` (sizes alone where it is NULL).
int64_t lay_out(MoeArgs& a, int parts, char* base) {
    const int64_t T = a.T, groups = (T + kGroup - 1) / kGroup, pairs = T * a.topk;
    a.slots = std::min(a.E, a.T * a.topk);
    const Down d = down_of(T, a.topk, a.E, a.H, a.I, parts);
    a.shares = d.shares;
    a.counters = (int)(a.H / d.rows * groups);
    int64_t n = 0;
    auto piece = [&](int64_t bytes) {
        char* at = base + n;
        n += align16(bytes);
        return at;
    };
    a.reached_count = reinterpret_cast<int32_t*>(piece(4));
    a.reached = reinterpret_cast<Reached*>(piece(groups * a.slots * (int64_t)sizeof(Reached)));
    a.entries = reinterpret_cast<Entry*>(piece(pairs * (int64_t)sizeof(Entry)));
    a.arrived = reinterpret_cast<int32_t*>(piece(4ll * a.counters));
    a.h = reinterpret_cast<uint16_t*>(piece(parts * pairs * a.I * 2));
    a.parts = reinterpret_cast<float*>(
        piece(a.shares == 1 ? 0 : 4ll * a.shares * groups * d.tokens * a.H));
    return n;
}

template <int PARTS>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
    // column tiles of a pass: one where no expert can have more, else two, with
    // passes that read the weights again from the caches (four lose 4% of the
    // layer for 64 tokens of 8 in 64 experts and 16% for 256 of 8 in 64)
    const int64_t up_tiles = (int64_t)a.slots * (a.I / kTile);
    const bool narrow = a.T > 16 && up_tiles < 1024;
    const dim3 up_grid((unsigned)(a.T <= 16 || narrow ? up_tiles : up_tiles / 2)), up_block(kUpWaves * 64);
    if (a.T <= 16) hipLaunchKernelGGL((moe_up_kernel<PARTS, 1, 1>), up_grid, up_block, 0, stream, a);
    else if (narrow) hipLaunchKernelGGL((moe_up_kernel<PARTS, 2, 1>), up_grid, up_block, 0, stream, a);
    else hipLaunchKernelGGL((moe_up_kernel<PARTS, 2, 2>), up_grid, up_block, 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const Down d = down_of(a.T, a.topk, a.E, a.H, a.I, PARTS);
    const dim3 grid((unsigned)(a.H / d.rows * d.shares), (unsigned)((a.T + d.tokens - 1) / d.tokens));
    const dim3 block(kDownWaves * 64);
    if (d.wide) hipLaunchKernelGGL((moe_down_wide_kernel<PARTS>), grid, block, 0, stream, a);
    else if (d.most == 1) hipLaunchKernelGGL((moe_down_kernel<PARTS, 1, 1>), grid, block, 0, stream, a);
    else if (d.rows == kTile) hipLaunchKernelGGL((moe_down_kernel<PARTS, 2, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((moe_down_kernel<PARTS, 2, 2>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int64_t moe_few_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I) {
    MoeArgs a{};
    a.T = (int)T; a.topk = (int)topk; a.E = (int)E; a.H = (int)H; a.I = (int)I;
    return std::max(lay_out(a, 2, nullptr), lay_out(a, 3, nullptr));
}

hipError_t launch_moe_few(const MoeFewProblem& p, hipStream_t stream) {
    MoeArgs a{};
    a.x = p.x; a.w1 = p.w1; a.s1 = p.s1; a.w2 = p.w2; a.s2 = p.s2;
    a.ids = p.ids; a.weights = p.weights; a.y = p.y;
    a.T = (int)p.T; a.topk = (int)p.topk; a.E = (int)p.E; a.H = (int)p.H; a.I = (int)p.I;
    lay_out(a, p.out_f32 ? 3 : 2, static_cast<char*>(p.workspace));
    return p.out_f32 ? launch<3>(a, stream) : launch<2>(a, stream);
}

}  // namespace dg
