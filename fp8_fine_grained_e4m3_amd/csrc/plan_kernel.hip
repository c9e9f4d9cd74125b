// Pages and slots of a paged cache from request lengths, gfx950.
//
// Request b holds held = ceil(c / p) pages of p tokens for its c, and after its length
// changes by a it needs need = ceil(max(c + a, 0) / p).  Pages that it lacks come
// from the pool, a ring of free pages, in the order of the requests:
//   take = max(need - held, 0), served where take = 0 or sum_{b' <= b} take <= free,
//   page j of b (held <= j < need) = ring[(head + sum_{b' < b} take + j - held) mod P].
// Pages that it no longer needs go behind the free ones, in order too.  A new token
// at position q has the slot page * p + q mod p.
//
// Everything hangs on three sums over the requests (pages taken, pages given back,
// tokens), so each workgroup takes these sums itself, 256 or 1024 requests at a time: a
// scan over the lanes and one over the waves.  It then does its share of the rows,
// the new pages and the returned ones of those requests, each found by a binary
// search in LDS; a new page is read from the ring, not from the table that another
// workgroup writes, so one launch does it all.  The ring's places that are read
// (the free ones) and written (those behind them, as far as there are any) are not the
// same ones.
//
// Bound: latency, of the lengths' loads, the scans and a page's or the ring's load, one
// after the other.  Measured, in graphs: 7 requests with a row each, 4.0 us; 256 requests
// with 131072 packed rows, 7.1 us (7.8 in 256 workgroups).  The grid goes by the rows: pages
// that come back beside few rows are one workgroup's work (beside 32 rows, pages of 16: one
// request of 100000, 14 us; 64 of them, 980).
#include "fp8_values.h"
#include "serve_internal.h"

#include <algorithm>

namespace dg {
namespace {

struct PlanArgs {
    int32_t* table;
    const int32_t* ctx;
    const int32_t* add;
    int32_t* ring;
    const int32_t* state;
    int32_t* slots;
    int32_t* positions;
    int32_t* lens;
    int32_t* new_state;
    int B, rows, per_request;             // rows in all; per request where they are padded, else -1
    int max_pages, num_pages, page_shift;
};

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Inclusive sum over the lanes up to each; what passes 2^32 - 1 stays there.
__device__ __forceinline__ uint32_t sum_sat_up_to_lane(uint32_t v) {
    v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));   // row_shr:1
    v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));   // row_shr:2
    v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));   // row_shr:4
    v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));   // row_shr:8
    v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));   // row_bcast:15 into rows 1 and 3
    v = add_sat(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));   // row_bcast:31 into rows 2 and 3
    return v;
}

// The first of n ascending sums that is above i (there is one).
__device__ __forceinline__ int first_above(const uint32_t* sums, int n, uint32_t i) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (sums[lo + half - 1] <= i) lo += half;
        n -= half;
    }
    return lo;
}

// A place of the ring, up to two rounds past its end.
__device__ __forceinline__ uint32_t in_ring(uint32_t i, uint32_t P) {
    i = i >= 2 * P ? i - 2 * P : i;
    return i >= P ? i - P : i;
}

struct Lengths {
    int c, held, need;
    uint32_t rows;
    bool fits;                            // the table and a padded row have the room
};

__device__ __forceinline__ Lengths lengths_of(const PlanArgs& a, int b) {
    const int most = a.max_pages << a.page_shift, round = (1 << a.page_shift) - 1;
    Lengths x;
    x.c = min(max(a.ctx[b], 0), most);
    const int add = a.add[b];
    const int64_t after = max((int64_t)x.c + add, (int64_t)0);
    x.fits = after <= most && (a.per_request < 0 || add <= a.per_request);
    x.held = (x.c + round) >> a.page_shift;
    x.need = x.fits ? (int)((after + round) >> a.page_shift) : x.held;
    x.rows = (uint32_t)max(a.per_request >= 0 ? min(add, a.per_request) : add, 0);
    return x;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv_cache_plan_kernel(PlanArgs a) {
    constexpr int WAVES = THREADS / 64;
    // of the chunk's requests: sums up to each, and what the rows have to know
    __shared__ uint32_t sm_take[THREADS], sm_give[THREADS], sm_rows[THREADS];
    __shared__ int sm_ctx[THREADS], sm_held[THREADS], sm_need[THREADS];
    __shared__ bool sm_served[THREADS];
    __shared__ uint32_t sm_wave[3][WAVES];
    __shared__ uint32_t sm_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t P = (uint32_t)a.num_pages;
    const uint32_t head = (uint32_t)uniform_input(a.state) % P;
    const uint32_t free = (uint32_t)min(max(uniform_input(a.state + 1), 0), a.num_pages);
    const uint32_t first = blockIdx.x * THREADS + tid, step = gridDim.x * THREADS;
    uint32_t taken = 0, given = 0, tokens = 0;         // of the requests before the chunk
    if (tid == 0) sm_last = 0;                         // pages that the served requests take
    for (int base = 0, chunk = 0; base < a.B; base += THREADS, ++chunk) {
        const int n = min(THREADS, a.B - base);
        Lengths x = {0, 0, 0, 0, true};
        if (tid < n) x = lengths_of(a, base + tid);
        const uint32_t own[3] = {(uint32_t)max(x.need - x.held, 0), (uint32_t)max(x.held - x.need, 0), x.rows};
        uint32_t upto[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            upto[k] = sum_sat_up_to_lane(own[k]);
            if (lane == 63) sm_wave[k][wave] = upto[k];
        }
        __syncthreads();
        const uint32_t before[3] = {taken, given, tokens};
        uint32_t all[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t w = sum_sat_up_to_lane(lane < WAVES ? sm_wave[k][lane] : 0);
            all[k] = add_sat(before[k], (uint32_t)__builtin_amdgcn_readlane(w, WAVES - 1));
            const uint32_t earlier = wave > 0 ? (uint32_t)__builtin_amdgcn_readlane(w, wave - 1) : 0;
            upto[k] = add_sat(before[k], add_sat(upto[k], earlier));
        }
        const bool served = x.fits && (own[0] == 0 || upto[0] <= free);
        sm_take[tid] = upto[0];
        sm_give[tid] = upto[1];
        sm_rows[tid] = upto[2];
        sm_ctx[tid] = x.c;
        sm_held[tid] = x.held;
        sm_need[tid] = x.need;
        sm_served[tid] = served;
        if (tid < n) {
            if (own[0] > 0 && served) atomicMax(&sm_last, upto[0]);
            if ((uint32_t)chunk % gridDim.x == blockIdx.x)
                a.lens[base + tid] = served ? max(x.c + a.add[base + tid], 0) : x.c;
        }
        __syncthreads();

        auto slot_of = [&](int i, int q) {             // position q of the chunk's request i
            if (!sm_served[i]) return -1;
            const int j = q >> a.page_shift, held = sm_held[i];
            int page;
            if (j < held) {
                page = a.table[(int64_t)(base + i) * a.max_pages + j];
            } else {
                const uint32_t taken_before = sm_take[i] - (uint32_t)(sm_need[i] - held);
                page = a.ring[in_ring(head + taken_before + (uint32_t)(j - held), P)];
            }
            return page >= 0 && page < a.num_pages ? (page << a.page_shift) + (q & ((1 << a.page_shift) - 1)) : -1;
        };
        if (a.per_request >= 0) {
            const uint32_t N = (uint32_t)a.per_request, end = (uint32_t)(base + n) * N;
            for (uint32_t r = (uint32_t)base * N + first; r < end; r += step) {
                const int i = (int)(r / N) - base;
                const uint32_t at = r % N, own_rows = sm_rows[i] - (i > 0 ? sm_rows[i - 1] : tokens);
                const bool live = at < own_rows;
                a.slots[r] = live ? slot_of(i, sm_ctx[i] + (int)at) : -1;
                a.positions[r] = live ? sm_ctx[i] + (int)at : 0;
            }
        } else {
            const uint32_t end = min(all[2], (uint32_t)a.rows);
            for (uint64_t r = (uint64_t)tokens + first; r < end; r += step) {
                const int i = first_above(sm_rows, n, (uint32_t)r);
                const int q = sm_ctx[i] + (int)((uint32_t)r - (i > 0 ? sm_rows[i - 1] : tokens));
                a.slots[r] = slot_of(i, q);
                a.positions[r] = q;
            }
        }
        // new pages: the served requests' are the first `free` of all
        for (uint64_t k = (uint64_t)taken + first; k < min(all[0], free); k += step) {
            const int i = first_above(sm_take, n, (uint32_t)k);
            if (!sm_served[i]) continue;
            const int j = sm_need[i] - (int)(sm_take[i] - (uint32_t)k);
            a.table[(int64_t)(base + i) * a.max_pages + j] = a.ring[in_ring(head + (uint32_t)k, P)];
        }
        for (uint64_t k = (uint64_t)given + first; k < min(all[1], P - free); k += step) {
            const int i = first_above(sm_give, n, (uint32_t)k);
            const int j = sm_held[i] - (int)(sm_give[i] - (uint32_t)k);
            a.ring[in_ring(head + free + (uint32_t)k, P)] = a.table[(int64_t)(base + i) * a.max_pages + j];
        }
        taken = all[0];
        given = all[1];
        tokens = all[2];
        __syncthreads();                               // before the next chunk's sums
    }
    // rows behind the last token
    if (a.per_request < 0)
        for (uint64_t r = (uint64_t)tokens + first; r < (uint32_t)a.rows; r += step) {
            a.slots[r] = -1;
            a.positions[r] = 0;
        }
    if (blockIdx.x == 0 && tid == 0) {
        const uint32_t last = a.B > 0 ? sm_last : 0;
        a.new_state[0] = (int)in_ring(head + last, P);
        a.new_state[1] = (int)(free - last + min(given, P - free));
    }
}

}  // namespace

hipError_t launch_kv_cache_plan(const KvPlan& p, hipStream_t stream) {
    PlanArgs a;
    a.table = p.page_table; a.ctx = p.context_lens; a.add = p.add_lens;
    a.ring = p.pool_pages; a.state = p.pool_state;
    a.slots = p.slots; a.positions = p.positions; a.lens = p.new_lens; a.new_state = p.new_state;
    a.B = (int)p.B;
    a.rows = (int)(p.padded ? p.B * p.rows : p.rows);
    a.per_request = p.padded ? (int)p.rows : -1;
    a.max_pages = (int)p.max_pages; a.num_pages = (int)p.num_pages;
    a.page_shift = __builtin_ctzll((unsigned long long)p.page_size);
    const int threads = p.B <= 256 ? 256 : 1024;
    const int64_t groups = std::min<int64_t>(1024, std::max<int64_t>(1, (a.rows + threads - 1) / threads));
    if (threads == 256) hipLaunchKernelGGL((kv_cache_plan_kernel<256>), dim3((unsigned)groups), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kv_cache_plan_kernel<1024>), dim3((unsigned)groups), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dg
