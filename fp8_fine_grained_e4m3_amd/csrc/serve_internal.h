// Internal interface between the C-ABI layer (dg_api.cpp) and the kernels of
// the few-token operators: the FP8 key/value cache, tree attention over it, the
// few-token mixture-of-experts layer, and the plan of a cache's pages and slots.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// A paged cache, for the keys and for the values: FP8, codes [num_pages, H, page_size,
// D] e4m3, scales [num_pages, H, page_size] fp32; or FP4, codes [num_pages, H,
// page_size, D / 2], two e2m1 a byte, scales [num_pages, H, page_size, D / 32] E8M0.
struct KvCache {
    uint8_t* k_codes;
    void* k_sf;
    uint8_t* v_codes;
    void* v_sf;
    int64_t num_pages, H, page_size, D;
    bool fp4;

    int64_t code_bytes() const { return num_pages * H * page_size * (fp4 ? D / 2 : D); }
    int64_t sf_bytes() const { return num_pages * H * page_size * (fp4 ? D / 32 : 4); }
};

// slots [T]: page * page_size + offset of each row; others are skipped (write)
// or read as zeros (read).  Strides in elements between tokens; heads and the
// D values of a head are dense.
struct KvCopy {
    KvCache cache;
    const int32_t* slots;
    void* k;                // const for a write
    void* v;
    int64_t k_stride, v_stride, T;
    bool f32;               // rows are fp32, else bf16
};
hipError_t launch_kv_cache_write(const KvCopy& p, hipStream_t stream);
hipError_t launch_kv_cache_read(const KvCopy& p, hipStream_t stream);
hipError_t launch_kv4_cache_write(const KvCopy& p, hipStream_t stream);
hipError_t launch_kv4_cache_read(const KvCopy& p, hipStream_t stream);

// Pages and slots from request lengths (dg_kv_cache_plan).
struct KvPlan {
    int32_t* page_table;           // [B, max_pages]
    const int32_t* context_lens;   // [B]
    const int32_t* add_lens;       // [B]
    int32_t* pool_pages;           // [num_pages], a ring
    const int32_t* pool_state;     // [2]: first free page's place, free pages
    int32_t* slots;                // [rows], or [B, rows] where padded
    int32_t* positions;
    int32_t* new_lens;             // [B]
    int32_t* new_state;            // [2]
    int64_t B, rows, max_pages, num_pages, page_size;
    bool padded;
};
hipError_t launch_kv_cache_plan(const KvPlan& p, hipStream_t stream);

// Norms of queries [0] and keys [1] with the rotation, or (backward) their gradients.
struct NormRope {
    const void* x[2];              // [T, heads, D], strides in elements between tokens
    const void* dz[2];             // backward
    void* out[2];                  // z, or dx
    int64_t x_stride[2], dz_stride[2], out_stride[2];
    const void* w[2];              // [D] or NULL
    float* dw[2];                  // backward, [D] or NULL
    const int32_t* positions;      // [T]
    const float* inv_freq;         // [R / 2]
    float eps;
    int64_t T, Hq, H, D, R;
    bool f32, w_f32, neighbours, backward;
    void* workspace;               // backward with a dw
};
int64_t norm_rope_workspace_bytes(int64_t T, int64_t Hq, int64_t H, int64_t D);
hipError_t launch_norm_rope(const NormRope& p, hipStream_t stream);

struct TreeAttnProblem {
    KvCache cache;
    const uint16_t* q;             // bf16 [B, N, Hq, D], q_stride elements between tokens
    int64_t q_stride;
    const int32_t* page_table;     // [B, max_pages]
    const int32_t* context_lens;   // [B]
    const int32_t* tree_lens;      // [B] or NULL (= N)
    const uint64_t* tree_mask;     // [B, N, ceil(N/64)] or NULL (= chain)
    uint16_t* o;                   // bf16 [B, N, Hq, D]
    float* lse;                    // [B, N, Hq]
    float scale;
    int64_t B, N, Hq, max_pages;
    void* workspace;
};
// Bytes of workspace, a function of the sizes alone (no HIP call).
int64_t tree_attn_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D,
                                  int64_t max_pages, int64_t page_size);
hipError_t launch_tree_attn(const TreeAttnProblem& p, hipStream_t stream);
// The same over the FP4 cache.
int64_t tree_attn4_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D,
                                   int64_t max_pages, int64_t page_size);
hipError_t launch_tree_attn4(const TreeAttnProblem& p, hipStream_t stream);

constexpr int64_t kMoeMaxTokens = 256;
constexpr int64_t kMoeMaxTopk = 16;
constexpr int64_t kMoeMaxExperts = 1024;

struct MoeFewProblem {
    const uint16_t* x;        // bf16 [T, H]
    const uint8_t* w1;        // e4m3 [E, 2I, H]: I gate rows, then I up rows
    const float* s1;          // [E, 2I/128, H/128]
    const uint8_t* w2;        // e4m3 [E, H, I]
    const float* s2;          // [E, H/128, I/128]
    const int32_t* ids;       // [T, topk]
    const float* weights;     // [T, topk]
    void* y;                  // [T, H]
    bool out_f32;
    int64_t T, topk, E, H, I;
    void* workspace;
};
int64_t moe_few_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I);
hipError_t launch_moe_few(const MoeFewProblem& p, hipStream_t stream);

}  // namespace dg
