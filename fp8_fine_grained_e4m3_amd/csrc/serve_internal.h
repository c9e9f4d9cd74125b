// Internal interface between the C-ABI layer (dg_api.cpp) and the kernels of
// the few-token operators: the FP8 key/value cache, tree attention over it and
// the few-token mixture-of-experts layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// A paged FP8 cache: codes [num_pages, H, page_size, D] e4m3, scales
// [num_pages, H, page_size] fp32, for the keys and for the values.
struct KvCache {
    uint8_t* k_codes;
    float* k_sf;
    uint8_t* v_codes;
    float* v_sf;
    int64_t num_pages, H, page_size, D;
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
