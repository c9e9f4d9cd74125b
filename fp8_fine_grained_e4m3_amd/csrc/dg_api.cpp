// C-ABI layer: argument validation (before any HIP call), device checks,
// CU-count cap, error reporting, and dispatch to the kernels.
#include "../../include/dg.h"
#include "dg_internal.h"
#include "serve_internal.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

namespace {

thread_local std::string g_last_error;

dg_status fail(dg_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

dg_status ok() {
    g_last_error.clear();
    return DG_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// c must be NULL, equal to d, or not overlap [d, d + bytes).
bool alias_ok(const void* c, const void* d, int64_t bytes) {
    if (c == nullptr || c == d) return true;
    const uintptr_t c0 = reinterpret_cast<uintptr_t>(c), d0 = reinterpret_cast<uintptr_t>(d);
    return c0 + (uintptr_t)bytes <= d0 || d0 + (uintptr_t)bytes <= c0;
}

#define REQUIRE(cond, ...)                                   \
    do {                                                     \
        if (!(cond)) return fail(DG_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)

#define REQUIRE_PTR(p, align)                                                         \
    do {                                                                              \
        if ((p) == nullptr) return fail(DG_ERR_INVALID_ARG, "%s is NULL", #p);        \
        if (!aligned((p), (align)))                                                   \
            return fail(DG_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p, (int)(align)); \
    } while (0)

constexpr int64_t kOffsetLimit = INT_MAX;   // kernels index one matrix with 32-bit offsets

// ---- device state -------------------------------------------------------------

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool probed = false;
    bool gfx950 = false;
    int cus = 0;
    char arch[64] = {0};
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mutex;
std::atomic<int> g_cu_cap{0};   // 0 = use every CU; process-wide, set from any thread

dg_status current_device(int& dev, DeviceInfo& info) {
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(DG_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(DG_ERR_UNSUPPORTED, "device index %d", dev);
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    DeviceInfo& d = g_dev[dev];
    if (!d.probed) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess)
            return fail(DG_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
        snprintf(d.arch, sizeof d.arch, "%s", prop.gcnArchName);
        d.gfx950 = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
        d.cus = prop.multiProcessorCount;
        d.probed = true;
    }
    info = d;
    if (!info.gfx950)
        return fail(DG_ERR_UNSUPPORTED, "device %d is %s; this library is built for gfx950", dev,
                    info.arch);
    return DG_OK;
}

int cu_cap_for(const DeviceInfo& info) {
    const int cap = g_cu_cap.load(std::memory_order_relaxed);
    return (cap > 0 && cap < info.cus) ? cap : info.cus;
}

bool print_configs() {
    // read once; the initialisation of a function-local static is thread-safe
    static const bool v = [] {
        const char* s = getenv("DG_PRINT_CONFIGS");
        return s != nullptr && s[0] == '1';
    }();
    return v;
}

dg_status run_tn(const dg::TnProblem& p, void* stream) {
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    if (print_configs()) fprintf(stderr, "[dg] %s\n", dg::describe_tn_config(p));
    hipError_t e = dg::launch_tn(p, cu_cap_for(info), reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

dg_status run_nt(dg::NtProblem p, void* stream) {
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    if (print_configs()) fprintf(stderr, "[dg] %s\n", dg::describe_nt_config(p));
    hipError_t e = dg::launch_nt(p, cu_cap_for(info), reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

// [p0, p0 + n0) and [p1, p1 + n1) do not overlap
bool disjoint(const void* p0, int64_t n0, const void* p1, int64_t n1) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(p0), a1 = reinterpret_cast<uintptr_t>(p1);
    return a0 + (uintptr_t)n0 <= a1 || a1 + (uintptr_t)n1 <= a0;
}

// The three NT forms take either fp32 scales or packed UE8M0 words; both are
// 4-byte elements, passed through as raw pointers.
// noalloc: the split-K workspace is the library's static scratch instead of
// the caller's (workspace / workspace_bytes are ignored).
dg_status gemm_nt(const uint8_t* a, const void* sfa_, const uint8_t* b, const void* sfb_,
                  const void* c, void* d, dg_dtype d_dtype, int64_t M, int64_t N, int64_t K,
                  void* workspace, int64_t workspace_bytes, bool ue8m0, void* stream,
                  bool noalloc = false) {
    const float* sfa = static_cast<const float*>(sfa_);
    const float* sfb = static_cast<const float*>(sfb_);
    REQUIRE(M >= 0 && N >= 0 && K >= 0, "negative size (M=%lld N=%lld K=%lld)", (long long)M,
            (long long)N, (long long)K);
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(N % 16 == 0, "N=%lld is not a multiple of 16", (long long)N);
    REQUIRE(d_dtype == DG_BF16 || d_dtype == DG_F32, "d_dtype must be DG_BF16 or DG_F32");
    if (M == 0 || N == 0) return ok();
    REQUIRE_PTR(d, 16);
    if (c) REQUIRE_PTR(c, 16);
    if (K > 0) {   // with K == 0 the operands are empty: D = C (or 0)
        REQUIRE_PTR(a, 16);
        REQUIRE_PTR(b, 16);
        REQUIRE_PTR(sfa, 16);
        REQUIRE_PTR(sfb, 16);
    }
    REQUIRE(M <= kOffsetLimit / (K > 0 ? K : 1) && N <= kOffsetLimit / (K > 0 ? K : 1),
            "M*K and N*K must stay below 2^31");
    REQUIRE(M <= INT_MAX && N <= INT_MAX, "size too large");
    // work units: 64 x 64 tiles (the smallest) times up to 8 K splits
    REQUIRE(((M + 63) / 64) * ((N + 63) / 64) <= INT_MAX / 8, "too many tiles");
    const int64_t dbytes = M * N * (d_dtype == DG_F32 ? 4 : 2);
    REQUIRE(alias_ok(c, d, dbytes), "c overlaps d without being equal to it");
    const int64_t need = dg::nt_dense_workspace_bytes(M, N, K);
    if (noalloc) {
        if (need > dg::nt_noalloc_scratch_bytes())
            return fail(DG_ERR_UNSUPPORTED,
                        "this shape needs %lld bytes of split-K scratch; the static scratch "
                        "holds %lld", (long long)need, (long long)dg::nt_noalloc_scratch_bytes());
        workspace = nullptr;
        workspace_bytes = 0;
    }
    REQUIRE(workspace_bytes >= 0, "workspace_bytes=%lld is negative", (long long)workspace_bytes);
    if (need > 0 && !noalloc) {
        REQUIRE(workspace != nullptr,
                "this shape splits K and needs a workspace of %lld bytes "
                "(dg_fp8_gemm_nt_workspace_bytes); workspace is NULL", (long long)need);
        REQUIRE_PTR(workspace, 16);
        REQUIRE(workspace_bytes >= need, "workspace_bytes=%lld < %lld needed for this shape",
                (long long)workspace_bytes, (long long)need);
        const int64_t KB = K / 128, sf_w = ue8m0 ? (KB + 3) / 4 : KB;
        const int64_t sfb_n = ue8m0 ? sf_w * N : ((N + 127) / 128) * KB;
        REQUIRE(disjoint(workspace, need, d, dbytes) && (c == nullptr || disjoint(workspace, need, c, dbytes)) &&
                    disjoint(workspace, need, a, M * K) && disjoint(workspace, need, b, N * K) &&
                    disjoint(workspace, need, sfa, 4 * sf_w * M) && disjoint(workspace, need, sfb, 4 * sfb_n),
                "workspace overlaps an operand or the output");
    }
    dg::NtProblem p{};
    p.form = dg::kDense;
    p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.c = c; p.d = d;
    p.rows = M; p.N = N; p.K = K; p.G = 1;
    p.out_f32 = d_dtype == DG_F32;
    p.ue8m0 = ue8m0;
    if (noalloc && need > 0) {
        // after host validation: the device check, then this device's scratch
        int dev = 0;
        DeviceInfo info;
        dg_status st = current_device(dev, info);
        if (st != DG_OK) return st;
        hipError_t e = dg::nt_noalloc_scratch(&workspace);
        if (e != hipSuccess)
            return fail(DG_ERR_HIP, "static scratch lookup: %s", hipGetErrorString(e));
        workspace_bytes = dg::nt_noalloc_scratch_bytes();
    }
    p.workspace = need > 0 ? workspace : nullptr;
    p.workspace_bytes = need > 0 ? workspace_bytes : 0;
    return run_nt(p, stream);
}

dg_status gemm_nt_contiguous(const uint8_t* a, const void* sfa_, const uint8_t* b,
                             const void* sfb_, const int32_t* m_indices, void* d, int64_t M_tot,
                             int64_t N, int64_t K, int64_t G, bool ue8m0, void* stream) {
    const float* sfa = static_cast<const float*>(sfa_);
    const float* sfb = static_cast<const float*>(sfb_);
    REQUIRE(M_tot >= 0 && N >= 0 && K >= 0, "negative size");
    REQUIRE(G >= 1, "G=%lld must be >= 1", (long long)G);
    REQUIRE(M_tot % 128 == 0, "M_tot=%lld is not a multiple of 128 (the contiguous-layout alignment)",
            (long long)M_tot);
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(N % 16 == 0, "N=%lld is not a multiple of 16", (long long)N);
    if (M_tot == 0 || N == 0) return ok();
    REQUIRE_PTR(a, 16);
    REQUIRE_PTR(b, 16);
    REQUIRE_PTR(d, 16);
    REQUIRE_PTR(sfa, 16);
    REQUIRE_PTR(sfb, 16);
    REQUIRE_PTR(m_indices, 16);
    REQUIRE(M_tot <= kOffsetLimit / (K > 0 ? K : 1) && N <= kOffsetLimit / (K > 0 ? K : 1),
            "M_tot*K and N*K must stay below 2^31");
    REQUIRE(G <= INT_MAX, "G too large");
    dg::NtProblem p{};
    p.form = dg::kContiguous;
    p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.c = nullptr; p.d = d;
    p.m_indices = m_indices;
    p.rows = M_tot; p.N = N; p.K = K; p.G = G;
    p.out_f32 = false;
    p.ue8m0 = ue8m0;
    return run_nt(p, stream);
}

dg_status gemm_nt_masked(const uint8_t* a, const void* sfa_, const uint8_t* b, const void* sfb_,
                         const int32_t* masked_m, void* d, int64_t G, int64_t M_max, int64_t N,
                         int64_t K, bool ue8m0, void* stream) {
    const float* sfa = static_cast<const float*>(sfa_);
    const float* sfb = static_cast<const float*>(sfb_);
    REQUIRE(G >= 0 && M_max >= 0 && N >= 0 && K >= 0, "negative size");
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(N % 16 == 0, "N=%lld is not a multiple of 16", (long long)N);
    if (G == 0 || M_max == 0 || N == 0) return ok();
    REQUIRE_PTR(a, 16);
    REQUIRE_PTR(b, 16);
    REQUIRE_PTR(d, 16);
    REQUIRE_PTR(sfa, 16);
    REQUIRE_PTR(sfb, 16);
    REQUIRE_PTR(masked_m, 16);
    REQUIRE(M_max <= kOffsetLimit / (K > 0 ? K : 1) && N <= kOffsetLimit / (K > 0 ? K : 1),
            "M_max*K and N*K must stay below 2^31");
    // bound for the smallest tile (64 x 64) any configuration uses (G first, so
    // the product below cannot overflow)
    REQUIRE(G <= INT_MAX, "G too large");
    REQUIRE(G * ((M_max + 63) / 64) * ((N + 63) / 64) <= INT_MAX, "too many tiles");
    dg::NtProblem p{};
    p.form = dg::kMasked;
    p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.c = nullptr; p.d = d;
    p.masked_m = masked_m;
    p.rows = M_max; p.N = N; p.K = K; p.G = G;
    p.out_f32 = false;
    p.ue8m0 = ue8m0;
    return run_nt(p, stream);
}

}  // namespace

extern "C" {

dg_status dg_fp8_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                         const void* c, void* d, dg_dtype d_dtype, int64_t M, int64_t N,
                         int64_t K, void* workspace, int64_t workspace_bytes, void* stream) {
    return gemm_nt(a, sfa, b, sfb, c, d, d_dtype, M, N, K, workspace, workspace_bytes, false,
                   stream);
}

dg_status dg_fp8_gemm_nt_noalloc(const uint8_t* a, const float* sfa, const uint8_t* b,
                                 const float* sfb, const void* c, void* d, dg_dtype d_dtype,
                                 int64_t M, int64_t N, int64_t K, void* stream) {
    return gemm_nt(a, sfa, b, sfb, c, d, d_dtype, M, N, K, nullptr, 0, false, stream, true);
}

int64_t dg_fp8_gemm_nt_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || K % 128 != 0 || N % 16 != 0) return 0;
    if (M > kOffsetLimit / K || N > kOffsetLimit / K) return 0;
    return dg::nt_dense_workspace_bytes(M, N, K);
}

dg_status dg_m_grouped_fp8_gemm_nt_contiguous(const uint8_t* a, const float* sfa,
                                              const uint8_t* b, const float* sfb,
                                              const int32_t* m_indices, void* d, int64_t M_tot,
                                              int64_t N, int64_t K, int64_t G, void* stream) {
    return gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d, M_tot, N, K, G, false, stream);
}

dg_status dg_m_grouped_fp8_gemm_nt_masked(const uint8_t* a, const float* sfa, const uint8_t* b,
                                          const float* sfb, const int32_t* masked_m, void* d,
                                          int64_t G, int64_t M_max, int64_t N, int64_t K,
                                          void* stream) {
    return gemm_nt_masked(a, sfa, b, sfb, masked_m, d, G, M_max, N, K, false, stream);
}

dg_status dg_fp8_gemm_nt_ue8m0(const uint8_t* a, const int32_t* sfa, const uint8_t* b,
                               const int32_t* sfb, const void* c, void* d, dg_dtype d_dtype,
                               int64_t M, int64_t N, int64_t K, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    return gemm_nt(a, sfa, b, sfb, c, d, d_dtype, M, N, K, workspace, workspace_bytes, true,
                   stream);
}

dg_status dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0(const uint8_t* a, const int32_t* sfa,
                                                    const uint8_t* b, const int32_t* sfb,
                                                    const int32_t* m_indices, void* d,
                                                    int64_t M_tot, int64_t N, int64_t K,
                                                    int64_t G, void* stream) {
    return gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d, M_tot, N, K, G, true, stream);
}

dg_status dg_m_grouped_fp8_gemm_nt_masked_ue8m0(const uint8_t* a, const int32_t* sfa,
                                                const uint8_t* b, const int32_t* sfb,
                                                const int32_t* masked_m, void* d, int64_t G,
                                                int64_t M_max, int64_t N, int64_t K,
                                                void* stream) {
    return gemm_nt_masked(a, sfa, b, sfb, masked_m, d, G, M_max, N, K, true, stream);
}

dg_status dg_pack_ue8m0_scales(const float* sf, int per_block, int32_t* packed, int64_t G,
                               int64_t MN, int64_t K, void* stream) {
    REQUIRE(G >= 0 && MN >= 0 && K >= 0, "negative size (G=%lld MN=%lld K=%lld)", (long long)G,
            (long long)MN, (long long)K);
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(per_block == 0 || per_block == 1, "per_block must be 0 or 1");
    if (G == 0 || MN == 0 || K == 0) return ok();
    REQUIRE_PTR(sf, 16);
    REQUIRE_PTR(packed, 16);
    const int64_t kb = K / 128, k4 = (kb + 3) / 4;
    REQUIRE(MN <= INT_MAX && G <= kOffsetLimit / k4 && G * k4 <= kOffsetLimit / MN,
            "G*ceil(K/512)*MN must stay below 2^31");
    const int64_t sf_count = per_block ? G * ((MN + 127) / 128) * kb : G * kb * MN;
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(sf), p0 = reinterpret_cast<uintptr_t>(packed);
    REQUIRE(s0 + (uintptr_t)(sf_count * 4) <= p0 || p0 + (uintptr_t)(G * k4 * MN * 4) <= s0,
            "sf and packed must not overlap");
    dg::PackProblem p{};
    p.sf = sf; p.per_block = per_block != 0; p.packed = packed;
    p.G = G; p.MN = MN; p.KB = kb;
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_pack_ue8m0(p, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

static dg_status k_grouped_tn(const uint8_t* a, const void* sfa, const uint8_t* b,
                              const void* sfb, const int32_t* k_sizes_host, const float* c,
                              float* d, int64_t G, int64_t M, int64_t N, int64_t K_tot,
                              bool ue8m0, void* stream);

dg_status dg_k_grouped_fp8_gemm_tn_contiguous(const uint8_t* a, const float* sfa,
                                              const uint8_t* b, const float* sfb,
                                              const int32_t* k_sizes_host, const float* c,
                                              float* d, int64_t G, int64_t M, int64_t N,
                                              int64_t K_tot, void* stream) {
    return k_grouped_tn(a, sfa, b, sfb, k_sizes_host, c, d, G, M, N, K_tot, false, stream);
}

dg_status dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0(const uint8_t* a, const int32_t* sfa,
                                                    const uint8_t* b, const int32_t* sfb,
                                                    const int32_t* k_sizes_host, const float* c,
                                                    float* d, int64_t G, int64_t M, int64_t N,
                                                    int64_t K_tot, void* stream) {
    return k_grouped_tn(a, sfa, b, sfb, k_sizes_host, c, d, G, M, N, K_tot, true, stream);
}

dg_status dg_pack_ue8m0_scales_k_grouped(const float* sf, const int32_t* k_sizes_host,
                                         int32_t* packed, int64_t G, int64_t MN, int64_t K_tot,
                                         void* stream) {
    REQUIRE(G >= 1 && G <= dg::kMaxTnGroups, "G=%lld must be in [1, %d]", (long long)G,
            dg::kMaxTnGroups);
    REQUIRE(MN >= 0 && K_tot >= 0, "negative size");
    REQUIRE(k_sizes_host != nullptr, "k_sizes_host is NULL");
    int64_t total = 0, words = 0;
    for (int64_t g = 0; g < G; ++g) {
        const int64_t kg = k_sizes_host[g];
        REQUIRE(kg >= 0 && kg % 128 == 0, "k_sizes_host[%lld]=%lld must be >= 0 and a multiple of 128",
                (long long)g, (long long)kg);
        total += kg;
        words += (kg / 128 + 3) / 4;
    }
    REQUIRE(total == K_tot, "sum of k_sizes_host (%lld) != K_tot (%lld)", (long long)total,
            (long long)K_tot);
    if (MN == 0 || words == 0) return ok();
    REQUIRE_PTR(sf, 16);
    REQUIRE_PTR(packed, 16);
    // the kernel's 32-bit column index runs up to one 256-thread block past MN
    REQUIRE(MN <= INT_MAX - 256, "MN=%lld too large", (long long)MN);
    REQUIRE(words <= 65535, "too many packed word rows");
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(sf), p0 = reinterpret_cast<uintptr_t>(packed);
    REQUIRE(s0 + (uintptr_t)((K_tot / 128) * MN * 4) <= p0 || p0 + (uintptr_t)(words * MN * 4) <= s0,
            "sf and packed must not overlap");
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_pack_ue8m0_k_grouped(sf, k_sizes_host, G, MN, packed,
                                                   reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

static dg_status k_grouped_tn(const uint8_t* a, const void* sfa_, const uint8_t* b,
                              const void* sfb_, const int32_t* k_sizes_host, const float* c,
                              float* d, int64_t G, int64_t M, int64_t N, int64_t K_tot,
                              bool ue8m0, void* stream) {
    const float* sfa = static_cast<const float*>(sfa_);
    const float* sfb = static_cast<const float*>(sfb_);
    REQUIRE(M >= 0 && N >= 0 && K_tot >= 0, "negative size");
    REQUIRE(G >= 1 && G <= dg::kMaxTnGroups, "G=%lld must be in [1, %d]", (long long)G,
            dg::kMaxTnGroups);
    REQUIRE(M % 16 == 0, "M=%lld is not a multiple of 16", (long long)M);
    REQUIRE(N % 16 == 0, "N=%lld is not a multiple of 16", (long long)N);
    REQUIRE(k_sizes_host != nullptr, "k_sizes_host is NULL");
    int64_t total = 0;
    for (int64_t g = 0; g < G; ++g) {
        const int64_t kg = k_sizes_host[g];
        REQUIRE(kg >= 0 && kg % 128 == 0, "k_sizes_host[%lld]=%lld must be >= 0 and a multiple of 128",
                (long long)g, (long long)kg);
        total += kg;
    }
    REQUIRE(total == K_tot, "sum of k_sizes_host (%lld) != K_tot (%lld)", (long long)total,
            (long long)K_tot);
    if (M == 0 || N == 0) return ok();
    REQUIRE_PTR(d, 16);
    if (c) REQUIRE_PTR(c, 16);
    if (K_tot > 0) {
        REQUIRE_PTR(a, 16);
        REQUIRE_PTR(b, 16);
        REQUIRE_PTR(sfa, 16);
        REQUIRE_PTR(sfb, 16);
    }
    REQUIRE(K_tot <= kOffsetLimit / M && K_tot <= kOffsetLimit / N,
            "K_tot*M and K_tot*N must stay below 2^31");
    REQUIRE(G * ((M + 127) / 128) * ((N + 127) / 128) <= INT_MAX, "too many tiles");
    REQUIRE(alias_ok(c, d, G * M * N * 4), "c overlaps d without being equal to it");
    dg::TnProblem p{};
    p.form = dg::kKGrouped;
    p.a_mk = false; p.b_nk = false; p.out_f32 = true; p.ue8m0 = ue8m0;
    p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.k_sizes_host = k_sizes_host;
    p.c = c; p.d = d; p.G = G; p.M = M; p.N = N; p.K_tot = K_tot;
    return run_tn(p, stream);
}

// Dense NN / TN / TT: A stored [M, K] (a_mk) or [K, M]; B stored [N, K] (b_nk)
// or [K, N]; sfa [K/128, M], sfb [K/128, N]; C like D (may equal it).
static dg_status gemm_layout(const uint8_t* a, bool a_mk, const float* sfa, const uint8_t* b,
                             bool b_nk, const float* sfb, const void* c, void* d,
                             dg_dtype d_dtype, int64_t M, int64_t N, int64_t K, void* stream) {
    REQUIRE(M >= 0 && N >= 0 && K >= 0, "negative size (M=%lld N=%lld K=%lld)", (long long)M,
            (long long)N, (long long)K);
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(N % 16 == 0, "N=%lld is not a multiple of 16", (long long)N);
    REQUIRE(a_mk || M % 16 == 0, "M=%lld is not a multiple of 16 (A stored [K, M])", (long long)M);
    REQUIRE(d_dtype == DG_BF16 || d_dtype == DG_F32, "d_dtype must be DG_BF16 or DG_F32");
    if (M == 0 || N == 0) return ok();
    REQUIRE_PTR(d, 16);
    if (c) REQUIRE_PTR(c, 16);
    if (K > 0) {
        REQUIRE_PTR(a, 16);
        REQUIRE_PTR(b, 16);
        REQUIRE_PTR(sfa, 16);
        REQUIRE_PTR(sfb, 16);
    }
    REQUIRE(M <= kOffsetLimit / (K > 0 ? K : 1) && N <= kOffsetLimit / (K > 0 ? K : 1),
            "M*K and N*K must stay below 2^31");
    REQUIRE(((M + 127) / 128) * ((N + 127) / 128) <= INT_MAX, "too many tiles");
    REQUIRE(alias_ok(c, d, M * N * (d_dtype == DG_F32 ? 4 : 2)),
            "c overlaps d without being equal to it");
    dg::TnProblem p{};
    p.form = dg::kDenseLayout;
    p.a_mk = a_mk; p.b_nk = b_nk; p.out_f32 = d_dtype == DG_F32;
    p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.c = c; p.d = d;
    p.G = 1; p.M = M; p.N = N; p.K_tot = K;
    return run_tn(p, stream);
}

dg_status dg_fp8_gemm_nn(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                         const void* c, void* d, dg_dtype d_dtype, int64_t M, int64_t N,
                         int64_t K, void* stream) {
    return gemm_layout(a, true, sfa, b, false, sfb, c, d, d_dtype, M, N, K, stream);
}

dg_status dg_fp8_gemm_tn(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                         const void* c, void* d, dg_dtype d_dtype, int64_t M, int64_t N,
                         int64_t K, void* stream) {
    return gemm_layout(a, false, sfa, b, false, sfb, c, d, d_dtype, M, N, K, stream);
}

dg_status dg_fp8_gemm_tt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                         const void* c, void* d, dg_dtype d_dtype, int64_t M, int64_t N,
                         int64_t K, void* stream) {
    return gemm_layout(a, false, sfa, b, true, sfb, c, d, d_dtype, M, N, K, stream);
}

dg_status dg_m_grouped_fp8_gemm_nn_contiguous(const uint8_t* a, const float* sfa,
                                              const uint8_t* b, const float* sfb,
                                              const int32_t* m_indices, void* d, int64_t M_tot,
                                              int64_t N, int64_t K, int64_t G, void* stream) {
    REQUIRE(M_tot >= 0 && N >= 0 && K >= 0, "negative size");
    REQUIRE(G >= 1, "G=%lld must be >= 1", (long long)G);
    REQUIRE(M_tot % 128 == 0, "M_tot=%lld is not a multiple of 128 (the contiguous-layout alignment)",
            (long long)M_tot);
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(N % 16 == 0, "N=%lld is not a multiple of 16", (long long)N);
    if (M_tot == 0 || N == 0) return ok();
    REQUIRE_PTR(a, 16);
    REQUIRE_PTR(b, 16);
    REQUIRE_PTR(d, 16);
    REQUIRE_PTR(sfa, 16);
    REQUIRE_PTR(sfb, 16);
    REQUIRE_PTR(m_indices, 16);
    REQUIRE(M_tot <= kOffsetLimit / (K > 0 ? K : 1) && N <= kOffsetLimit / (K > 0 ? K : 1),
            "M_tot*K and K*N must stay below 2^31");
    REQUIRE(G <= INT_MAX && (M_tot / 128) * ((N + 255) / 256) <= INT_MAX, "too many tiles");
    dg::TnProblem p{};
    p.form = dg::kMGroupedNN;
    p.a_mk = true; p.b_nk = false; p.out_f32 = false;
    p.a = a; p.sfa = sfa; p.b = b; p.sfb = sfb; p.m_indices = m_indices; p.c = nullptr; p.d = d;
    p.G = G; p.M = M_tot; p.N = N; p.K_tot = K;
    return run_tn(p, stream);
}

static dg_status run_cast(const void* x, dg_dtype dtype, uint8_t* codes, float* sf, int64_t G,
                          int64_t R, int64_t K, int flags, bool block_scale, void* stream) {
    REQUIRE(G >= 0 && R >= 0 && K >= 0, "negative size (G=%lld rows=%lld K=%lld)", (long long)G,
            (long long)R, (long long)K);
    REQUIRE(K % 128 == 0, "K=%lld is not a multiple of 128", (long long)K);
    REQUIRE(dtype == DG_BF16 || dtype == DG_F32, "input dtype must be DG_BF16 or DG_F32");
    REQUIRE(flags == 0 || flags == DG_CAST_POW2_SCALE, "flags must be 0 or DG_CAST_POW2_SCALE");
    if (G == 0 || R == 0 || K == 0) return ok();
    REQUIRE_PTR(x, 16);
    REQUIRE_PTR(codes, 16);
    REQUIRE_PTR(sf, 16);
    REQUIRE(R <= kOffsetLimit && K <= kOffsetLimit, "size too large");
    REQUIRE(G <= kOffsetLimit && R <= kOffsetLimit / K, "rows*K must stay below 2^31");
    const int64_t n = G * R * K;   // < 2^62
    const int64_t in_bytes = n * (dtype == DG_F32 ? 4 : 2);
    const int64_t kb = K / 128;
    const int64_t sf_count = block_scale ? G * ((R + 127) / 128) * kb : G * kb * R;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), c0 = reinterpret_cast<uintptr_t>(codes),
                    s0 = reinterpret_cast<uintptr_t>(sf);
    auto disjoint = [](uintptr_t a, int64_t na, uintptr_t b, int64_t nb) {
        return a + (uintptr_t)na <= b || b + (uintptr_t)nb <= a;
    };
    REQUIRE(disjoint(x0, in_bytes, c0, n) && disjoint(x0, in_bytes, s0, sf_count * 4) &&
                disjoint(c0, n, s0, sf_count * 4),
            "input, codes and sf must not overlap");
    dg::CastProblem p{};
    p.x = x; p.in_f32 = dtype == DG_F32; p.block_scale = block_scale;
    p.pow2 = flags == DG_CAST_POW2_SCALE;
    p.codes = codes; p.sf = sf; p.G = G; p.R = R; p.K = K;
    REQUIRE(dg::cast_grid(p) <= INT_MAX, "too many blocks");
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_cast(p, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

dg_status dg_per_token_cast_to_fp8(const void* x, dg_dtype x_dtype, uint8_t* codes, float* sf,
                                   int64_t G, int64_t R, int64_t K, int flags, void* stream) {
    return run_cast(x, x_dtype, codes, sf, G, R, K, flags, false, stream);
}

dg_status dg_per_block_cast_to_fp8(const void* w, dg_dtype w_dtype, uint8_t* codes, float* sf,
                                   int64_t G, int64_t N, int64_t K, int flags, void* stream) {
    return run_cast(w, w_dtype, codes, sf, G, N, K, flags, true, stream);
}

dg_status dg_fp8_mqa_logits(const uint8_t* q, const uint8_t* kv, const float* kv_sf,
                            const float* weights, const int32_t* ks, const int32_t* ke,
                            float* logits, int64_t S, int64_t S_kv, int64_t H, int64_t D,
                            int clean_logits, void* stream) {
    REQUIRE(S >= 0 && S_kv >= 0, "negative size (seq_len=%lld seq_len_kv=%lld)", (long long)S,
            (long long)S_kv);
    REQUIRE(D == 128, "head_dim=%lld: only 128 is supported (one MFMA K step)", (long long)D);
    REQUIRE(H == 16 || H == 32 || H == 64, "num_heads=%lld must be 16, 32 or 64", (long long)H);
    REQUIRE(clean_logits == 0 || clean_logits == 1, "clean_logits must be 0 or 1");
    if (S == 0 || S_kv == 0) return ok();
    REQUIRE_PTR(q, 16);
    REQUIRE_PTR(kv, 16);
    REQUIRE_PTR(weights, 16);
    REQUIRE_PTR(logits, 16);
    REQUIRE_PTR(kv_sf, 16);
    REQUIRE_PTR(ks, 16);
    REQUIRE_PTR(ke, 16);
    // token indices are 32-bit and run up to one workgroup (256 tokens) past S_kv
    REQUIRE(S <= 65535LL * 16 && S_kv <= INT_MAX - 4096,
            "seq_len must be <= 1048560 and seq_len_kv <= 2^31 - 4097");
    dg::MqaProblem p{};
    p.q = q; p.kv = kv; p.kv_sf = kv_sf; p.weights = weights; p.ks = ks; p.ke = ke;
    p.logits = logits; p.S = S; p.S_kv = S_kv; p.H = H; p.clean = clean_logits != 0;
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_mqa(p, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

// ---- few tokens at a time ---------------------------------------------------------

static bool cache_page_ok(int64_t page_size) {
    return page_size >= 16 && page_size <= 4096 && (page_size & (page_size - 1)) == 0;
}

static bool cache_dim_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

static dg_status check_cache(const dg::KvCache& c) {
    const uint8_t *k_codes = c.k_codes, *v_codes = c.v_codes;
    const void *k_sf = c.k_sf, *v_sf = c.v_sf;
    REQUIRE_PTR(k_codes, 16);
    REQUIRE_PTR(k_sf, 16);
    REQUIRE_PTR(v_codes, 16);
    REQUIRE_PTR(v_sf, 16);
    return DG_OK;
}

static dg_status check_cache_sizes(const dg::KvCache& c) {
    REQUIRE(c.H >= 0 && c.num_pages >= 0, "negative size (H=%lld num_pages=%lld)", (long long)c.H,
            (long long)c.num_pages);
    REQUIRE(cache_dim_ok(c.D), "D=%lld must be 64, 128 or 256", (long long)c.D);
    REQUIRE(cache_page_ok(c.page_size), "page_size=%lld must be a power of two from 16 to 4096",
            (long long)c.page_size);
    REQUIRE(c.H <= 65535, "H=%lld too large", (long long)c.H);
    REQUIRE(c.num_pages <= INT_MAX / c.page_size, "num_pages * page_size must stay below 2^31");
    return DG_OK;
}

// Whether [p, p + n) stays clear of the cache's four arrays.
static bool clear_of_cache(const dg::KvCache& c, const void* p, int64_t n) {
    return disjoint(p, n, c.k_codes, c.code_bytes()) && disjoint(p, n, c.v_codes, c.code_bytes()) &&
           disjoint(p, n, c.k_sf, c.sf_bytes()) && disjoint(p, n, c.v_sf, c.sf_bytes());
}

static dg_status kv_cache_copy(dg::KvCopy p, dg_dtype dtype, bool write, void* stream) {
    dg_status st = check_cache_sizes(p.cache);
    if (st != DG_OK) return st;
    REQUIRE(p.T >= 0, "negative size (T=%lld)", (long long)p.T);
    REQUIRE(dtype == DG_BF16 || dtype == DG_F32, "dtype must be DG_BF16 or DG_F32");
    const int64_t H = p.cache.H, D = p.cache.D, size = dtype == DG_F32 ? 4 : 2;
    REQUIRE(p.T <= INT_MAX, "T=%lld too large", (long long)p.T);
    REQUIRE(p.k_stride >= H * D && p.v_stride >= H * D && p.k_stride <= kOffsetLimit && p.v_stride <= kOffsetLimit,
            "k_stride=%lld and v_stride=%lld must be from H * D = %lld to 2^31", (long long)p.k_stride,
            (long long)p.v_stride, (long long)(H * D));
    REQUIRE(p.k_stride * size % 16 == 0 && p.v_stride * size % 16 == 0,
            "k_stride and v_stride must be multiples of 16 bytes");
    if (p.T == 0 || H == 0) return ok();
    REQUIRE(p.cache.num_pages >= 1, "num_pages=0: the cache is empty");
    const void *k = p.k, *v = p.v;
    const int32_t* slots = p.slots;
    REQUIRE_PTR(k, 16);
    REQUIRE_PTR(v, 16);
    REQUIRE_PTR(slots, 4);
    st = check_cache(p.cache);
    if (st != DG_OK) return st;
    REQUIRE(p.T <= INT_MAX / H, "T * H must stay below 2^31");
    const int64_t kn = ((p.T - 1) * p.k_stride + H * D) * size, vn = ((p.T - 1) * p.v_stride + H * D) * size;
    REQUIRE(clear_of_cache(p.cache, k, kn) && clear_of_cache(p.cache, v, vn) &&
                clear_of_cache(p.cache, slots, 4 * p.T),
            "k, v or slots overlap the cache");
    if (write) {
        const dg::KvCache& c = p.cache;
        const int64_t codes = c.code_bytes(), sf = c.sf_bytes();
        REQUIRE(disjoint(c.k_codes, codes, c.v_codes, codes) && disjoint(c.k_sf, sf, c.v_sf, sf) &&
                    disjoint(c.k_codes, codes, c.k_sf, sf) && disjoint(c.k_codes, codes, c.v_sf, sf) &&
                    disjoint(c.v_codes, codes, c.k_sf, sf) && disjoint(c.v_codes, codes, c.v_sf, sf),
                "the cache's arrays overlap");
    } else {
        REQUIRE(disjoint(k, kn, v, vn) && disjoint(k, kn, slots, 4 * p.T) && disjoint(v, vn, slots, 4 * p.T),
                "k, v and slots must not overlap");
    }
    p.f32 = dtype == DG_F32;
    int dev = 0;
    DeviceInfo info;
    st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipStream_t on = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = p.cache.fp4 ? (write ? dg::launch_kv4_cache_write(p, on) : dg::launch_kv4_cache_read(p, on))
                               : (write ? dg::launch_kv_cache_write(p, on) : dg::launch_kv_cache_read(p, on));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

dg_status dg_fp8_kv_cache_write(const void* k, const void* v, dg_dtype dtype, int64_t k_stride,
                                int64_t v_stride, const int32_t* slots, uint8_t* k_codes,
                                float* k_sf, uint8_t* v_codes, float* v_sf, int64_t T, int64_t H,
                                int64_t D, int64_t num_pages, int64_t page_size, void* stream) {
    dg::KvCopy p{};
    p.cache = dg::KvCache{k_codes, k_sf, v_codes, v_sf, num_pages, H, page_size, D, false};
    p.slots = slots;
    p.k = const_cast<void*>(k); p.v = const_cast<void*>(v);
    p.k_stride = k_stride; p.v_stride = v_stride; p.T = T;
    return kv_cache_copy(p, dtype, true, stream);
}

dg_status dg_fp8_kv_cache_read(const uint8_t* k_codes, const float* k_sf, const uint8_t* v_codes,
                               const float* v_sf, const int32_t* slots, void* k, void* v,
                               dg_dtype dtype, int64_t T, int64_t H, int64_t D, int64_t num_pages,
                               int64_t page_size, void* stream) {
    dg::KvCopy p{};
    p.cache = dg::KvCache{const_cast<uint8_t*>(k_codes), const_cast<float*>(k_sf),
                          const_cast<uint8_t*>(v_codes), const_cast<float*>(v_sf),
                          num_pages, H, page_size, D, false};
    p.slots = slots;
    p.k = k; p.v = v;
    p.k_stride = p.v_stride = H > 0 && H <= 65535 && cache_dim_ok(D) ? H * D : 0;
    p.T = T;
    return kv_cache_copy(p, dtype, false, stream);
}

dg_status dg_fp4_kv_cache_write(const void* k, const void* v, dg_dtype dtype, int64_t k_stride,
                                int64_t v_stride, const int32_t* slots, uint8_t* k_codes,
                                uint8_t* k_sf, uint8_t* v_codes, uint8_t* v_sf, int64_t T, int64_t H,
                                int64_t D, int64_t num_pages, int64_t page_size, void* stream) {
    dg::KvCopy p{};
    p.cache = dg::KvCache{k_codes, k_sf, v_codes, v_sf, num_pages, H, page_size, D, true};
    p.slots = slots;
    p.k = const_cast<void*>(k); p.v = const_cast<void*>(v);
    p.k_stride = k_stride; p.v_stride = v_stride; p.T = T;
    return kv_cache_copy(p, dtype, true, stream);
}

dg_status dg_fp4_kv_cache_read(const uint8_t* k_codes, const uint8_t* k_sf, const uint8_t* v_codes,
                               const uint8_t* v_sf, const int32_t* slots, void* k, void* v,
                               dg_dtype dtype, int64_t T, int64_t H, int64_t D, int64_t num_pages,
                               int64_t page_size, void* stream) {
    dg::KvCopy p{};
    p.cache = dg::KvCache{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_sf),
                          const_cast<uint8_t*>(v_codes), const_cast<uint8_t*>(v_sf),
                          num_pages, H, page_size, D, true};
    p.slots = slots;
    p.k = k; p.v = v;
    p.k_stride = p.v_stride = H > 0 && H <= 65535 && cache_dim_ok(D) ? H * D : 0;
    p.T = T;
    return kv_cache_copy(p, dtype, false, stream);
}

dg_status dg_kv_cache_plan(int32_t* page_table, const int32_t* context_lens, const int32_t* add_lens,
                           int32_t* pool_pages, const int32_t* pool_state, int32_t* slots,
                           int32_t* positions, int32_t* new_lens, int32_t* new_state, int64_t B,
                           int64_t rows, int padded, int64_t max_pages, int64_t num_pages,
                           int64_t page_size, void* stream) {
    REQUIRE(B >= 0 && rows >= 0, "negative size (B=%lld rows=%lld)", (long long)B, (long long)rows);
    REQUIRE(padded == 0 || padded == 1, "padded must be 0 or 1");
    REQUIRE(cache_page_ok(page_size), "page_size=%lld must be a power of two from 16 to 4096", (long long)page_size);
    REQUIRE(num_pages >= 1 && num_pages <= INT_MAX / page_size,
            "num_pages=%lld: num_pages * page_size must be from page_size to 2^31", (long long)num_pages);
    REQUIRE(max_pages >= 1 && max_pages <= (1LL << 30) / page_size,
            "max_pages=%lld: max_pages * page_size must be from page_size to 2^30", (long long)max_pages);
    REQUIRE(B <= 65536, "B=%lld must be at most 65536", (long long)B);
    REQUIRE(rows <= INT_MAX && (!padded || B == 0 || rows <= INT_MAX / B), "rows=%lld: too many rows", (long long)rows);
    const int64_t all = padded ? B * rows : rows;
    if (B > 0) {
        REQUIRE_PTR(page_table, 4);
        REQUIRE_PTR(context_lens, 4);
        REQUIRE_PTR(add_lens, 4);
        REQUIRE_PTR(new_lens, 4);
    }
    REQUIRE_PTR(pool_pages, 4);
    REQUIRE_PTR(pool_state, 4);
    REQUIRE_PTR(new_state, 4);
    if (all > 0) {
        REQUIRE_PTR(slots, 4);
        REQUIRE_PTR(positions, 4);
    }
    const struct { const void* p; int64_t n; bool written; } buffers[] = {
        {page_table, B * max_pages, true}, {pool_pages, num_pages, true}, {slots, all, true}, {positions, all, true},
        {new_lens, B, true}, {new_state, 2, true}, {context_lens, B, false}, {add_lens, B, false}, {pool_state, 2, false}};
    for (size_t i = 0; i < sizeof buffers / sizeof buffers[0]; ++i)
        for (size_t j = 0; j < i; ++j)
            REQUIRE(buffers[i].n == 0 || buffers[j].n == 0 || !buffers[j].written ||
                        disjoint(buffers[i].p, buffers[i].n * 4, buffers[j].p, buffers[j].n * 4),
                    "what the call writes overlaps something else");
    dg::KvPlan p{};
    p.page_table = page_table; p.context_lens = context_lens; p.add_lens = add_lens;
    p.pool_pages = pool_pages; p.pool_state = pool_state;
    p.slots = slots; p.positions = positions; p.new_lens = new_lens; p.new_state = new_state;
    p.B = B; p.rows = rows; p.padded = padded != 0;
    p.max_pages = max_pages; p.num_pages = num_pages; p.page_size = page_size;
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_kv_cache_plan(p, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

// What the sizes of a norm and rotation have to be; "" where they are right.
static const char* norm_rope_sizes_wrong(int64_t T, int64_t Hq, int64_t H, int64_t D) {
    if (T < 0 || Hq < 0 || H < 0) return "T, Hq and H must not be negative";
    if (!cache_dim_ok(D)) return "D must be 64, 128 or 256";
    if (Hq > 65535 || H > 65535) return "Hq and H must be at most 65535";
    if (T > INT_MAX || T * Hq > INT_MAX || T * H > INT_MAX) return "T * Hq and T * H must stay below 2^31";
    return "";
}

// A buffer: its bytes from first to last, and for strided rows their distance and width.
struct Rows {
    const void* p;
    int64_t n, stride, width;
};

// Whether two share no byte; rows side by side in the same wider rows do not.
static bool rows_disjoint(const Rows& a, const Rows& b) {
    if (a.n == 0 || b.n == 0 || disjoint(a.p, a.n, b.p, b.n)) return true;
    if (a.stride == 0 || a.stride != b.stride) return false;
    const int64_t d = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
    const int64_t at = (d % a.stride + a.stride) % a.stride;
    return at >= a.width && at + b.width <= a.stride;
}

// Both directions: what they share is checked here.
static dg_status norm_rope(dg::NormRope p, dg_dtype dtype, dg_dtype w_dtype, int interleaved,
                           int64_t workspace_bytes, void* stream) {
    const char* wrong = norm_rope_sizes_wrong(p.T, p.Hq, p.H, p.D);
    REQUIRE(!*wrong, "%s (T=%lld Hq=%lld H=%lld D=%lld)", wrong, (long long)p.T, (long long)p.Hq, (long long)p.H,
            (long long)p.D);
    REQUIRE(p.R >= 0 && p.R <= p.D && p.R % 16 == 0, "R=%lld must be a multiple of 16 from 0 to D", (long long)p.R);
    REQUIRE(dtype == DG_BF16 || dtype == DG_F32, "dtype must be DG_BF16 or DG_F32");
    REQUIRE(w_dtype == DG_BF16 || w_dtype == DG_F32, "w_dtype must be DG_BF16 or DG_F32");
    REQUIRE(interleaved == 0 || interleaved == 1, "interleaved must be 0 or 1");
    REQUIRE(std::isfinite(p.eps) && p.eps >= 0x1p-100f, "eps=%g must be finite and 2^-100 at least", (double)p.eps);
    const int64_t size = dtype == DG_F32 ? 4 : 2, heads[2] = {p.Hq, p.H};
    const bool any = p.T > 0 && (p.Hq > 0 || p.H > 0);
    Rows in[9], out[5];                    // x, dz and w of both, positions, inv_freq; out and dw of both, workspace
    int ins = 0, outs = 0, own[5] = {-1, -1, -1, -1, -1};      // the input that an output is in place of
    for (int i = 0; i < 2; ++i) {
        const struct { const void* p; int64_t stride; const char* name; bool used, written; } rows[3] = {
            {p.x[i], p.x_stride[i], i ? "k" : "q", true, false},
            {p.dz[i], p.dz_stride[i], i ? "dk" : "dq", p.backward, false},
            {p.out[i], p.out_stride[i], p.backward ? (i ? "dk_in" : "dq_in") : (i ? "k_out" : "q_out"), true, true}};
        for (const auto& r : rows) {
            if (!r.used) continue;
            REQUIRE(r.stride >= heads[i] * p.D && r.stride <= kOffsetLimit && r.stride * size % 16 == 0,
                    "%s_stride=%lld must be a multiple of 16 bytes, from heads * D = %lld to 2^31", r.name,
                    (long long)r.stride, (long long)(heads[i] * p.D));
            if (p.T == 0 || heads[i] == 0) continue;
            REQUIRE(r.p != nullptr, "%s is NULL", r.name);
            REQUIRE(aligned(r.p, 16), "%s is not 16-byte aligned", r.name);
            // forward, a tensor's own input and output may be one: a row is written by the lanes that have read it
            if (r.written && !p.backward && r.p == p.x[i] && r.stride == p.x_stride[i]) own[outs] = ins - 1;
            (r.written ? out[outs++] : in[ins++]) = Rows{r.p, ((p.T - 1) * r.stride + heads[i] * p.D) * size,
                                                         r.stride * size, heads[i] * p.D * size};
        }
        REQUIRE(aligned(p.w[i], 16), "%s is not 16-byte aligned", i ? "k_weight" : "q_weight");
        REQUIRE(aligned(p.dw[i], 16), "%s is not 16-byte aligned", i ? "dk_weight" : "dq_weight");
        if (p.w[i]) in[ins++] = Rows{p.w[i], p.D * (w_dtype == DG_F32 ? 4 : 2), 0, 0};
        if (p.dw[i]) out[outs++] = Rows{p.dw[i], p.D * 4, 0, 0};
    }
    if (!any && !p.dw[0] && !p.dw[1]) return ok();
    if (any && p.R > 0) {
        const int32_t* positions = p.positions;
        const float* inv_freq = p.inv_freq;
        REQUIRE_PTR(positions, 4);
        REQUIRE_PTR(inv_freq, 4);
        in[ins++] = Rows{positions, p.T * 4, 0, 0};
        in[ins++] = Rows{inv_freq, p.R * 2, 0, 0};
    }
    if (any && (p.dw[0] || p.dw[1])) {
        const int64_t need = dg::norm_rope_workspace_bytes(p.T, p.Hq, p.H, p.D);
        void* workspace = p.workspace;
        REQUIRE_PTR(workspace, 16);
        REQUIRE(workspace_bytes >= need, "workspace_bytes=%lld < %lld needed for these sizes",
                (long long)workspace_bytes, (long long)need);
        out[outs++] = Rows{workspace, need, 0, 0};
    }
    for (int i = 0; i < outs; ++i) {
        for (int k = 0; k < ins; ++k)
            REQUIRE(own[i] == k || rows_disjoint(out[i], in[k]), "an output or the workspace overlaps an input");
        for (int k = 0; k < i; ++k) REQUIRE(rows_disjoint(out[i], out[k]), "the outputs or the workspace overlap");
    }
    p.f32 = dtype == DG_F32;
    p.w_f32 = w_dtype == DG_F32;
    p.neighbours = interleaved != 0;
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_norm_rope(p, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

dg_status dg_qk_norm_rope(const void* q, const void* k, dg_dtype dtype, int64_t q_stride, int64_t k_stride,
                          const void* q_weight, const void* k_weight, dg_dtype w_dtype,
                          const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                          int64_t q_out_stride, int64_t k_out_stride, float eps, int interleaved,
                          int64_t T, int64_t Hq, int64_t H, int64_t D, int64_t R, void* stream) {
    dg::NormRope p{};
    p.x[0] = q; p.x[1] = k;
    p.out[0] = q_out; p.out[1] = k_out;
    p.x_stride[0] = q_stride; p.x_stride[1] = k_stride;
    p.out_stride[0] = q_out_stride; p.out_stride[1] = k_out_stride;
    p.w[0] = q_weight; p.w[1] = k_weight;
    p.positions = positions; p.inv_freq = inv_freq; p.eps = eps;
    p.T = T; p.Hq = Hq; p.H = H; p.D = D; p.R = R;
    return norm_rope(p, dtype, w_dtype, interleaved, 0, stream);
}

int64_t dg_qk_norm_rope_backward_workspace_bytes(int64_t T, int64_t Hq, int64_t H, int64_t D) {
    if (*norm_rope_sizes_wrong(T, Hq, H, D)) return 0;
    return dg::norm_rope_workspace_bytes(T, Hq, H, D);
}

dg_status dg_qk_norm_rope_backward(const void* dq, const void* dk, const void* q, const void* k, dg_dtype dtype,
                                   int64_t dq_stride, int64_t dk_stride, int64_t q_stride, int64_t k_stride,
                                   const void* q_weight, const void* k_weight, dg_dtype w_dtype,
                                   const int32_t* positions, const float* inv_freq, void* dq_in, void* dk_in,
                                   int64_t dq_in_stride, int64_t dk_in_stride, float* dq_weight,
                                   float* dk_weight, float eps, int interleaved, int64_t T, int64_t Hq,
                                   int64_t H, int64_t D, int64_t R, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    dg::NormRope p{};
    p.x[0] = q; p.x[1] = k;
    p.dz[0] = dq; p.dz[1] = dk;
    p.out[0] = dq_in; p.out[1] = dk_in;
    p.x_stride[0] = q_stride; p.x_stride[1] = k_stride;
    p.dz_stride[0] = dq_stride; p.dz_stride[1] = dk_stride;
    p.out_stride[0] = dq_in_stride; p.out_stride[1] = dk_in_stride;
    p.w[0] = q_weight; p.w[1] = k_weight;
    p.dw[0] = dq_weight; p.dw[1] = dk_weight;
    p.positions = positions; p.inv_freq = inv_freq; p.eps = eps;
    p.T = T; p.Hq = Hq; p.H = H; p.D = D; p.R = R;
    p.backward = true;
    p.workspace = workspace;
    return norm_rope(p, dtype, w_dtype, interleaved, workspace_bytes, stream);
}

// What the sizes of a tree attention call have to be; "" where they are right.
static const char* tree_attn_sizes_wrong(int64_t B, int64_t N, int64_t Hq, int64_t H, int64_t D,
                                         int64_t page_size, int64_t max_pages) {
    if (B < 0 || N < 0 || Hq < 0 || H < 1 || max_pages < 1) return "B, N, Hq >= 0, H >= 1 and max_pages >= 1 are needed";
    if (!cache_dim_ok(D)) return "D must be 64, 128 or 256";
    if (!cache_page_ok(page_size)) return "page_size must be a power of two from 16 to 4096";
    if (H > 65535 || Hq > 65535 || Hq % H != 0) return "Hq must be a multiple of H, both at most 65535";
    if (max_pages > (1LL << 30) / page_size) return "max_pages * page_size must be at most 2^30";
    if (N >= (1LL << 20) || N * Hq >= (1LL << 20)) return "N * Hq must stay below 2^20";
    if (B > (1LL << 20) || B * H > (1LL << 20)) return "B * H must be at most 2^20";
    return "";
}

int64_t dg_fp8_tree_attention_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H,
                                              int64_t D, int64_t page_size, int64_t max_pages) {
    if (B <= 0 || N <= 0 || Hq <= 0 || *tree_attn_sizes_wrong(B, N, Hq, H, D, page_size, max_pages)) return 0;
    return dg::tree_attn_workspace_bytes(B, N, Hq, H, D, max_pages, page_size);
}

static dg_status tree_attention(bool fp4, const void* q, int64_t q_stride, const uint8_t* k_codes,
                                const void* k_sf, const uint8_t* v_codes, const void* v_sf,
                                const int32_t* page_table, const int32_t* context_lens,
                                const int32_t* tree_lens, const uint64_t* tree_mask, void* o,
                                float* lse, float scale, int64_t B, int64_t N, int64_t Hq,
                                int64_t H, int64_t D, int64_t num_pages, int64_t page_size,
                                int64_t max_pages, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    const char* wrong = tree_attn_sizes_wrong(B, N, Hq, H, D, page_size, max_pages);
    REQUIRE(!*wrong, "%s (B=%lld N=%lld Hq=%lld H=%lld D=%lld page_size=%lld max_pages=%lld)", wrong,
            (long long)B, (long long)N, (long long)Hq, (long long)H, (long long)D, (long long)page_size,
            (long long)max_pages);
    REQUIRE(num_pages >= 1 && num_pages <= INT_MAX / page_size,
            "num_pages=%lld: num_pages * page_size must be from page_size to 2^31", (long long)num_pages);
    REQUIRE(q_stride >= Hq * D && q_stride % 8 == 0 && q_stride <= kOffsetLimit,
            "q_stride=%lld must be a multiple of 8 from Hq * D = %lld to 2^31", (long long)q_stride,
            (long long)(Hq * D));
    REQUIRE(std::isfinite(scale), "scale is not finite");
    if (B == 0 || N == 0 || Hq == 0) return ok();
    dg::TreeAttnProblem p{};
    p.cache = dg::KvCache{const_cast<uint8_t*>(k_codes), const_cast<void*>(k_sf),
                          const_cast<uint8_t*>(v_codes), const_cast<void*>(v_sf),
                          num_pages, H, page_size, D, fp4};
    REQUIRE_PTR(q, 16);
    dg_status st = check_cache(p.cache);
    if (st != DG_OK) return st;
    REQUIRE_PTR(page_table, 4);
    REQUIRE_PTR(context_lens, 4);
    if (tree_lens) REQUIRE_PTR(tree_lens, 4);
    if (tree_mask) REQUIRE_PTR(tree_mask, 8);
    REQUIRE_PTR(o, 16);
    REQUIRE_PTR(lse, 4);
    const int64_t need = fp4 ? dg::tree_attn4_workspace_bytes(B, N, Hq, H, D, max_pages, page_size)
                             : dg::tree_attn_workspace_bytes(B, N, Hq, H, D, max_pages, page_size);
    REQUIRE(workspace_bytes >= need, "workspace_bytes=%lld < %lld needed for these sizes",
            (long long)workspace_bytes, (long long)need);
    if (need > 0) REQUIRE_PTR(workspace, 16);
    const int64_t tokens = B * N, on = tokens * Hq * D * 2, ln = tokens * Hq * 4,
                  qn = ((tokens - 1) * q_stride + Hq * D) * 2;
    const struct { const void* p; int64_t n; } in[] = {
        {q, qn}, {page_table, B * max_pages * 4}, {context_lens, B * 4},
        {tree_lens, tree_lens ? B * 4 : 0}, {tree_mask, tree_mask ? tokens * ((N + 63) / 64) * 8 : 0}},
                 out[] = {{o, on}, {lse, ln}, {workspace, need}};
    for (int i = 0; i < 3; ++i) {
        if (out[i].n == 0) continue;
        REQUIRE(clear_of_cache(p.cache, out[i].p, out[i].n), "o, lse or workspace overlaps the cache");
        for (const auto& x : in)
            REQUIRE(x.n == 0 || disjoint(out[i].p, out[i].n, x.p, x.n), "o, lse or workspace overlaps an input");
        for (int j = 0; j < i; ++j)
            REQUIRE(disjoint(out[i].p, out[i].n, out[j].p, out[j].n), "o, lse and workspace overlap");
    }
    p.q = static_cast<const uint16_t*>(q); p.q_stride = q_stride;
    p.page_table = page_table; p.context_lens = context_lens;
    p.tree_lens = tree_lens; p.tree_mask = tree_mask;
    p.o = static_cast<uint16_t*>(o); p.lse = lse; p.scale = scale;
    p.B = B; p.N = N; p.Hq = Hq; p.max_pages = max_pages;
    p.workspace = workspace;
    int dev = 0;
    DeviceInfo info;
    st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipStream_t on_stream = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = fp4 ? dg::launch_tree_attn4(p, on_stream) : dg::launch_tree_attn(p, on_stream);
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

dg_status dg_fp8_tree_attention(const void* q, int64_t q_stride, const uint8_t* k_codes,
                                const float* k_sf, const uint8_t* v_codes, const float* v_sf,
                                const int32_t* page_table, const int32_t* context_lens,
                                const int32_t* tree_lens, const uint64_t* tree_mask, void* o,
                                float* lse, float scale, int64_t B, int64_t N, int64_t Hq,
                                int64_t H, int64_t D, int64_t num_pages, int64_t page_size,
                                int64_t max_pages, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    return tree_attention(false, q, q_stride, k_codes, k_sf, v_codes, v_sf, page_table, context_lens, tree_lens,
                          tree_mask, o, lse, scale, B, N, Hq, H, D, num_pages, page_size, max_pages, workspace,
                          workspace_bytes, stream);
}

dg_status dg_fp4_tree_attention(const void* q, int64_t q_stride, const uint8_t* k_codes,
                                const uint8_t* k_sf, const uint8_t* v_codes, const uint8_t* v_sf,
                                const int32_t* page_table, const int32_t* context_lens,
                                const int32_t* tree_lens, const uint64_t* tree_mask, void* o,
                                float* lse, float scale, int64_t B, int64_t N, int64_t Hq,
                                int64_t H, int64_t D, int64_t num_pages, int64_t page_size,
                                int64_t max_pages, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    return tree_attention(true, q, q_stride, k_codes, k_sf, v_codes, v_sf, page_table, context_lens, tree_lens,
                          tree_mask, o, lse, scale, B, N, Hq, H, D, num_pages, page_size, max_pages, workspace,
                          workspace_bytes, stream);
}

int64_t dg_fp4_tree_attention_workspace_bytes(int64_t B, int64_t N, int64_t Hq, int64_t H,
                                              int64_t D, int64_t page_size, int64_t max_pages) {
    if (B <= 0 || N <= 0 || Hq <= 0 || *tree_attn_sizes_wrong(B, N, Hq, H, D, page_size, max_pages)) return 0;
    return dg::tree_attn4_workspace_bytes(B, N, Hq, H, D, max_pages, page_size);
}

static const char* moe_few_sizes_wrong(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I) {
    if (T < 0 || T > dg::kMoeMaxTokens) return "T must be from 0 to 256";
    if (topk < 1 || topk > dg::kMoeMaxTopk) return "topk must be from 1 to 16";
    if (E < 1 || E > dg::kMoeMaxExperts) return "E must be from 1 to 1024";
    if (H < 128 || H % 128 != 0 || H > (1 << 17)) return "H must be a multiple of 128 up to 2^17";
    if (I < 128 || I % 128 != 0 || I > (1 << 17)) return "I must be a multiple of 128 up to 2^17";
    return "";
}

int64_t dg_fp8_moe_few_tokens_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t H,
                                              int64_t I) {
    if (*moe_few_sizes_wrong(T, topk, E, H, I) || T == 0) return 0;
    return dg::moe_few_workspace_bytes(T, topk, E, H, I);
}

dg_status dg_fp8_moe_few_tokens(const void* x, const uint8_t* w1, const float* s1,
                                const uint8_t* w2, const float* s2, const int32_t* topk_ids,
                                const float* topk_weights, void* y, dg_dtype y_dtype, int64_t T,
                                int64_t topk, int64_t E, int64_t H, int64_t I, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    const char* wrong = moe_few_sizes_wrong(T, topk, E, H, I);
    REQUIRE(!*wrong, "%s (T=%lld topk=%lld E=%lld H=%lld I=%lld)", wrong, (long long)T, (long long)topk,
            (long long)E, (long long)H, (long long)I);
    REQUIRE(y_dtype == DG_BF16 || y_dtype == DG_F32, "y_dtype must be DG_BF16 or DG_F32");
    if (T == 0) return ok();
    REQUIRE_PTR(x, 16);
    REQUIRE_PTR(w1, 16);
    REQUIRE_PTR(s1, 16);
    REQUIRE_PTR(w2, 16);
    REQUIRE_PTR(s2, 16);
    REQUIRE_PTR(topk_ids, 4);
    REQUIRE_PTR(topk_weights, 4);
    REQUIRE_PTR(y, 16);
    const int64_t need = dg::moe_few_workspace_bytes(T, topk, E, H, I);
    REQUIRE(workspace != nullptr, "workspace is NULL: %lld bytes are needed "
            "(dg_fp8_moe_few_tokens_workspace_bytes)", (long long)need);
    REQUIRE_PTR(workspace, 16);
    REQUIRE(workspace_bytes >= need, "workspace_bytes=%lld < %lld needed for these sizes",
            (long long)workspace_bytes, (long long)need);
    const int64_t yn = T * H * (y_dtype == DG_F32 ? 4 : 2);
    const struct { const void* p; int64_t n; } in[] = {
        {x, T * H * 2}, {w1, E * 2 * I * H}, {s1, E * (2 * I / 128) * (H / 128) * 4}, {w2, E * H * I},
        {s2, E * (H / 128) * (I / 128) * 4}, {topk_ids, T * topk * 4}, {topk_weights, T * topk * 4}};
    for (const auto& b : in)
        REQUIRE(disjoint(y, yn, b.p, b.n) && disjoint(workspace, need, b.p, b.n),
                "y or workspace overlaps an input");
    REQUIRE(disjoint(y, yn, workspace, need), "y and workspace overlap");
    dg::MoeFewProblem p{};
    p.x = static_cast<const uint16_t*>(x);
    p.w1 = w1; p.s1 = s1; p.w2 = w2; p.s2 = s2;
    p.ids = topk_ids; p.weights = topk_weights;
    p.y = y; p.out_f32 = y_dtype == DG_F32;
    p.T = T; p.topk = topk; p.E = E; p.H = H; p.I = I;
    p.workspace = workspace;
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    hipError_t e = dg::launch_moe_few(p, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

const char* dg_last_error(void) { return g_last_error.c_str(); }

int dg_get_num_cus(void) {
    int dev = 0;
    DeviceInfo info;
    if (current_device(dev, info) != DG_OK && !info.probed) return 0;
    return cu_cap_for(info);
}

dg_status dg_set_num_cus(int n) {
    if (n == 0) {
        g_cu_cap.store(0, std::memory_order_relaxed);
        return ok();
    }
    int dev = 0;
    DeviceInfo info;
    dg_status st = current_device(dev, info);
    if (st != DG_OK) return st;
    if (n < 0 || n > info.cus)
        return fail(DG_ERR_INVALID_ARG, "num_cus=%d must be in [1, %d] (or 0 for all)", n, info.cus);
    g_cu_cap.store(n, std::memory_order_relaxed);
    return ok();
}

int dg_get_mk_alignment_for_contiguous_layout(void) { return 128; }

const char* dg_kernel_config_name(int form, int64_t rows, int64_t N, int64_t K, int out_f32) {
    if (form >= 0 && form <= 2) {
        dg::NtProblem p{};
        p.form = static_cast<dg::NtForm>(form);
        p.rows = rows; p.N = N; p.K = K; p.G = 1;
        p.out_f32 = form == 0 && out_f32 != 0;
        return dg::nt_config_name(p);
    }
    if (form >= 3 && form <= 7) {
        dg::TnProblem p{};
        p.M = rows; p.N = N; p.K_tot = K; p.G = 1;
        p.out_f32 = out_f32 != 0;
        p.form = form == 3 ? dg::kKGrouped : (form == 7 ? dg::kMGroupedNN : dg::kDenseLayout);
        p.a_mk = form == 4;           // 4 NN, 5 TN, 6 TT
        p.b_nk = form == 6;
        return dg::tn_config_name(p);
    }
    return "";
}

}  // extern "C"
