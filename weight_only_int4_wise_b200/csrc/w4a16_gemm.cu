// The host side of the tensor-core products (kernel: w4a16_gemm_kernel.cuh): plans,
// tactics, and the C entry points of the dense, grouped, 8-bit, gated and adapter
// products.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <algorithm>
#include <atomic>
#include <mutex>
#include <unordered_map>

#include "../../include/w4a16.h"
#include "w4a16_gemm_kernel.cuh"
#include "w4a16_internal.h"

namespace w4a16 {

// ====================================================================== host

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

enum Kind { kInt4 = 0, kInt8 = 1, kGatedInt4 = 2, kLoraInt4 = 3, kKinds = 4 };

struct Variant {
    int bn;
    int threads;
    int nominal_per_sm;  // the residency the variant is sized for (used when no device is present)
    int tmem_cols;       // TMEM columns each resident CTA allocates
    int smem;
};

#define W4A16_VARIANT(BN, LS, TC, MINB, DQ) {BN, threads_for(DQ), MINB, TC, Layout<BN, LS, TC>::kAlloc},
constexpr Variant kVariants[] = {W4A16_TOKEN_TILES(W4A16_VARIANT)};
#undef W4A16_VARIANT
constexpr int kNumVariants = sizeof(kVariants) / sizeof(kVariants[0]);

GemmKernel kernel_of(Kind kind, int variant, int any_group) {
    switch (kind) {
        case kInt8: return kernel_of<8, kPlain>(variant, any_group);
        case kGatedInt4: return gated_kernel(variant, any_group);
        case kLoraInt4: return lora_kernel(variant, any_group);
        default: return kernel_of<4, kPlain>(variant, any_group);
    }
}

const Variant& variant_for(int bn) {
    for (const Variant& v : kVariants)
        if (v.bn == bn) return v;
    return kVariants[kNumVariants - 1];
}

struct DeviceState {
    bool ready[kKinds] = {};
    int ctas_per_sm[kKinds][kNumVariants] = {};
};

// Prepares the kernels of one kind on the current device, at its first use: a kind that a
// process never calls costs it no preparation and no device memory, and cannot refuse
// another (a first plain product that prepared all four took 32 ms and 8 MB of device
// memory for code; with its own kind and module alone 6 ms and 2 MB).
int prepare_device(Kind kind, DeviceState** out) {
    static DeviceState states[64];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W4A16_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    DeviceState& st = states[dev];
    if (!st.ready[kind]) {
        for (int i = 0; i < kNumVariants; ++i) {
            const Variant& v = kVariants[i];
            int n = 1 << 30;
            for (int any_group = 0; any_group < 2; ++any_group) {
                const void* fn = kernel_of(kind, i, any_group).fn;
                if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess ||
                    cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared) != cudaSuccess)
                    return W4A16_ERR_CUDA;
                // Residency from the SM's limits (shared memory with its per-block
                // reservation, registers per warp, threads, TMEM columns); the
                // smaller of the variant's two forms.
                cudaFuncAttributes fa;
                if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess) return W4A16_ERR_CUDA;
                int smem_sm = 0, resv = 0, regs_sm = 0, threads_sm = 0;
                cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
                cudaDeviceGetAttribute(&resv, cudaDevAttrReservedSharedMemoryPerBlock, dev);
                cudaDeviceGetAttribute(&regs_sm, cudaDevAttrMaxRegistersPerMultiprocessor, dev);
                cudaDeviceGetAttribute(&threads_sm, cudaDevAttrMaxThreadsPerMultiProcessor, dev);
                const int per_warp_regs = ((fa.numRegs * 32 + 255) / 256) * 256;
                n = std::min(n, smem_sm / (v.smem + static_cast<int>(fa.sharedSizeBytes) + resv));
                n = std::min(n, regs_sm / (per_warp_regs * (v.threads / 32)));
                n = std::min(n, threads_sm / v.threads);
                n = std::min(n, 512 / v.tmem_cols);  // every resident CTA holds its TMEM columns
            }
            if (n < 1) return W4A16_ERR_UNSUPPORTED;
            st.ctas_per_sm[kind][i] = n;
        }
        st.ready[kind] = true;
    }
    *out = &st;
    return W4A16_OK;
}

int variant_index(int bn) {
    for (int i = 0; i < kNumVariants; ++i)
        if (kVariants[i].bn == bn) return i;
    return kNumVariants - 1;
}

int launch_kind(Kind kind, int bn, const CUtensorMap& map, const Params& p, dim3 grid, int cluster_x,
                cudaStream_t stream) {
    const int vi = variant_index(bn);
    return kernel_of(kind, vi, p.G % kTileK ? 1 : 0).launch(map, p, grid, cluster_x, kVariants[vi].smem, stream);
}

int token_tile_for(int64_t rows_per_tile) {
    if (rows_per_tile <= 16) return 16;
    if (rows_per_tile <= 32) return 32;
    if (rows_per_tile <= 64) return 64;
    if (rows_per_tile <= 128) return 128;
    if (rows_per_tile <= 192) return 192;
    return 256;
}


struct Plan {
    int bn;
    int splits;
    dim3 grid;
    int smem;
    int ctas_per_sm;
};

// bn_force / splits_force > 0 select a tactic's token tile and K split (the
// split only with a single token tile, a power of two that leaves every
// cluster rank at least two K stages); 0 takes the heuristic.
int plan_dense(int64_t M, int64_t N, int64_t K, Plan* plan, bool need_device, int bn_force = 0,
               int splits_force = 0, Kind kind = kInt4) {
    const int bn = bn_force > 0 ? bn_force : token_tile_for(M);
    if (variant_for(bn).bn != bn) return W4A16_ERR_UNSUPPORTED;
    const int vi = variant_index(bn);
    int per_sm = kVariants[vi].nominal_per_sm, sms = 148;
    if (need_device) {
        DeviceState* st = nullptr;
        int rc = prepare_device(kind, &st);
        if (rc) return rc;
        per_sm = st->ctas_per_sm[kind][vi];
        sms = sm_count();
    }
    const int cols = kind == kGatedInt4 ? kTileN / 2 : kTileN;  // output columns of a CTA
    const int64_t NT = (N + cols - 1) / cols;
    const int64_t MT = (M + bn - 1) / bn;
    const int64_t KT = (K + kTileK - 1) / kTileK;
    if (NT > 65535 || MT > 65535) return W4A16_ERR_UNSUPPORTED;
    int splits = 1;
    if (splits_force > 0) {
        if ((splits_force & (splits_force - 1)) || splits_force > 8 ||
            (splits_force > 1 && (MT != 1 || KT < 2 * splits_force)))
            return W4A16_ERR_UNSUPPORTED;
        splits = splits_force;
    } else if (MT == 1) {
        const int64_t slots = static_cast<int64_t>(sms) * per_sm;
        while (splits < 8 && NT * splits * 2 <= slots && KT >= splits * 4) splits *= 2;
    }
    plan->bn = bn;
    plan->splits = splits;
    plan->grid = dim3(static_cast<unsigned>(splits), static_cast<unsigned>(NT), static_cast<unsigned>(MT));
    plan->smem = kVariants[vi].smem;
    plan->ctas_per_sm = per_sm;
    return W4A16_OK;
}

int plan_grouped(int64_t E, int64_t total_rows, int64_t N, int64_t K, Plan* plan, bool need_device) {
    // Token tile sized for an expert's average row count with headroom, so that
    // most experts need one tile; each tile's MMA covers only its valid rows
    // rounded up to 16.
    const int64_t avg = (total_rows + E - 1) / E;
    const int bn = token_tile_for(avg + avg / 4);
    const int vi = variant_index(bn);
    int per_sm = kVariants[vi].nominal_per_sm;
    if (need_device) {
        DeviceState* st = nullptr;
        int rc = prepare_device(kInt4, &st);
        if (rc) return rc;
        per_sm = st->ctas_per_sm[kInt4][vi];
    }
    const int64_t NT = (N + kTileN - 1) / kTileN;
    const int64_t slots = total_rows / bn + E;  // >= sum over experts of ceil(rows_e / bn)
    if (NT > 65535 || slots > 65535) return W4A16_ERR_UNSUPPORTED;
    (void)K;
    plan->bn = bn;
    plan->splits = 1;
    plan->grid = dim3(1, static_cast<unsigned>(NT), static_cast<unsigned>(slots));
    plan->smem = kVariants[vi].smem;
    plan->ctas_per_sm = per_sm;
    return W4A16_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

void fill_info(const Plan& plan, w4a16_launch_info* info) {
    info->token_tile = plan.bn;
    info->k_splits = plan.splits;
    info->grid_x = static_cast<int32_t>(plan.grid.x);
    info->grid_y = static_cast<int32_t>(plan.grid.y);
    info->grid_z = static_cast<int32_t>(plan.grid.z);
    info->threads_per_cta = variant_for(plan.bn).threads;
    info->smem_bytes = plan.smem;
    info->ctas_per_sm = plan.ctas_per_sm;
}

// ---------------------------------------------------------------- tactics
// A tactic is one launch form of w4a16_gemm for a shape (the plugin page's
// getValidTactics / setTactic): the skinny kernel with a given K split, K
// halves and ring depth (M <= 16 only), or the tensor-core kernel with a given
// token tile and K split. Ids are 1-based positions in the shape's list of
// valid forms, skinny forms first; 0 means the built-in heuristic.
struct Choice {
    bool skinny;
    SkinnyPlan sk;
    Plan tc;
};

constexpr int kTileChoices[] = {16, 32, 64, 128, 192, 256};

void enumerate_tactics(int64_t M, int64_t N, int64_t K, int64_t G, bool need_device, Choice* out, int* count,
                       int capacity) {
    int n = 0;
    auto push = [&](const Choice& c) {
        if (n < capacity) out[n] = c;
        ++n;
    };
    if (M <= kSkinnyMaxM) {
        for (int kh = 1; kh <= 2; ++kh)
            for (int splits = 1; splits <= 8; ++splits)
                for (int deep = 0; deep <= 1; ++deep) {
                    Choice c{};
                    c.skinny = true;
                    if (skinny_plan_fill(M, N, K, G, splits, kh, deep, &c.sk) == W4A16_OK) push(c);
                }
    }
    for (int bn : kTileChoices)
        for (int splits = 1; splits <= 8; splits *= 2) {
            Choice c{};
            c.skinny = false;
            if (plan_dense(M, N, K, &c.tc, need_device, bn, splits) == W4A16_OK) push(c);
        }
    *count = n;
}

constexpr int kMaxTactics = 96;

int tactic_choice(int64_t M, int64_t N, int64_t K, int64_t G, int tactic, bool need_device, Choice* out) {
    Choice all[kMaxTactics];
    int n = 0;
    enumerate_tactics(M, N, K, G, need_device, all, &n, kMaxTactics);
    if (tactic < 1 || tactic > n || tactic > kMaxTactics) return W4A16_ERR_INVALID_ARG;
    *out = all[tactic - 1];
    return W4A16_OK;
}

struct TacticKey {
    int dev;
    int64_t M, N, K, G;
    bool operator==(const TacticKey& o) const {
        return dev == o.dev && M == o.M && N == o.N && K == o.K && G == o.G;
    }
};
struct TacticKeyHash {
    size_t operator()(const TacticKey& k) const {
        uint64_t h = static_cast<uint64_t>(k.dev) * 0x9E3779B97F4A7C15ull;
        for (int64_t v : {k.M, k.N, k.K, k.G}) h = (h ^ static_cast<uint64_t>(v)) * 0x100000001B3ull;
        return static_cast<size_t>(h);
    }
};
struct TacticEntry {
    int tactic;
    Choice choice;
};

std::mutex g_tactic_mu;
std::unordered_map<TacticKey, TacticEntry, TacticKeyHash> g_tactics;
std::atomic<int> g_tactic_count{0};  // lets the GEMM skip the lookup while the table is empty

int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

// The table's choice for a shape on the current device, if it holds one.
bool lookup_tactic(int64_t M, int64_t N, int64_t K, int64_t G, Choice* out, int* tactic) {
    if (g_tactic_count.load(std::memory_order_acquire) == 0) return false;
    const TacticKey key{current_device(), M, N, K, G};
    std::lock_guard<std::mutex> lock(g_tactic_mu);
    auto it = g_tactics.find(key);
    if (it == g_tactics.end()) return false;
    *out = it->second.choice;
    if (tactic) *tactic = it->second.tactic;
    return true;
}

void store_tactic(int64_t M, int64_t N, int64_t K, int64_t G, int tactic, const Choice& c) {
    const TacticKey key{current_device(), M, N, K, G};
    std::lock_guard<std::mutex> lock(g_tactic_mu);
    if (tactic == 0) {
        g_tactics.erase(key);
    } else {
        g_tactics[key] = TacticEntry{tactic, c};
    }
    g_tactic_count.store(static_cast<int>(g_tactics.size()), std::memory_order_release);
}

// The table's tactic for the shape, else the heuristic: the skinny kernel for
// decode-sized M, the tensor-core kernel otherwise.
int choose(int64_t M, int64_t N, int64_t K, int64_t G, bool need_device, Choice* c) {
    if (lookup_tactic(M, N, K, G, c, nullptr)) return W4A16_OK;
    c->skinny = skinny_plan(M, N, K, G, &c->sk) == W4A16_OK;
    if (c->skinny) return W4A16_OK;
    return plan_dense(M, N, K, &c->tc, need_device);
}

void fill_info_skinny(const SkinnyPlan& sk, w4a16_launch_info* info) {
    info->token_tile = 8 * sk.mt;
    info->k_splits = sk.splits;
    info->grid_x = sk.grid_x;
    info->grid_y = sk.grid_y;
    info->grid_z = 1;
    info->threads_per_cta = sk.threads;
    info->smem_bytes = sk.smem;
    info->ctas_per_sm = (228 * 1024) / (sk.smem + 1024) < 2 ? (228 * 1024) / (sk.smem + 1024) : 2;
}

}  // namespace

int launch_choice(const Choice& c, const w4a16_half* A_dev, const uint8_t* Wt_dev, const w4a16_half* S_dev,
                  w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G, cudaStream_t stream);
int dense_launch(const Plan& plan, int bits, const w4a16_half* A_dev, const uint8_t* Wt_dev,
                 const w4a16_half* S_dev, w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G,
                 cudaStream_t stream);

int encode_activation_map(CUtensorMap* map, const void* A, int64_t rows, int64_t K, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return W4A16_ERR_CUDA;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * 2};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(kTileK), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(A), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? W4A16_OK : W4A16_ERR_CUDA;
}

int check_shape(int64_t N, int64_t K, int64_t G) {
    if (N <= 0 || K <= 0 || G <= 0) return W4A16_ERR_INVALID_ARG;
    if (N % 8 || K % 8 || G % 16) return W4A16_ERR_UNSUPPORTED;
    if (N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    return W4A16_OK;
}

int activation_map(CUtensorMap* map, const void* A, int64_t rows, int64_t K, int box_rows) {
    // A small per-thread cache: the encoder costs more than the rest of a
    // decode-sized call on the host, and the same activation buffers recur.
    struct Entry {
        const void* A;
        int64_t rows, K;
        int box, dev;
        CUtensorMap map;
    };
    constexpr int kEntries = 16;
    thread_local Entry cache[kEntries];
    thread_local int used = 0, next = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return W4A16_ERR_CUDA;
    for (int i = 0; i < used; ++i) {
        const Entry& e = cache[i];
        if (e.A == A && e.rows == rows && e.K == K && e.box == box_rows && e.dev == dev) {
            *map = e.map;
            return W4A16_OK;
        }
    }
    const int rc = encode_activation_map(map, A, rows, K, box_rows);
    if (rc) return rc;
    Entry& e = cache[next];
    e.A = A;
    e.rows = rows;
    e.K = K;
    e.box = box_rows;
    e.dev = dev;
    e.map = *map;
    next = (next + 1) % kEntries;
    if (used < kEntries) ++used;
    return W4A16_OK;
}

int make_half_map_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes,
                     uint32_t box_inner, uint32_t box_outer) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return W4A16_ERR_CUDA;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? W4A16_OK : W4A16_ERR_CUDA;
}

int check_device() {
    // per device: 0 unknown, 1 supported, 2 not (cached: this runs on every call)
    static std::atomic<int> state[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return W4A16_ERR_UNSUPPORTED;
    }
    if (dev < 0 || dev >= 64) return W4A16_ERR_UNSUPPORTED;
    int st = state[dev].load(std::memory_order_acquire);
    if (st == 0) {
        int major = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
            cudaGetLastError();
            return W4A16_ERR_UNSUPPORTED;
        }
        st = (major == 10) ? 1 : 2;
        state[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? W4A16_OK : W4A16_ERR_UNSUPPORTED;
}

namespace {
std::atomic<int> g_static_weights{0};
std::atomic<long long> g_wait_limit{kTimeoutCycles};  // test aid: w4a16_set_fault_injection
std::atomic<int> g_stall_stage{-1};
}

long long device_wait_limit() { return g_wait_limit.load(std::memory_order_relaxed); }
int injected_stall_stage() { return g_stall_stage.load(std::memory_order_relaxed); }

// Set by the entry points with per-call flags for the duration of one call on this host thread.
thread_local int t_call_static_weights = 0;

bool static_weights_enabled() {
    return t_call_static_weights != 0 || g_static_weights.load(std::memory_order_relaxed) != 0;
}

int sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    n = cached[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" const char* w4a16_status_string(int status) {
    switch (status) {
        case W4A16_OK: return "ok";
        case W4A16_ERR_INVALID_ARG: return "invalid argument";
        case W4A16_ERR_MISALIGNED: return "pointer not 16-byte aligned";
        case W4A16_ERR_UNSUPPORTED: return "unsupported shape or device";
        case W4A16_ERR_CUDA: return "CUDA runtime error";
        case W4A16_ERR_TIMEOUT: return "bounded device wait ran out";
        case W4A16_ERR_BAD_OFFSETS: return "malformed expert offsets";
        case W4A16_ERR_BAD_ROUTING: return "expert id or gathered-row index out of range";
        case W4A16_ERR_SCRATCH_TOO_SMALL: return "shape needs more than the static scratch of the no-allocation entry point";
        case W4A16_ERR_BAD_ADAPTER: return "adapter index out of range";
        default: return "unknown status";
    }
}

extern "C" int w4a16_set_static_weights(int enable) {
    const int previous = g_static_weights.exchange(enable ? 1 : 0);
    return previous;
}

extern "C" int w4a16_gemm_launch_info(int64_t M, int64_t N, int64_t K, int64_t G, w4a16_launch_info* info) {
    if (!info || M <= 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    const bool dev = check_device() == W4A16_OK;
    Choice c;
    rc = choose(M, N, K, G, dev, &c);
    if (rc) return rc;
    if (c.skinny)
        fill_info_skinny(c.sk, info);
    else
        fill_info(c.tc, info);
    return W4A16_OK;
}

extern "C" int w4a16_grouped_launch_info(int64_t E, int64_t total_rows, int64_t N, int64_t K, int64_t G,
                                         w4a16_launch_info* info) {
    if (!info || E <= 0 || E > W4A16_MAX_EXPERTS || total_rows <= 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (total_rows >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    const bool dev = check_device() == W4A16_OK;
    SkinnyPlan sk;
    if (skinny_plan_grouped(total_rows, N, K, G, &sk) == W4A16_OK) {
        fill_info_skinny(sk, info);
        info->grid_z = static_cast<int32_t>(E);
        return W4A16_OK;
    }
    Plan plan;
    rc = plan_grouped(E, total_rows, N, K, &plan, dev);
    if (rc) return rc;
    fill_info(plan, info);
    return W4A16_OK;
}

extern "C" int w4a16_gemm(const w4a16_half* A_dev, const uint8_t* Wt_dev, const w4a16_half* S_dev,
                          w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G, void* stream) {
    if (!A_dev || !Wt_dev || !S_dev || !C_dev || M < 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    if (!aligned16(A_dev) || !aligned16(Wt_dev) || !aligned16(S_dev) ||
        (reinterpret_cast<uintptr_t>(C_dev) & 1u))
        return W4A16_ERR_MISALIGNED;
    if (M == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    Choice c;
    rc = choose(M, N, K, G, true, &c);
    if (rc) return rc;
    return launch_choice(c, A_dev, Wt_dev, S_dev, C_dev, M, N, K, G, static_cast<cudaStream_t>(stream));
}

namespace w4a16 {

int launch_choice(const Choice& c, const w4a16_half* A_dev, const uint8_t* Wt_dev, const w4a16_half* S_dev,
                  w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G, cudaStream_t stream) {
    if (c.skinny) return skinny_launch(c.sk, A_dev, Wt_dev, S_dev, C_dev, M, N, K, G, stream);
    return dense_launch(c.tc, 4, A_dev, Wt_dev, S_dev, C_dev, M, N, K, G, stream);
}

// The tensor-core kernel on a dense product, int4 (bits = 4) or 8-bit codes.
int dense_launch(const Plan& plan, int bits, const w4a16_half* A_dev, const uint8_t* Wt_dev,
                 const w4a16_half* S_dev, w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G,
                 cudaStream_t stream) {
    int rc;
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.wt[0] = Wt_dev;
    p.sc[0] = reinterpret_cast<const __half*>(S_dev);
    p.offsets = nullptr;
    p.C = reinterpret_cast<__half*>(C_dev);
    p.rows = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + kTileK - 1) / kTileK);
    p.E = 1;
    p.splits = plan.splits;
    p.grouped = 0;
    p.prefetch = static_weights_enabled() ? 1 : 0;
    p.vec_out = (N % 8) == 0 && aligned16(C_dev);
    p.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
    p.stall_stage = g_stall_stage.load(std::memory_order_relaxed);

    CUtensorMap map;
    rc = activation_map(&map, A_dev, M, K, plan.bn);
    if (rc) return rc;
    return launch_kind(bits == 8 ? kInt8 : kInt4, plan.bn, map, p, plan.grid, plan.splits, stream);
}

}  // namespace w4a16

namespace w4a16 {

int grouped_gemm_act(const w4a16_half* A_dev, const uint8_t* const* Wt, const w4a16_half* const* S,
                     const int32_t* offsets_dev, w4a16_half* C_dev, int64_t E, int64_t total_rows, int64_t N,
                     int64_t K, int64_t G, int act, cudaStream_t stream) {
    if (!A_dev || !Wt || !S || !offsets_dev || !C_dev || E <= 0 || E > W4A16_MAX_EXPERTS || total_rows < 0)
        return W4A16_ERR_INVALID_ARG;
    if (act < W4A16_ACT_IDENTITY || act > W4A16_ACT_GELU_TANH) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (total_rows >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    for (int64_t e = 0; e < E; ++e) {
        if (!Wt[e] || !S[e]) return W4A16_ERR_INVALID_ARG;
        if (!aligned16(Wt[e]) || !aligned16(S[e])) return W4A16_ERR_MISALIGNED;
    }
    if (!aligned16(A_dev) || (reinterpret_cast<uintptr_t>(C_dev) & 1u) ||
        (reinterpret_cast<uintptr_t>(offsets_dev) & 3u))
        return W4A16_ERR_MISALIGNED;
    if (total_rows == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    SkinnyPlan sk;
    if (skinny_plan_grouped(total_rows, N, K, G, &sk) == W4A16_OK)  // decode-sized batches: at most 16 rows in all
        return skinny_grouped_launch(sk, A_dev, Wt, reinterpret_cast<const void* const*>(S), offsets_dev, C_dev, E,
                                     total_rows, N, K, G, act, stream);
    Plan plan;
    rc = plan_grouped(E, total_rows, N, K, &plan, true);
    if (rc) return rc;

    Params p;
    std::memset(&p, 0, sizeof(p));
    for (int64_t e = 0; e < E; ++e) {
        p.wt[e] = Wt[e];
        p.sc[e] = reinterpret_cast<const __half*>(S[e]);
    }
    p.offsets = offsets_dev;
    p.C = reinterpret_cast<__half*>(C_dev);
    p.rows = static_cast<int32_t>(total_rows);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + kTileK - 1) / kTileK);
    p.E = static_cast<int32_t>(E);
    p.splits = 1;
    p.grouped = 1;
    p.vec_out = (N % 8) == 0 && aligned16(C_dev);
    p.prefetch = 0;  // expert weights are read only after the offsets, which follow the wait
    p.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
    p.stall_stage = g_stall_stage.load(std::memory_order_relaxed);
    p.act = act;

    CUtensorMap map;
    rc = activation_map(&map, A_dev, total_rows, K, plan.bn);
    if (rc) return rc;
    return launch_kind(kInt4, plan.bn, map, p, plan.grid, 1, stream);
}

}  // namespace w4a16

namespace w4a16 {

int lora_plan(int64_t M, int64_t N, int64_t K, int64_t G, LoraPlan* plan) {
    plan->tile_rows = 0;
    if (decode_takes(M, N, K, G)) return W4A16_OK;
    Plan tc;
    const int rc = plan_dense(M, N, K, &tc, true, 0, 0, kLoraInt4);
    if (rc) return rc;
    plan->tile_rows = tc.bn;
    plan->splits = tc.splits;
    plan->grid_y = static_cast<int>(tc.grid.y);
    plan->grid_z = static_cast<int>(tc.grid.z);
    return W4A16_OK;
}

int lora_product(const LoraPlan& plan, const LoraOperands& lora, const w4a16_half* A, const uint8_t* Wt,
                 const w4a16_half* S, w4a16_half* C, int64_t M, int64_t N, int64_t K, int64_t G,
                 cudaStream_t stream) {
    if (plan.tile_rows == 0) return decode_lora_launch(lora, A, Wt, S, C, M, N, K, G, stream);
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.wt[0] = Wt;
    p.sc[0] = reinterpret_cast<const __half*>(S);
    p.C = reinterpret_cast<__half*>(C);
    p.rows = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + kTileK - 1) / kTileK);
    p.E = 1;
    p.splits = plan.splits;
    p.vec_out = aligned16(C);
    p.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
    p.stall_stage = g_stall_stage.load(std::memory_order_relaxed);
    p.lora = lora;
    CUtensorMap map;
    const int rc = encode_activation_map(&map, A, M, K, plan.tile_rows);
    if (rc) return rc;
    const dim3 grid(static_cast<unsigned>(plan.splits), static_cast<unsigned>(plan.grid_y),
                    static_cast<unsigned>(plan.grid_z));
    return launch_kind(kLoraInt4, plan.tile_rows, map, p, grid, plan.splits, stream);
}

namespace {

int gated_gemm(const w4a16_half* A_dev, const uint8_t* Wt_gate, const w4a16_half* S_gate, const uint8_t* Wt_up,
               const w4a16_half* S_up, w4a16_half* H_dev, w4a16_half* Pg_dev, w4a16_half* Pu_dev, int64_t M, int64_t N,
               int64_t K, int64_t G, int act, cudaStream_t stream) {
    if (decode_takes(M, N, K, G))
        return decode_gated_launch(A_dev, Wt_gate, S_gate, Wt_up, S_up, H_dev, Pg_dev, Pu_dev, M, N, K, G, act, stream);
    Plan plan;
    int rc = plan_dense(M, N, K, &plan, true, 0, 0, kGatedInt4);
    if (rc) return rc;
    if (wide_gated_takes(M, N, K, G, plan.bn, plan.splits, plan.ctas_per_sm))
        return wide_gated_launch(A_dev, Wt_gate, S_gate, Wt_up, S_up, H_dev, Pg_dev, Pu_dev, M, N, K, G, act, stream);
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.wt[0] = Wt_gate;
    p.wt[1] = Wt_up;
    p.sc[0] = reinterpret_cast<const __half*>(S_gate);
    p.sc[1] = reinterpret_cast<const __half*>(S_up);
    p.C = reinterpret_cast<__half*>(H_dev);
    p.Pg = reinterpret_cast<__half*>(Pg_dev);
    p.Pu = reinterpret_cast<__half*>(Pu_dev);
    p.rows = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + kTileK - 1) / kTileK);
    p.E = 1;
    p.splits = plan.splits;
    p.act = act;
    p.prefetch = static_weights_enabled() ? 1 : 0;
    p.vec_out = aligned16(H_dev) && aligned16(Pg_dev) && aligned16(Pu_dev);
    p.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
    p.stall_stage = g_stall_stage.load(std::memory_order_relaxed);
    CUtensorMap map;
    rc = encode_activation_map(&map, A_dev, M, K, plan.bn);
    if (rc) return rc;
    return launch_kind(kGatedInt4, plan.bn, map, p, plan.grid, plan.splits, stream);
}

}  // namespace
}  // namespace w4a16

extern "C" int w4a16_gated_gemm(const w4a16_half* A_dev, const uint8_t* Wt_gate_dev, const w4a16_half* S_gate_dev,
                                const uint8_t* Wt_up_dev, const w4a16_half* S_up_dev, w4a16_half* H_dev,
                                w4a16_half* Pg_dev, w4a16_half* Pu_dev, int64_t M, int64_t N, int64_t K, int64_t G,
                                int act, uint32_t flags, void* stream) {
    if (!A_dev || !Wt_gate_dev || !S_gate_dev || !Wt_up_dev || !S_up_dev || !H_dev || M < 0)
        return W4A16_ERR_INVALID_ARG;
    if ((Pg_dev == nullptr) != (Pu_dev == nullptr)) return W4A16_ERR_INVALID_ARG;
    if (act < W4A16_ACT_IDENTITY || act > W4A16_ACT_SILU) return W4A16_ERR_INVALID_ARG;
    if (flags & ~static_cast<uint32_t>(W4A16_FLAG_STATIC_WEIGHTS)) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    if (!aligned16(A_dev) || !aligned16(Wt_gate_dev) || !aligned16(S_gate_dev) || !aligned16(Wt_up_dev) ||
        !aligned16(S_up_dev) ||
        ((reinterpret_cast<uintptr_t>(H_dev) | reinterpret_cast<uintptr_t>(Pg_dev) |
          reinterpret_cast<uintptr_t>(Pu_dev)) & 1u))
        return W4A16_ERR_MISALIGNED;
    if (M == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    const CallStaticWeights scope((flags & W4A16_FLAG_STATIC_WEIGHTS) != 0);
    return gated_gemm(A_dev, Wt_gate_dev, S_gate_dev, Wt_up_dev, S_up_dev, H_dev, Pg_dev, Pu_dev, M, N, K, G, act,
                      static_cast<cudaStream_t>(stream));
}

extern "C" int w4a16_grouped_gemm(const w4a16_half* A_dev, const uint8_t* const* Wt, const w4a16_half* const* S,
                                  const int32_t* offsets_dev, w4a16_half* C_dev, int64_t E, int64_t total_rows,
                                  int64_t N, int64_t K, int64_t G, void* stream) {
    return grouped_gemm_act(A_dev, Wt, S, offsets_dev, C_dev, E, total_rows, N, K, G, W4A16_ACT_IDENTITY,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int w4a16_grouped_gemm_act(const w4a16_half* A_dev, const uint8_t* const* Wt,
                                      const w4a16_half* const* S, const int32_t* offsets_dev, w4a16_half* C_dev,
                                      int64_t E, int64_t total_rows, int64_t N, int64_t K, int64_t G, int act,
                                      void* stream) {
    return grouped_gemm_act(A_dev, Wt, S, offsets_dev, C_dev, E, total_rows, N, K, G, act,
                            static_cast<cudaStream_t>(stream));
}

extern "C" int w4a16_device_status(int clear) {
    if (check_device() != W4A16_OK) return W4A16_ERR_CUDA;
    if (cudaDeviceSynchronize() != cudaSuccess) return W4A16_ERR_CUDA;
    const int v = read_gemm_status(clear != 0);
    const int vf = forms_device_status(clear != 0);
    const int vs = skinny_device_status(clear != 0);
    const int vq = quant_device_status(clear != 0);
    const int vm = moe_device_status(clear != 0);
    const int vd = dgrad_device_status(clear != 0);
    const int vl = lora_device_status(clear != 0);
    const int vx = decode_device_status(clear != 0);
    if (v < 0 || vf < 0 || vs < 0 || vq < 0 || vm < 0 || vd < 0 || vl < 0 || vx < 0) return W4A16_ERR_CUDA;
    for (int x : {v, vf, vs, vq, vm, vd, vx})
        if (x != 0) return x;
    return vl;
}

extern "C" int w4a16_set_fault_injection(int64_t stall_stage, int64_t wait_limit_cycles) {
    g_stall_stage.store(stall_stage < 0 || stall_stage > (1 << 30) ? -1 : static_cast<int>(stall_stage));
    g_wait_limit.store(wait_limit_cycles > 0 ? static_cast<long long>(wait_limit_cycles) : kTimeoutCycles);
    return W4A16_OK;
}

// ---------------------------------------------------------------- tactics
extern "C" int w4a16_get_valid_tactics(int64_t M, int64_t N, int64_t K, int64_t G, int32_t* tactics,
                                       int32_t capacity, int32_t* count) {
    if (!count || M <= 0 || capacity < 0 || (capacity > 0 && !tactics)) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    Choice all[kMaxTactics];
    int n = 0;
    enumerate_tactics(M, N, K, G, check_device() == W4A16_OK, all, &n, kMaxTactics);
    n = std::min(n, kMaxTactics);
    for (int i = 0; i < n && i < capacity; ++i) tactics[i] = i + 1;
    *count = n;
    return W4A16_OK;
}

extern "C" int w4a16_tactic_launch_info(int64_t M, int64_t N, int64_t K, int64_t G, int32_t tactic,
                                        w4a16_launch_info* info) {
    if (!info || M <= 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    Choice c;
    rc = tactic_choice(M, N, K, G, tactic, check_device() == W4A16_OK, &c);
    if (rc) return rc;
    if (c.skinny)
        fill_info_skinny(c.sk, info);
    else
        fill_info(c.tc, info);
    return W4A16_OK;
}

extern "C" int w4a16_set_tactic(int64_t M, int64_t N, int64_t K, int64_t G, int32_t tactic) {
    if (M <= 0 || tactic < 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    Choice c{};
    if (tactic > 0) {
        rc = tactic_choice(M, N, K, G, tactic, check_device() == W4A16_OK, &c);
        if (rc) return rc;
    }
    store_tactic(M, N, K, G, tactic, c);
    return W4A16_OK;
}

extern "C" int w4a16_get_tactic(int64_t M, int64_t N, int64_t K, int64_t G, int32_t* tactic) {
    if (!tactic) return W4A16_ERR_INVALID_ARG;
    Choice c;
    int t = 0;
    *tactic = lookup_tactic(M, N, K, G, &c, &t) ? t : 0;
    return W4A16_OK;
}

extern "C" int w4a16_clear_tactics(void) {
    std::lock_guard<std::mutex> lock(g_tactic_mu);
    g_tactics.clear();
    g_tactic_count.store(0, std::memory_order_release);
    return W4A16_OK;
}

extern "C" int w4a16_autotune(const w4a16_half* A_dev, const uint8_t* const* Wt, const w4a16_half* const* S,
                              int32_t copies, w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G,
                              int32_t reps, int32_t* best_tactic, float* best_us, float* times_us,
                              int32_t times_capacity, void* stream) {
    if (!A_dev || !Wt || !S || !C_dev || !best_tactic || M <= 0 || copies < 1 || copies > 1024 || reps < 1 ||
        reps > 10000 || times_capacity < 0 || (times_capacity > 0 && !times_us))
        return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    for (int32_t c = 0; c < copies; ++c) {
        if (!Wt[c] || !S[c]) return W4A16_ERR_INVALID_ARG;
        if (!aligned16(Wt[c]) || !aligned16(S[c])) return W4A16_ERR_MISALIGNED;
    }
    if (!aligned16(A_dev) || (reinterpret_cast<uintptr_t>(C_dev) & 1u)) return W4A16_ERR_MISALIGNED;
    rc = check_device();
    if (rc) return rc;
    Choice all[kMaxTactics];
    int n = 0;
    enumerate_tactics(M, N, K, G, true, all, &n, kMaxTactics);
    n = std::min(n, kMaxTactics);
    if (n == 0) return W4A16_ERR_UNSUPPORTED;

    // Each tactic's `reps` launches, rotating over the weight copies, are
    // recorded on a private stream into a CUDA graph and replayed on the
    // caller's stream: back to back, as a model's layers run them, with the
    // launch overlap that programmatic dependent launch gives.
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStream_t cap = nullptr;
    cudaEvent_t e0 = nullptr, e1 = nullptr;
    if (cudaStreamCreateWithFlags(&cap, cudaStreamNonBlocking) != cudaSuccess) return W4A16_ERR_CUDA;
    if (cudaEventCreate(&e0) != cudaSuccess || cudaEventCreate(&e1) != cudaSuccess) {
        if (e0) cudaEventDestroy(e0);
        cudaStreamDestroy(cap);
        return W4A16_ERR_CUDA;
    }
    float best = 0.f;
    int best_id = 0;
    for (int i = 0; i < n && rc == W4A16_OK; ++i) {
        rc = launch_choice(all[i], A_dev, Wt[0], S[0], C_dev, M, N, K, G, st);  // first use outside the graph
        if (rc == W4A16_OK && cudaStreamSynchronize(st) != cudaSuccess) rc = W4A16_ERR_CUDA;
        if (rc) break;
        cudaGraph_t graph = nullptr;
        cudaGraphExec_t exec = nullptr;
        if (cudaStreamBeginCapture(cap, cudaStreamCaptureModeThreadLocal) != cudaSuccess) {
            rc = W4A16_ERR_CUDA;
            break;
        }
        int lrc = W4A16_OK;
        for (int r = 0; r < reps && lrc == W4A16_OK; ++r)
            lrc = launch_choice(all[i], A_dev, Wt[r % copies], S[r % copies], C_dev, M, N, K, G, cap);
        const cudaError_t ce = cudaStreamEndCapture(cap, &graph);
        if (lrc != W4A16_OK || ce != cudaSuccess || cudaGraphInstantiate(&exec, graph, 0) != cudaSuccess) {
            rc = lrc != W4A16_OK ? lrc : W4A16_ERR_CUDA;
        } else {
            float ms = 0.f, best_ms = 0.f;
            // one warm replay, then the fastest of three timed ones
            if (cudaGraphLaunch(exec, st) != cudaSuccess) rc = W4A16_ERR_CUDA;
            for (int t = 0; t < 3 && rc == W4A16_OK; ++t) {
                if (cudaEventRecord(e0, st) != cudaSuccess || cudaGraphLaunch(exec, st) != cudaSuccess ||
                    cudaEventRecord(e1, st) != cudaSuccess || cudaEventSynchronize(e1) != cudaSuccess ||
                    cudaEventElapsedTime(&ms, e0, e1) != cudaSuccess) {
                    rc = W4A16_ERR_CUDA;
                    break;
                }
                if (t == 0 || ms < best_ms) best_ms = ms;
            }
            const float us = best_ms * 1000.f / static_cast<float>(reps);
            if (i < times_capacity) times_us[i] = us;
            if (rc == W4A16_OK && (best_id == 0 || us < best)) {
                best = us;
                best_id = i + 1;
            }
        }
        if (exec) cudaGraphExecDestroy(exec);
        if (graph) cudaGraphDestroy(graph);
    }
    cudaEventDestroy(e0);
    cudaEventDestroy(e1);
    cudaStreamDestroy(cap);
    if (rc) return rc;
    store_tactic(M, N, K, G, best_id, all[best_id - 1]);
    *best_tactic = best_id;
    if (best_us) *best_us = best;
    return W4A16_OK;
}

// ---------------------------------------------------------------- W8A16
extern "C" int w8a16_gemm_launch_info(int64_t M, int64_t N, int64_t K, int64_t G, w4a16_launch_info* info) {
    if (!info || M <= 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    Plan plan;
    rc = plan_dense(M, N, K, &plan, check_device() == W4A16_OK, 0, 0, kInt8);
    if (rc) return rc;
    fill_info(plan, info);
    return W4A16_OK;
}

extern "C" int w8a16_gemm(const w4a16_half* A_dev, const uint8_t* Wt8_dev, const w4a16_half* S_dev,
                          w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G, void* stream) {
    if (!A_dev || !Wt8_dev || !S_dev || !C_dev || M < 0) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    if (!aligned16(A_dev) || !aligned16(Wt8_dev) || !aligned16(S_dev) ||
        (reinterpret_cast<uintptr_t>(C_dev) & 1u))
        return W4A16_ERR_MISALIGNED;
    if (M == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    Plan plan;
    rc = plan_dense(M, N, K, &plan, true, 0, 0, kInt8);
    if (rc) return rc;
    return dense_launch(plan, 8, A_dev, Wt8_dev, S_dev, C_dev, M, N, K, G, static_cast<cudaStream_t>(stream));
}

extern "C" int w4a16_gemm_ex(const w4a16_half* A_dev, const uint8_t* Wt_dev, const w4a16_half* S_dev,
                             w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G, uint32_t flags,
                             void* stream) {
    if (flags & ~static_cast<uint32_t>(W4A16_FLAG_STATIC_WEIGHTS)) return W4A16_ERR_INVALID_ARG;
    const CallStaticWeights scope((flags & W4A16_FLAG_STATIC_WEIGHTS) != 0);
    return w4a16_gemm(A_dev, Wt_dev, S_dev, C_dev, M, N, K, G, stream);
}
