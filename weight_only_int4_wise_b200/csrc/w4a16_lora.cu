// Low-rank adapters of many requests beside one shared 4-bit projection:
//     C[m] = fp16( A[m] W + scaling[i] * (A[m] LA[i]^T) LB[i]^T ),  i = ids[m],
// LA [L, R, K], LB [L, N, R] fp16, one adapter index per row (negative: none).
// (The Int4GroupwiseGemmPluginV2 page describes the shared projection only.)
//
// Two launches. The first, here, makes V[m, r] = scaling[i] * sum_k A[m, k]
// LA[i, r, k], summed in fp32 and rounded to fp16, the MMA's operand type (up to 2^-11
// of the adapter's part, as every weight of it already carries); the second is the
// shared product with V LB^T added to its fp32 sums before their one rounding
// (w4a16_decode.cu for M <= 16, w4a16_gemm_kernel.cuh above). Keeping V apart costs
// M * R * 2 bytes and a launch, and spares every column tile of the product the
// R * K products of its rows. The second launch starts as soon as this one's CTAs run: this kernel
// signals its dependents only after its own wait for the previous kernel, so
// whatever this call's caller wrote is complete by then, and the product waits
// for this kernel only where it reads V.
//
// down kernel: one CTA takes 16 rows, 8 * RT ranks and one distinct adapter of
// those rows at a time (grid y strides over them); its 16 (or 4) warps split K into
// 32-deep blocks, read both operands straight from global memory into MMA
// fragments (16 bytes per lane: inside a block the order of k is free as long
// as both operands use it), and add their fp32 partials in warp order through
// shared memory. It is
// bound by latency (two to eight rounds of loads per warp): 8.9 us cold at 16 tokens
// with 16 adapters of rank 64, 18.7 us in the narrow form at 2048 rows, where the two
// launches together take 8 us more than without an adapter. Extra CTAs behind the row
// groups list the distinct adapters of each token tile of the tensor-core product.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/w4a16.h"
#include "once.h"
#include "ptx.cuh"
#include "w4a16_internal.h"

namespace w4a16 {

namespace {

__device__ int g_lora_status;  // latched device-side error (0 = none)

constexpr int kRows = 16;

struct DownParams {
    const __half* A;
    const __half* LA;
    const int32_t* ids;
    const float* scaling;  // null: 1
    __half* V;             // [M, R]
    int32_t* list;         // [tiles][tile_rows] distinct adapters of each token tile
    int32_t* count;        // [tiles]
    int32_t M, K, L, R;
    int32_t groups;        // row groups of 16; CTAs behind them make the lists
    int32_t tile_rows;     // token tile of the product (0: no lists)
};

__device__ __forceinline__ int adapter_of(const DownParams& p, int m) {
    if (m >= p.M) return -1;
    const int id = p.ids[m];
    if (id >= p.L) {
        atomicCAS(&g_lora_status, 0, W4A16_ERR_BAD_ADAPTER);  // the row is computed without an adapter
        return -1;
    }
    return id;
}

// The distinct adapters of token tile z (at most 256 rows), in the order of their
// first rows: each warp's own by a match over its lanes, then, for those only,
// against the lists of the warps before it.
template <int W>
__device__ void list_adapters(const DownParams& p, int z, int* lists /* [8][32] */, int* counts /* [2][8] */) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kPer = W >= 8 ? 1 : 8 / W;  // 32-row sets of a warp: warp, warp + W, ...
    int id[kPer];
    uint32_t b[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int w = warp + x * W, r = w * 32 + lane;
        id[x] = w < 8 && r < p.tile_rows ? adapter_of(p, z * p.tile_rows + r) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, id[x]);
        const bool first = id[x] >= 0 && (same & ((1u << lane) - 1u)) == 0;
        b[x] = __ballot_sync(0xffffffffu, first);
        if (w < 8) {
            lists[w * 32 + lane] = -1;
            __syncwarp();
            if (first) lists[w * 32 + __popc(b[x] & ((1u << lane) - 1u))] = id[x];
            if (lane == 0) counts[w] = __popc(b[x]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int w = warp + x * W;
        bool first = (b[x] >> lane) & 1u;
        if (w < 8 && b[x]) {
            for (int v = 0; v < w; ++v)
                for (int i = 0; i < counts[v]; i += 4) {  // (padded with -1)
                    const int4 l = *reinterpret_cast<const int4*>(lists + v * 32 + i);
                    first = first && l.x != id[x] && l.y != id[x] && l.z != id[x] && l.w != id[x];
                }
        }
        b[x] = __ballot_sync(0xffffffffu, first);
        if (w < 8 && lane == 0) counts[8 + w] = __popc(b[x]);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int w = warp + x * W;
        if (w >= 8) continue;
        int at = __popc(b[x] & ((1u << lane) - 1u));
        for (int v = 0; v < w; ++v) at += counts[8 + v];
        if ((b[x] >> lane) & 1u) p.list[static_cast<int64_t>(z) * p.tile_rows + at] = id[x];
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int v = 0; v < 8; ++v) n += counts[8 + v];
        p.count[z] = n;
    }
}

// W = 16 warps where this kernel's latency counts. With many row groups W = 4: small
// CTAs leave an SM soon, and the product's CTA (576 threads, 55 K registers) starts
// there while others still run; at 110 registers a thread it does not start beside one
// of them (bounded to 80 registers it would: 125 instead of 105 us with 8 adapters mixed
// over 2048 rows, 95 -> 108 us for a call alone, no gain for prompts). Narrow against wide
// form, 4096 -> 4096, rank 16: 1024 rows in prompts 36.2 / 38.3 us, 2048 75.1 / 74.6, with
// rank 64 84.5 / 83.0, one adapter for all 77.5 / 76.1, 8 mixed 105 / 101; 1100 rows ->
// 14336 138 / 139. (Both kernels ask for the largest shared-memory carve-out: an SM
// changes it only when it is empty.)
template <int RT, int W>
__global__ void __launch_bounds__(W * 32) lora_down_kernel(const DownParams p) {
    constexpr int kWarps = W, kThreads = W * 32;
    __shared__ __align__(16) float red[kWarps * kRows * 8 * RT];
    __shared__ int group_ids[kRows];
    grid_dependency_wait();    // the operands may come from the previous kernel
    __threadfence();
    grid_launch_dependents();  // (only now: the product's early loads rely on that kernel being complete)
    if (static_cast<int>(blockIdx.x) >= p.groups) {
        if (blockIdx.y == 0 && blockIdx.z == 0)
            list_adapters<W>(p, blockIdx.x - p.groups, reinterpret_cast<int*>(red), reinterpret_cast<int*>(red) + 256);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int m0 = blockIdx.x * kRows;
    const int r0 = blockIdx.z * 8 * RT;
    // Distinct adapters of the group: the lowest lane of each set of equal rows.
    const int mine = lane < kRows ? adapter_of(p, m0 + lane) : -1;
    const float my_scale = mine >= 0 && p.scaling ? p.scaling[mine] : 1.f;
    if (warp == 0 && lane < kRows) group_ids[lane] = mine;  // (read after the first barrier below)
    const uint32_t same = __match_any_sync(0xffffffffu, mine);
    uint32_t leaders = __ballot_sync(0xffffffffu, mine >= 0 && (same & ((1u << lane) - 1u)) == 0);
    for (int slot = 0; leaders; ++slot, leaders &= leaders - 1) {
        if (slot % static_cast<int>(gridDim.y) != static_cast<int>(blockIdx.y)) continue;
        const int id = __shfl_sync(0xffffffffu, mine, __ffs(leaders) - 1);
        const float s = __shfl_sync(0xffffffffu, my_scale, __ffs(leaders) - 1);
        float acc[RT][4];
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        // Rows of another adapter (or past M) read this adapter's first row along with
        // it, ranks past R the last rank; their sums are not written. (No load is
        // conditional: a branch around a load would wait for its value where the two
        // paths meet.)
        const int lead = __ffs(leaders) - 1;
        const int row0 = __shfl_sync(0xffffffffu, mine, g) == id ? g : lead;
        const int row1 = __shfl_sync(0xffffffffu, mine, g + 8) == id ? g + 8 : lead;
        const __half* a0 = p.A + static_cast<int64_t>(m0 + row0) * p.K + 8 * t;
        const __half* a1 = p.A + static_cast<int64_t>(m0 + row1) * p.K + 8 * t;
        const __half* lb[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j)
            lb[j] = p.LA + (static_cast<int64_t>(id) * p.R + min(r0 + 8 * j + g, p.R - 1)) * p.K + 8 * t;
        // Batches of blocks: all loads of a batch are issued before its first MMA.
        // Chunks past K read the row's first one and are taken as zeros.
        constexpr int kBatch = RT == 4 ? 2 : (RT == 2 ? 4 : 8);
        for (int k0 = 32 * warp; k0 < p.K; k0 += 32 * kWarps * kBatch) {
            uint4 x0[kBatch], x1[kBatch], y[kBatch][RT];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + 32 * kWarps * u;
                const int kk = k + 8 * t < p.K ? k : -8 * t;
                x0[u] = ld_v4(a0 + kk);
                x1[u] = ld_v4(a1 + kk);
#pragma unroll
                for (int j = 0; j < RT; ++j) y[u][j] = ld_v4(lb[j] + kk);
            }
            __syncwarp();  // (keeps the loads together: the compiler would move each down to its MMA)
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (k0 + 32 * kWarps * u + 32 > p.K) {  // (the same for the whole warp)
                    const uint32_t keep = k0 + 32 * kWarps * u + 8 * t < p.K ? 0xFFFFFFFFu : 0u;
                    auto mask = [&](uint4& v) {
                        v = make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep);
                    };
                    mask(x0[u]);
                    mask(x1[u]);
#pragma unroll
                    for (int j = 0; j < RT; ++j) mask(y[u][j]);
                }
                const uint32_t f0[4] = {x0[u].x, x1[u].x, x0[u].y, x1[u].y};
                const uint32_t f1[4] = {x0[u].z, x1[u].z, x0[u].w, x1[u].w};
#pragma unroll
                for (int j = 0; j < RT; ++j) {
                    mma_m16n8k16(acc[j], f0, y[u][j].x, y[u][j].y);
                    mma_m16n8k16(acc[j], f1, y[u][j].z, y[u][j].w);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            float* d = red + (warp * kRows + g) * 8 * RT + 8 * j + 2 * t;
            *reinterpret_cast<float2*>(d) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2*>(d + 8 * 8 * RT) = make_float2(acc[j][2], acc[j][3]);
        }
        __syncthreads();
        for (int o = threadIdx.x; o < kRows * 8 * RT; o += kThreads) {
            const int m = m0 + o / (8 * RT), r = r0 + o % (8 * RT);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += red[w * kRows * 8 * RT + o];  // warp order
            if (m < p.M && r < p.R && group_ids[m - m0] == id) 
                p.V[static_cast<int64_t>(m) * p.R + r] = __float2half_rn(s * sum);
        }
        __syncthreads();
    }
}

// Row groups from which the narrow form is taken (both sides measured above).
constexpr int kNarrowGroups = 64;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t round256(int64_t b) { return (b + 255) & ~int64_t(255); }

template <int RT, int W>
int launch_down(const DownParams& p, dim3 grid, cudaStream_t stream) {
    static OncePerDevice prepared;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W4A16_ERR_CUDA;
    const int rc = prepared.run(dev, [] {
        return cudaFuncSetAttribute(reinterpret_cast<const void*>(&lora_down_kernel<RT, W>),
                                    cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared) == cudaSuccess
                   ? W4A16_OK
                   : W4A16_ERR_CUDA;
    });
    if (rc) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(W * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_down_kernel<RT, W>, p) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

int lora_down(DownParams& p, int tiles, cudaStream_t stream) {
    p.groups = (p.M + kRows - 1) / kRows;
    // Ranks per CTA: few row groups spread the ranks over CTAs (8 each); many
    // keep 16 or 32 together, so that A is read once per 16 or 32 ranks.
    // (The narrow form has registers for 16.)
    const bool narrow = p.groups >= kNarrowGroups;
    const int rt = p.groups <= 8 ? 1 : (p.R <= 16 || narrow ? 2 : 4);
    const int chunks = (p.R + 8 * rt - 1) / (8 * rt);
    // Adapters of a group side by side while that leaves one CTA per SM, and always
    // two: a group where one prompt ends and the next begins would take twice as long.
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const int slots = std::min({kRows, static_cast<int>(p.M), std::max(2, sms / (p.groups * chunks))});
    const dim3 grid(static_cast<unsigned>(p.groups + tiles), static_cast<unsigned>(slots),
                    static_cast<unsigned>(chunks));
    if (narrow) return launch_down<2, 4>(p, grid, stream);
    switch (rt) {
        case 1: return launch_down<1, 16>(p, grid, stream);
        case 2: return launch_down<2, 16>(p, grid, stream);
        default: return launch_down<4, 16>(p, grid, stream);
    }
}

}  // namespace

int lora_device_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_lora_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_lora_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" int64_t w4a16_lora_workspace_size(int64_t M, int64_t R) {
    if (M < 0 || M >= (int64_t(1) << 31) || R < 8 || R > W4A16_MAX_RANK || R % 8) return -1;
    // V, the tiles' lists (at most 255 rows of padding), their lengths (tiles of at least 16 rows)
    return round256(M * R * 2) + round256((M + 256) * 4) + round256((M / 16 + 1) * 4);
}

extern "C" int w4a16_lora_gemm(const w4a16_half* A_dev, const uint8_t* Wt_dev, const w4a16_half* S_dev,
                               const w4a16_half* LA_dev, const w4a16_half* LB_dev, const int32_t* ids_dev,
                               const float* scaling_dev, w4a16_half* C_dev, int64_t M, int64_t N, int64_t K, int64_t G,
                               int64_t L, int64_t R, void* workspace_dev, int64_t workspace_bytes, void* stream) {
    if (!A_dev || !Wt_dev || !S_dev || !LA_dev || !LB_dev || !ids_dev || !C_dev || !workspace_dev || M < 0 || L < 1 ||
        R < 1)
        return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31) || L >= (int64_t(1) << 31) || R % 8 || R > W4A16_MAX_RANK)
        return W4A16_ERR_UNSUPPORTED;
    if (workspace_bytes < w4a16_lora_workspace_size(M, R)) return W4A16_ERR_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(A_dev), static_cast<const void*>(Wt_dev),
                          static_cast<const void*>(S_dev), static_cast<const void*>(LA_dev),
                          static_cast<const void*>(LB_dev), static_cast<const void*>(workspace_dev)})
        if (!aligned(q, 16)) return W4A16_ERR_MISALIGNED;
    if (!aligned(C_dev, 2) || !aligned(ids_dev, 4) || !aligned(scaling_dev, 4)) return W4A16_ERR_MISALIGNED;
    if (M == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
    DownParams d{};
    d.A = reinterpret_cast<const __half*>(A_dev);
    d.LA = reinterpret_cast<const __half*>(LA_dev);
    d.ids = ids_dev;
    d.scaling = scaling_dev;
    d.V = reinterpret_cast<__half*>(ws);
    d.list = reinterpret_cast<int32_t*>(ws + round256(M * R * 2));
    d.count = reinterpret_cast<int32_t*>(ws + round256(M * R * 2) + round256((M + 256) * 4));
    d.M = static_cast<int32_t>(M);
    d.K = static_cast<int32_t>(K);
    d.L = static_cast<int32_t>(L);
    d.R = static_cast<int32_t>(R);
    LoraOperands lora{reinterpret_cast<const __half*>(LB_dev), ids_dev, d.V, d.list, d.count, d.L, d.R};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LoraPlan plan;
    rc = lora_plan(M, N, K, G, &plan);
    if (rc) return rc;
    d.tile_rows = plan.tile_rows;
    rc = lora_down(d, plan.tile_rows ? static_cast<int>((M + plan.tile_rows - 1) / plan.tile_rows) : 0, s);
    if (rc) return rc;
    return lora_product(plan, lora, A_dev, Wt_dev, S_dev, C_dev, M, N, K, G, s);
}
