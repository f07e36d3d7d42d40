// W4A16 group-wise GEMM on sm_100a: C[M,N] = A[M,K] x dequant(W)[K,N].
//
// The operation is the one the Int4GroupwiseGemmPluginV2 page describes
// (class description: activations [b,seq,K] fp16, int4 weights, scales
// [ceil(K/G),N] fp16, output [b,seq,N] fp16; constructor: N columns, K rows,
// groupSize G). The grouped-expert entry point applies it per expert segment
// of gathered rows (Int4MoePlugin page, constructor parameters).
//
// One kernel template serves M > 16 (decode-sized M runs on the skinny
// kernel) and the grouped-expert form. It computes the transposed product
//     D[n, m] = sum_k W[k, n] * A[m, k]
// on the 5th-generation tensor core: each CTA owns 128 weight columns (the MMA
// M extent, one TMEM lane per column) and a tile of BN activation rows (the
// MMA N extent, 16..256), so that small token counts cost no padding of the
// weight side. Warp roles inside a CTA (320 or 576 threads):
//   warp 0      producer: per 64-deep K stage, one TMA tile load of the
//               activations (128-byte swizzle, zero fill past M and K) into a
//               ring of stages, and an L2 prefetch of the column tile's int4
//               stages well ahead of use.
//   warp 1      TMEM allocation and the single MMA-issuing thread
//               (tcgen05.mma kind::f16, A = weights from TMEM, B = activations
//               from shared memory, fp32 accumulator in TMEM); it waits on one
//               barrier per pair of stages.
//   warps 2..   dequantisation, in groups of four warps (one per TMEM lane
//               quadrant; group g takes stages g, g + groups, ...): each thread
//               loads its column's 64 int4 codes of a stage (two 16-byte halves
//               of the tiled layout) and their scale straight into registers,
//               two of its stages ahead, turns them into fp16 (magic-exponent
//               decode, times the group scale) and stores them into the
//               stage's tensor-memory slot; then the epilogue (tcgen05.ld ->
//               fp16 tile in shared memory -> 16-byte row stores).
// Small-M shapes split K across up to 8 CTAs of one thread-block cluster; the
// fp32 partial tiles are summed in rank order through distributed shared
// memory (deterministic, no global workspace).
//
// Every wait is bounded: a wait that runs out latches W4A16_ERR_TIMEOUT in the
// device status word, and the CTA drains its copies, frees its TMEM and exits.
//
// The template and its launch; w4a16_gemm.cu instantiates the plain products and
// w4a16_gemm_forms.cu the gated and adapter forms, so that a process which only
// calls the former does not load the latter's code.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/w4a16.h"
#include "dequant.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"
#include "w4a16_internal.h"
#include "waits.cuh"

namespace w4a16 {

constexpr int kTileN = 128;                 // weight columns per CTA (MMA M)
constexpr int kTileK = 64;                  // K per pipeline stage
constexpr int kRawBytes = 4096;             // int4 codes of one 128 x 64 tile (8-bit codes: twice that)
constexpr int kSlotCols = kTileK / 2;       // TMEM columns of one dequantised 128 x 64 fp16 tile
constexpr int kGroupWarps = 4;             // one dequantisation group: the 4 TMEM lane quadrants
constexpr int kAhead = 2;                  // stages of its own a dequantising thread loads ahead
constexpr int kPrefetchStages = 12;        // int4 tile stages the producer pulls into L2 ahead of use
// Threads of a CTA with DQ dequantisation groups (each group takes every
// DQ-th stage, so DQ groups keep DQ stages in flight).
__host__ __device__ constexpr int threads_for(int dq) { return (2 + kGroupWarps * dq) * 32; }
static_assert(threads_for(4) <= 1024, "the 256-row tile's four dequantisation groups fit a CTA");

struct Params {
    const uint8_t* wt[W4A16_MAX_EXPERTS];   // tiled weights (dense: [0])
    const __half* sc[W4A16_MAX_EXPERTS];    // scales [ceil(K/G), N]
    const int32_t* offsets;                 // grouped: [E+1] on the device
    __half* C;
    int32_t rows;       // dense: M; grouped: total gathered rows
    int32_t N, K, G;
    int32_t ngroups;    // ceil(K/G)
    int32_t KT;         // ceil(K/64)
    int32_t E;          // grouped: number of experts; dense: 1
    int32_t splits;     // CTAs along K (cluster size along x)
    int32_t grouped;
    int32_t prefetch;   // weights/scales may be read before the previous kernel finishes
    int32_t vec_out;    // C rows start on 16-byte boundaries (16-byte output stores)
    long long wait_limit;   // bound of every device wait, in SM clock cycles
    int32_t stall_stage;    // test aid: the dequantising warps withhold this stage's ready signal (< 0: never)
    int32_t act;            // W4A16_ACT_*: elementwise activation of the fp16 result (no K split); gated: the gate's
    // Gated form: wt[0] / sc[0] are the gate's, wt[1] / sc[1] the up projection's; C
    // is H, and Pg / Pu (both or neither) take the projections themselves.
    __half* Pg;
    __half* Pu;
    LoraOperands lora;  // adapter form
};

// What a launch computes. kPlain: the dense or the grouped-expert product.
// kGated: H = act(A W_gate) * (A W_up): a CTA owns 64 output columns, TMEM lanes
// 0..63 hold their gate columns and lanes 64..127 the same up columns, so one
// MMA sequence over one activation stream makes both projections, at the cost
// of a dense product twice as wide; the epilogue pairs the two halves. (Few rows,
// or a K split; w4a16_dgrad.cu takes the gated product of many rows.) Measured: 38 us
// for 17 and 32 rows x 4096 -> 14336, 40 for 64, bound by the stages' hand-off and decoding.
// kLora: the dense product plus V[m] LB[ids[m]]^T. The distinct adapters of the
// CTA's token tile form further contraction stages behind those of K, 64 values
// of (adapter, rank) each: the dequantising warps put LB's rows in the weights'
// TMEM slot and, in the activations' slot, V's rows rounded to fp16 where the row
// uses that adapter and zeros elsewhere. So the adapters join the same fp32
// accumulator and cost D * R / 64 more stages for D adapters in the tile. Measured
// at 2048 x 4096 -> 4096 with rank 16, call after call: 57 us without an adapter (the
// dense product takes 55), 65 with four prompts of one adapter each and one without, 76
// with one adapter for all rows, 111 with eight mixed; V's kernel is part of each.
enum GemmForm { kPlain = 0, kGated = 1, kLora = 2 };

// One kernel of a form and its launch, for one token tile and one kind of group size.
typedef int (*GemmLaunch)(const CUtensorMap&, const Params&, dim3, int, int, cudaStream_t);
struct GemmKernel {
    const void* fn;
    GemmLaunch launch;
};

// Token tiles and their pipeline depths: small tiles keep two CTAs per SM; the
// 256-row tile (one CTA per SM) runs four dequantisation groups of four warps
// (576 threads): each group has four stage periods to decode and store its
// stage. More groups (more warps competing for issue slots, and register
// spills above five) and fewer groups (too little time per stage) both ran
// slower on the prefill and grouped-expert shapes.
// <token tile, ring stages, TMEM columns, CTAs per SM, dequantisation groups>
#define W4A16_TOKEN_TILES(X) \
    X(16, 6, 256, 2, 2) X(32, 6, 256, 2, 2) X(64, 6, 256, 2, 2) X(128, 4, 256, 2, 2) X(192, 8, 512, 1, 4) X(256, 6, 512, 1, 4)

// The gated and adapter kernels (w4a16_gemm_forms.cu): token tile `variant`, any_group
// 0 for G a multiple of 64 (one scale per stage) or 1 for any G.
GemmKernel gated_kernel(int variant, int any_group);
GemmKernel lora_kernel(int variant, int any_group);
int forms_device_status(bool clear);  // their latched device status (0 = none, -1 if it could not be read)

namespace {

__device__ int g_status;  // latched device-side error (0 = none) of this file's kernels

// One ring of LS stages. Stage s owns, in shared memory, an activation tile
// and, in tensor memory, a 32-column slot for the dequantised fp16 weights;
// TMEM also holds the fp32 accumulator (BN columns). The int4 codes and the
// scales go straight from global memory into the dequantising threads'
// registers, a few stages ahead, so the copy engine only moves activations.
template <int BN, int LS, int TMEM_COLS>
struct Layout {
    static constexpr int kActBytes = BN * 128;
    static constexpr int kAct = 0;
    static constexpr int kBar = kAct + LS * kActBytes;
    static constexpr int kNumBars = LS + LS / 2 + LS + 1;  // full, afull (per stage pair), done, accfull
    static constexpr int kMisc = kBar + kNumBars * 8;  // tmem base, abort flag, tile info
    static constexpr int kTotal = kMisc + 32;
    static constexpr int kAlloc = kTotal + 1024;       // slack for aligning the base to 1024
    static constexpr int kAccCols = BN < 32 ? 32 : BN;
    static constexpr int kRedBytes = BN * kTileN * 4;  // split-K partials, alias the load ring
    static_assert(kAccCols + LS * kSlotCols <= TMEM_COLS, "TMEM ring does not fit the allocation");
    static_assert(TMEM_COLS == 32 || TMEM_COLS == 64 || TMEM_COLS == 128 || TMEM_COLS == 256 || TMEM_COLS == 512,
                  "TMEM allocations are powers of two");
    static_assert(kRedBytes <= kBar, "split-K buffer must fit in the activation ring");
    static_assert(BN * kTileN * 3 <= kBar, "the gated epilogue's exchange and output tiles fit in the activation ring");
    static_assert((kActBytes % 1024) == 0, "activation tiles need 1024-byte alignment");
    static_assert((LS % 2) == 0, "the MMA thread takes the ring two stages at a time");
};

__device__ __forceinline__ void latch_status(int code) { atomicCAS(&g_status, 0, code); }

__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit) {
    return w4a16::wait_phase(bar, parity, abort_flag, limit, &g_status);
}
__device__ __forceinline__ bool drain_phase(uint64_t* bar, uint32_t parity) {
    return w4a16::drain_phase(bar, parity, &g_status);
}
__device__ __forceinline__ bool warp_wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                long long limit) {
    return w4a16::warp_wait_phase(bar, parity, abort_flag, limit, &g_status);
}
__device__ __forceinline__ bool warp_drain_phase(uint64_t* bar, uint32_t parity) {
    return w4a16::warp_drain_phase(bar, parity, &g_status);
}

// Adapter form: the index of the first adapter stage (the ring is taken by whole
// pairs of stages), and this CTA's range of the tile's adapter stages, which the
// CTAs of a K split share. V and the tile's list come from the kernel before.
__device__ __forceinline__ int lora_first(int nst) { return (nst + 1) & ~1; }
__device__ __forceinline__ void lora_range(const Params& p, int split, int* begin, int* count) {
    grid_dependency_wait();
    const int all = (__ldcg(p.lora.count + blockIdx.z) * (p.lora.R / 8) + 7) / 8;
    *begin = split * all / p.splits;
    *count = (split + 1) * all / p.splits - *begin;
}

// 0xFFFF in each half of x that holds an infinity or NaN (its exponent field is all ones).
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t x) {
    return ((((x & 0x7C007C00u) + 0x04000400u) >> 15) & 0x00010001u) * 0xFFFFu;
}

// OG: G is a multiple of 64, so a stage lies inside one scale group.
// BITS: 4 for the int4 tiled layout, 8 for the 8-bit code layout (W8A16): a
// stage's tile is 4 or 8 KB, and a thread loads 2 or 4 16-byte chunks of its
// column per stage; everything after the decode is the same.
template <int BN, int LS, int TMEM_COLS, int MINB, int DQ, bool OG, int BITS, int FORM>
__global__ void __launch_bounds__(threads_for(DQ), MINB)
    w4a16_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ Params p) {
    using L = Layout<BN, LS, TMEM_COLS>;
    static_assert(BITS == 4 || BITS == 8, "int4 or 8-bit codes");
    constexpr bool GATED = FORM == kGated, LORA = FORM == kLora;
    static_assert(FORM == kPlain || BITS == 4, "the gated and adapter forms read int4 codes");
    constexpr int kCols = GATED ? kTileN / 2 : kTileN;  // output columns of a CTA
    constexpr int kTileBytes = BITS == 4 ? kRawBytes : 2 * kRawBytes;  // one 128 x 64 tile of codes
    constexpr int kChunks = BITS / 2;                                  // 16-byte chunks per column and stage
    constexpr int kScales = OG ? 1 : 8;  // scale registers per stage and thread
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base_addr = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (base_addr & 1023u)) & 1023u);

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);   // stage's copies landed
    uint64_t* afull = full + LS;                                     // stage pair ready for the MMAs
    uint64_t* done = afull + LS / 2;                                 // stage's MMAs completed
    uint64_t* accfull = done + LS;                                   // accumulator complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
    int* tile_info = reinterpret_cast<int*>(smem + L::kMisc + 8);  // has_tile, expert, m0, rows, staged, bad LB

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int nt = blockIdx.y;

    // ---------------------------------------------------------------- tile
    if (threadIdx.x == 0) {
        int has = 1, expert = 0, m0 = 0, rows = 0;
        if (p.grouped) {
            grid_dependency_wait();  // the offsets may come from the previous kernel
            const int32_t* off = p.offsets;
            bool ok = off[0] == 0 && off[p.E] == p.rows;
            for (int e = 0; e < p.E && ok; ++e) ok = off[e + 1] >= off[e];
            has = 0;
            if (!ok) {
                latch_status(W4A16_ERR_BAD_OFFSETS);
            } else {
                int z = blockIdx.z;
                for (int e = 0; e < p.E; ++e) {
                    const int cnt = off[e + 1] - off[e];
                    const int tiles = (cnt + BN - 1) / BN;
                    if (z < tiles) {
                        has = 1;
                        expert = e;
                        m0 = off[e] + z * BN;
                        rows = min(BN, off[e + 1] - m0);
                        break;
                    }
                    z -= tiles;
                }
            }
        } else {
            m0 = blockIdx.z * BN;
            rows = min(BN, p.rows - m0);
        }
        tile_info[0] = has;
        tile_info[1] = expert;
        tile_info[2] = m0;
        tile_info[3] = rows;
        tile_info[4] = 1;
    }
    __syncthreads();
    if (!tile_info[0]) return;  // grouped slot beyond the routed tiles (no cluster in that mode)
    const int expert = tile_info[1];
    const int m0 = tile_info[2];
    const int rows = tile_info[3];
    const int split = p.grouped ? 0 : static_cast<int>(blockIdx.x);
    const int kb = static_cast<int>((static_cast<int64_t>(split) * p.KT) / p.splits);
    const int ke = static_cast<int>((static_cast<int64_t>(split + 1) * p.KT) / p.splits);
    const int nst = ke - kb;
    const int n_mma = min(BN, (rows + 15) & ~15);
    const uint32_t idesc = idesc_f16_f32(128, static_cast<uint32_t>(n_mma));

    auto issue_act = [&](int i) {
        const int s = i % LS;
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(L::kActBytes));
        tma_load_2d(smem + L::kAct + s * L::kActBytes, &tmA, (kb + i) * kTileK, m0, &full[s]);
    };

    // ---- dequantisation threads' state (warps 2..). Their first look-ahead
    // loads go out before the barrier and TMEM setup below, so that the
    // first stage's memory latency overlaps it.
    const int dw = warp - 2;
    const int grp = dw >> 2;          // dequantisation group: stages grp, grp + DQ, ...
    const int quad = warp & 3;        // TMEM lane quadrant this warp may access
    const int j = quad * 32 + lane;   // weight column inside the tile = TMEM lane
    const int n = GATED ? nt * kCols + (j & (kCols - 1)) : nt * kTileN + j;
    const bool col_ok = n < p.N;
    const uint32_t tlane = static_cast<uint32_t>(quad * 32) << 16;
    // Codes and scales of this thread's stages (i = grp, grp + DQ, ...) are
    // loaded kAhead of its stages ahead into registers: the two 16-byte
    // halves (k 0..31 and 32..63) of the column's stage and its scales (one
    // when G is a multiple of 64, else one per 8-deep word). Loaded values
    // are left exactly as loaded until the stage is decoded: any instruction
    // that reads a register whose load is in flight waits for that load.
    // kk is the first k of the next stage to load, gk = floor(kk / G).
    // (A padded column past N reads column 0's scales; its codes are 0.)
    // (Gated: the lane's half picks the matrix, and a CTA's 64 columns are one half of a 128-column weight tile.)
    const int half = GATED ? j / kCols : 0;
    const int wtile_n = GATED ? nt >> 1 : nt;
    const int wtile_j = GATED ? (nt & 1) * kCols + (j & (kCols - 1)) : j;
    const uint8_t* wcol =
        p.wt[GATED ? half : expert] + static_cast<int64_t>(wtile_n) * p.KT * kTileBytes + wtile_j * 16;
    const __half* scol = p.sc[GATED ? half : expert] + (col_ok ? n : 0);
    // (Adapter form: weights, scales and activations are read past L1 without waiting
    // for the kernel that makes V, which lets this one start only once everything
    // before it is complete; see the wait before the adapter stages.)
    auto load_scale = [](const __half* q) { return FORM == kPlain ? __ldg(q) : __ldcg(q); };
    int li = grp;
    int kk = (kb + grp) * kTileK;
    int gk = kk / p.G;
    auto load_next = [&](uint4 (&r)[kChunks], __half (&sv)[kScales]) {
        if (li < nst) {
            const uint8_t* src = wcol + static_cast<int64_t>(kb + li) * kTileBytes;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                r[c] = FORM == kPlain ? ld_nc_v4(src + c * 2048) : ld_cg_v4(src + c * 2048);
            if constexpr (OG) {
                sv[0] = load_scale(scol + static_cast<int64_t>(min(gk, p.ngroups - 1)) * p.N);
            } else {
                const int rem = kk - gk * p.G;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    int g = gk, r2 = rem + 8 * q;
                    while (r2 >= p.G) {
                        r2 -= p.G;
                        ++g;
                    }
                    sv[q] = load_scale(scol + static_cast<int64_t>(min(g, p.ngroups - 1)) * p.N);
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) r[c] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int q = 0; q < kScales; ++q) sv[q] = __float2half(0.f);
        }
        li += DQ;
        kk += kTileK * DQ;
        while ((gk + 1) * p.G <= kk) ++gk;
    };
    uint4 rq0[kChunks], rq1[kChunks];
    __half sq0[kScales], sq1[kScales];
    if (warp >= 2) {
        if (!LORA && !p.prefetch) grid_dependency_wait();  // weights and scales may come from the previous kernel
        load_next(rq0, sq0);
        load_next(rq1, sq1);
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < LS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 1);
        }
        for (int q = 0; q < LS / 2; ++q) mbar_init(&afull[q], 2 * kGroupWarps);
        mbar_init(accfull, 1);
        *abort_flag = 0;
        tile_info[5] = 0;
        fence_mbar_init();
        prefetch_tensor_map(&tmA);
        grid_launch_dependents();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_acc = *tmem_slot;                 // accumulator: columns [0, BN)
    const uint32_t tmem_ring = tmem_acc + L::kAccCols;    // weight slots: kSlotCols columns each

    if (warp == 0) {
        // ------------------------------------------------------ producer
        // A stage's slot is free again once the MMAs that read it completed
        // (which also means the dequantisation warps finished reading it).
        if (lane == 0) {
            if (!LORA) grid_dependency_wait();  // the activations may be written by the previous kernel
            // The int4 tile of a stage is one contiguous 4 KB block: pull it into
            // L2 kPrefetchStages ahead, so that the dequantising threads' own
            // loads (issued only kAhead of their stages ahead) find it there.
            // (The ring's first LS activation tiles go out before the prefetches.)
            // (Gated: two neighbouring CTAs read the same two tiles; the even one fetches the gate's, the odd
            // one the up projection's.)
            const uint8_t* wtile =
                p.wt[GATED ? nt & 1 : expert] + (static_cast<int64_t>(GATED ? nt >> 1 : nt) * p.KT + kb) * kTileBytes;
            const int first = min(nst, LS);
            for (int i = 0; i < first; ++i) issue_act(i);
            for (int i = 0; i < min(nst, kPrefetchStages + first); ++i)
                bulk_prefetch_l2(wtile + static_cast<int64_t>(i) * kTileBytes, kTileBytes);
            int issued = first;
            for (; issued < nst; ++issued) {
                const int i = issued;
                if (i >= LS &&
                    !wait_phase(&done[i % LS], static_cast<uint32_t>((i / LS) - 1) & 1u, abort_flag, p.wait_limit))
                    break;
                issue_act(i);
                if (i + kPrefetchStages < nst)
                    bulk_prefetch_l2(wtile + static_cast<int64_t>(i + kPrefetchStages) * kTileBytes, kTileBytes);
            }
            // Every issued copy must land before the CTA's shared memory is released.
            for (int i = max(0, issued - LS); i < issued; ++i)
                drain_phase(&full[i % LS], static_cast<uint32_t>(i / LS) & 1u);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            // One barrier per pair of stages covers both operands of both stages:
            // the dequantised weights and, through each group's first warp, the
            // landed activation tiles. (Each wait costs the single issuing thread
            // about as long as an MMA, so it is paid once per eight MMAs.)
            // (The ring is unrolled: each slot's descriptors are constants.)
            const uint64_t bdesc0 = smem_desc_k_sw128(smem_addr(smem + L::kAct));
            bool stop = false;
            for (int base = 0; base < nst && !stop; base += LS) {
                const uint32_t par = static_cast<uint32_t>(base / LS) & 1u;
#pragma unroll
                for (int qq = 0; qq < LS / 2; ++qq) {
                    const int i = base + 2 * qq;
                    if (i >= nst) break;
                    if (!wait_phase(&afull[qq], par, abort_flag, p.wait_limit)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after_sync();
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (i + t < nst) {
                            constexpr uint64_t kStep = static_cast<uint64_t>(L::kActBytes >> 4);
                            const int s = 2 * qq + t;
                            const uint64_t bdesc = bdesc0 + static_cast<uint64_t>(s) * kStep;
                            const uint32_t a0 = tmem_ring + static_cast<uint32_t>(s * kSlotCols);
                            mma_f16_ts(tmem_acc, a0, bdesc, idesc, (i + t) > 0 ? 1u : 0u);
                            mma_f16_ts(tmem_acc, a0 + 8, bdesc + 2, idesc, 1u);
                            mma_f16_ts(tmem_acc, a0 + 16, bdesc + 4, idesc, 1u);
                            mma_f16_ts(tmem_acc, a0 + 24, bdesc + 6, idesc, 1u);
                            mma_commit(&done[s]);
                        } else if (LORA) {
                            mma_commit(&done[2 * qq + t]);  // the skipped partner of an odd last stage
                        }
                    }
                }
            }
            if constexpr (LORA) {
                // The adapter stages, in the same ring from the next whole pair on.
                int begin, count;
                lora_range(p, split, &begin, &count);
                const int first = lora_first(nst), end = first + count;
                for (int i = first; i < end && !stop; ++i) {
                    const int s = i % LS;
                    if ((i & 1) == 0 &&
                        !wait_phase(&afull[s >> 1], static_cast<uint32_t>(i / LS) & 1u, abort_flag, p.wait_limit))
                        break;
                    tc_fence_after_sync();
                    const uint64_t bdesc = smem_desc_k_sw128(smem_addr(smem + L::kAct + s * L::kActBytes));
                    const uint32_t a0 = tmem_ring + static_cast<uint32_t>(s * kSlotCols);
                    mma_f16_ts(tmem_acc, a0, bdesc, idesc, 1u);
                    mma_f16_ts(tmem_acc, a0 + 8, bdesc + 2, idesc, 1u);
                    mma_f16_ts(tmem_acc, a0 + 16, bdesc + 4, idesc, 1u);
                    mma_f16_ts(tmem_acc, a0 + 24, bdesc + 6, idesc, 1u);
                    mma_commit(&done[s]);
                }
            }
            mma_commit(accfull);  // fires once every MMA issued above has completed
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ dequant + epilogue
        // One stage: decode the codes and scales held in (r, sv), refill them
        // with the thread's stage kAhead of its stages later, store the fp16
        // weights into the stage's TMEM slot and arrive. False when aborting.
        auto stage = [&](int i, uint4 (&r)[kChunks], __half (&sv)[kScales]) -> bool {
            const int s = i % LS;
            uint32_t v[2][16];  // (k, k+1) pairs: k 0..31, k 32..63
            if constexpr (BITS == 4) {
                const uint32_t raw[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
                for (int q = 0; q < 8; ++q) {  // word q: k 8q .. 8q+7
                    const uint4 o = dequant_word(raw[q], __half2half2(sv[OG ? 0 : q]));
                    v[q >> 2][4 * (q & 3)] = o.x;
                    v[q >> 2][4 * (q & 3) + 1] = o.y;
                    v[q >> 2][4 * (q & 3) + 2] = o.z;
                    v[q >> 2][4 * (q & 3) + 3] = o.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // chunk c: k 16c .. 16c+15
                    const uint32_t raw[4] = {r[c].x, r[c].y, r[c].z, r[c].w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {  // word w: k 16c+4w .. +3, scale word (16c+4w)/8
                        const uint2 o = dequant_word8(raw[w], __half2half2(sv[OG ? 0 : 2 * c + (w >> 1)]));
                        const int pr = 8 * c + 2 * w;  // index of the pair (k, k+1) with k = 16c+4w
                        v[pr >> 4][pr & 15] = o.x;
                        v[pr >> 4][(pr & 15) + 1] = o.y;
                    }
                }
            }
            load_next(r, sv);
            // (Columns past N hold code 0 in the tiled layout and get scale 0: v is 0.)
            if (i >= LS &&
                !warp_wait_phase(&done[s], static_cast<uint32_t>((i / LS) - 1) & 1u, abort_flag, p.wait_limit))
                return false;
            tc_fence_after_sync();
            tmem_st_32x32b_x16(tmem_ring + tlane + s * kSlotCols, v[0]);
            tmem_st_32x32b_x16(tmem_ring + tlane + s * kSlotCols + 16, v[1]);
            tmem_st_wait();
            tc_fence_before_sync();
            // The group's first warp also sees the stage's activation tile land,
            // so that the MMA thread waits on one barrier per stage pair. The
            // last stage of an odd count arrives for its missing partner too.
            if ((dw & 3) == 0 &&
                !warp_wait_phase(&full[s], static_cast<uint32_t>(i / LS) & 1u, abort_flag, p.wait_limit))
                return false;
            __syncwarp();
            if (lane == 0 && i != p.stall_stage)
                mbar_arrive_cnt(&afull[(i >> 1) % (LS / 2)], ((i & 1) == 0 && i + 1 == nst) ? 2u : 1u);
            return true;
        };
        // kAhead = 2 register slots, used alternately: a stage's codes stay in
        // the registers they were loaded into (moving a register whose load is
        // still in flight would wait for that load).
        static_assert(kAhead == 2, "the stage loop below alternates two register slots");
        for (int i = grp; i < nst; i += 2 * DQ) {
            if (!stage(i, rq0, sq0)) break;
            if (i + DQ < nst && !stage(i + DQ, rq1, sq1)) break;
        }

        if constexpr (LORA) {
            int begin, count;
            lora_range(p, split, &begin, &count);
            const int first = lora_first(nst), end = first + count;
            const int tid = static_cast<int>(threadIdx.x - 64) & (kGroupWarps * 32 - 1);  // inside the group
            const int32_t* list = p.lora.list + static_cast<int64_t>(blockIdx.z) * BN;
            const int used = __ldcg(p.lora.count + blockIdx.z);
            const int per = p.lora.R / 8;  // 8-rank chunks of one adapter
            // The adapters of this thread's activation rows (tid, tid + 128).
            constexpr int kRowsPer = (BN + kGroupWarps * 32 - 1) / (kGroupWarps * 32);
            int row_id[kRowsPer];
#pragma unroll
            for (int x = 0; x < kRowsPer; ++x) {
                const int row = tid + x * kGroupWarps * 32;
                row_id[x] = row < rows ? __ldcg(p.lora.ids + m0 + row) : -1;
            }
            int i = first + ((grp - first) % DQ + DQ) % DQ;
            for (; i < end; i += DQ) {
                const int s = i % LS;
                // Chunk q of the stage holds ranks 8 rr .. + 7 of the d-th adapter of the
                // list, (d, rr) = divmod(q0 + q, per). All loads of a kind go out together.
                const int q0 = (begin + i - first) * 8;
                int who[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int d = (q0 + q) / per;
                    who[q] = d < used ? __ldcg(list + d) : -1;
                }
                uint32_t v[2][16];
                uint32_t bad = 0;
                {
                    uint4 x[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        x[q] = make_uint4(0u, 0u, 0u, 0u);
                        if (who[q] >= 0 && col_ok)
                            x[q] = __ldcg(reinterpret_cast<const uint4*>(
                                p.lora.LB + (static_cast<int64_t>(who[q]) * p.N + n) * p.lora.R + (q0 + q) % per * 8));
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        // An infinity or NaN would meet the zeros of rows that do not use
                        // this adapter: it is left out here, and its own rows get it in
                        // the epilogue.
                        const uint32_t xs[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t m = nonfinite_halves(xs[e]);
                            bad |= m;
                            v[q >> 2][4 * (q & 3) + e] = xs[e] & ~m;
                        }
                    }
                }
                if (bad) tile_info[5] = 1;
                if (i >= LS &&
                    !warp_wait_phase(&done[s], static_cast<uint32_t>((i / LS) - 1) & 1u, abort_flag, p.wait_limit))
                    break;
                tc_fence_after_sync();
                tmem_st_32x32b_x16(tmem_ring + tlane + s * kSlotCols, v[0]);
                tmem_st_32x32b_x16(tmem_ring + tlane + s * kSlotCols + 16, v[1]);
#pragma unroll
                for (int x = 0; x < kRowsPer; ++x) {
                    const int row = tid + x * kGroupWarps * 32;
                    if (row >= BN) break;
                    const uint32_t dst = smem_addr(smem + L::kAct + s * L::kActBytes) + row * 128;
                    const __half* vrow = p.lora.V + static_cast<int64_t>(m0 + row) * p.lora.R;
                    uint4 y[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        y[q] = make_uint4(0u, 0u, 0u, 0u);
                        if (row_id[x] >= 0 && who[q] == row_id[x])
                            y[q] = __ldcg(reinterpret_cast<const uint4*>(vrow + (q0 + q) % per * 8));
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) sts128(dst + ((q ^ (row & 7)) << 4), y[q]);
                }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cnt(&afull[s >> 1], ((i & 1) == 0 && i + 1 == end) ? 2u : 1u);
            }
        }

        // -------------------------------------------------- epilogue
        // The accumulator is complete (or the CTA is aborting) once accfull fires;
        // either way no MMA may still run when TMEM is released.
        const bool drained = warp_drain_phase(accfull, 0);
        tc_fence_after_sync();
        grid_dependency_wait();  // the output may still be read by the previous kernel
        const int aborted = __shfl_sync(0xffffffffu, *abort_flag, 0);
        bool have_acc = drained && !aborted && nst > 0;
        // Adapter form, an LB with infinities or NaN: each output adds its own
        // adapter's terms that the MMA left out.
        const bool fix = LORA && have_acc && *(volatile int*)&tile_info[5] != 0;
        auto lora_fix = [&](uint32_t (&v)[16], int c) {
#pragma unroll  // (v stays in registers)
            for (int t = 0; t < 16; ++t) {
                const int row = c * 16 + t;
                const int id = row < rows && col_ok ? __ldcg(p.lora.ids + m0 + row) : -1;
                if (id < 0 || id >= p.lora.L) continue;
                const __half* b = p.lora.LB + (static_cast<int64_t>(id) * p.N + n) * p.lora.R;
                float acc = 0.f;
                for (int rr = 0; rr < p.lora.R; ++rr) {
                    const float x = __half2float(__ldcg(b + rr));
                    if (!isfinite(x))
                        acc += __half2float(__ldcg(p.lora.V + static_cast<int64_t>(m0 + row) * p.lora.R + rr)) * x;
                }
                v[t] = __float_as_uint(__uint_as_float(v[t]) + acc);
            }
        };
        if constexpr (GATED) {
            // The epilogue's barriers need one answer for every warp: the tile is
            // written only if each of them found it complete.
            if (lane == 0 && !have_acc) tile_info[4] = 0;
            named_barrier(1 + DQ, kGroupWarps * 32 * DQ);
            have_acc = tile_info[4] != 0;
        } else {
            if (dw == 0 && lane == 0) tile_info[4] = have_acc ? 1 : 0;
        }
        if (GATED && p.splits == 1) {
            // Pair the halves: of each 16-token chunk a gate lane hands over its last
            // eight tokens and keeps the first eight, an up lane the other way round,
            // through an fp32 tile [token][64 columns] in the idle activation ring.
            // Each then owns both projections of eight outputs of its column. The
            // projections to keep are staged afterwards, over the exchange tile.
            if (have_acc) {
                float* xch = reinterpret_cast<float*>(smem + L::kAct);
                __half* htile = reinterpret_cast<__half*>(smem + L::kAct + BN * kCols * 4);
                const int jc = j & (kCols - 1);
                const int keep = half ? 8 : 0, give = 8 - keep;
                const int nch = n_mma / 16;
                for (int c = grp; c < nch; c += DQ) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(tmem_acc + tlane + c * 16, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        xch[(c * 16 + give + t) * kCols + jc] = __uint_as_float(half ? v[t] : v[8 + t]);
                    named_barrier(1 + grp, kGroupWarps * 32);  // (the chunk's four warps: both halves of its 64 columns)
                    const int act = p.act;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const float mine = __uint_as_float(half ? v[8 + t] : v[t]);
                        const float other = xch[(c * 16 + keep + t) * kCols + jc];
                        const float h = half ? gate_value(other, act) * mine : gate_value(mine, act) * other;
                        htile[(c * 16 + keep + t) * kCols + jc] = __float2half_rn(h);
                    }
                }
                if (p.Pg) {
                    named_barrier(1 + DQ, kGroupWarps * 32 * DQ);  // every thread is done with the exchange tile
                    __half* ptile = reinterpret_cast<__half*>(smem + L::kAct);  // [token][gate 64 | up 64]
                    for (int c = grp; c < nch; c += DQ) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(tmem_acc + tlane + c * 16, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            ptile[(c * 16 + t) * kTileN + j] = __float2half_rn(__uint_as_float(v[t]));
                    }
                }
            }
        } else if (p.splits == 1) {
            // Stage the fp16 tile, row-major [token][128 columns], in the idle
            // activation ring (every copy into it was consumed by a completed
            // MMA), so that the global stores below are whole 16-byte vectors.
            // Two 16-token chunks per TMEM wait.
            if (have_acc) {
                __half* stile = reinterpret_cast<__half*>(smem + L::kAct);
                const int nch = n_mma / 16;
                for (int c = grp; c < nch; c += 2 * DQ) {
                    const bool two = c + DQ < nch;
                    uint32_t v[16], w[16];
                    tmem_ld_32x32b_x16(tmem_acc + tlane + c * 16, v);
                    if (two) tmem_ld_32x32b_x16(tmem_acc + tlane + (c + DQ) * 16, w);
                    tmem_ld_wait();
                    if (LORA && fix) {
                        lora_fix(v, c);
                        if (two) lora_fix(w, c + DQ);
                    }
                    const int act = LORA ? static_cast<int>(W4A16_ACT_IDENTITY) : p.act;
                    if (act == W4A16_ACT_IDENTITY) {
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            stile[(c * 16 + t) * kTileN + j] = __float2half_rn(__uint_as_float(v[t]));
                        if (two) {
#pragma unroll
                            for (int t = 0; t < 16; ++t)
                                stile[((c + DQ) * 16 + t) * kTileN + j] = __float2half_rn(__uint_as_float(w[t]));
                        }
                    } else {
                        for (int t = 0; t < 16; ++t)
                            stile[(c * 16 + t) * kTileN + j] = epilogue_value(__uint_as_float(v[t]), act);
                        if (two) {
                            for (int t = 0; t < 16; ++t)
                                stile[((c + DQ) * 16 + t) * kTileN + j] = epilogue_value(__uint_as_float(w[t]), act);
                        }
                    }
                }
            }
        } else {
            float* red = reinterpret_cast<float*>(smem + L::kAct);
            for (int c = grp; c < BN / 16; c += DQ) {
                uint32_t v[16];
                if (have_acc && c * 16 < n_mma) {
                    tmem_ld_32x32b_x16(tmem_acc + tlane + c * 16, v);
                    tmem_ld_wait();
                    if (LORA && fix) lora_fix(v, c);
                } else {
#pragma unroll
                    for (int t = 0; t < 16; ++t) v[t] = 0u;
                }
#pragma unroll
                for (int t = 0; t < 16; ++t) red[(c * 16 + t) * kTileN + j] = __uint_as_float(v[t]);
            }
        }
        tc_fence_before_sync();
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_acc, TMEM_COLS);
    }

    if (GATED && p.splits == 1 && tile_info[4]) {
        // Rows of 64 columns, 8 chunks of 16 bytes each: H, then the projections.
        const int n0 = nt * kCols;
        auto store_rows = [&](const __half* tile, int stride, __half* out) {
            for (int o = threadIdx.x; o < rows * 8; o += static_cast<int>(blockDim.x)) {
                const int r = o >> 3;
                const int cc = (o & 7) * 8;
                __half* dst = out + static_cast<int64_t>(m0 + r) * p.N + n0 + cc;
                if (p.vec_out && n0 + cc + 8 <= p.N) {
                    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(tile + r * stride + cc);
                } else {
                    for (int e = 0; e < 8 && n0 + cc + e < p.N; ++e) dst[e] = tile[r * stride + cc + e];
                }
            }
        };
        store_rows(reinterpret_cast<const __half*>(smem + L::kAct + BN * kCols * 4), kCols, p.C);
        if (p.Pg) {
            const __half* ptile = reinterpret_cast<const __half*>(smem + L::kAct);
            store_rows(ptile, kTileN, p.Pg);
            store_rows(ptile + kCols, kTileN, p.Pu);
        }
    }

    if (!GATED && p.splits == 1 && tile_info[4]) {
        // Row r of the tile is 16 chunks of 8 columns; a warp writes two rows
        // per instruction.
        const __half* stile = reinterpret_cast<const __half*>(smem + L::kAct);
        const int n0 = nt * kTileN;
        for (int o = threadIdx.x; o < rows * 16; o += static_cast<int>(blockDim.x)) {
            const int r = o >> 4;
            const int cc = (o & 15) * 8;
            __half* dst = p.C + static_cast<int64_t>(m0 + r) * p.N + n0 + cc;
            if (p.vec_out && n0 + cc + 8 <= p.N) {
                *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(stile + r * kTileN + cc);
            } else {
                for (int e = 0; e < 8 && n0 + cc + e < p.N; ++e) dst[e] = stile[r * kTileN + cc + e];
            }
        }
    }

    if (p.splits > 1) {
        // Sum the cluster's partial tiles in rank order; rank r writes columns
        // [r*128/S, (r+1)*128/S) of the tile.
        cluster_sync_all();
        const int S = p.splits;
        const int cw = kCols / S;
        const int rank = static_cast<int>(cluster_ctarank());
        const float* red = reinterpret_cast<const float*>(smem + L::kAct);
        // A CTA that stopped early left its partial tile incomplete: if any CTA of
        // the cluster did, none writes the tile.
        bool aborted = false;
        for (int src = 0; src < S; ++src)
            aborted |= __float_as_int(ld_dsmem_f32(const_cast<int*>(abort_flag), static_cast<uint32_t>(src))) != 0;
        for (int o = threadIdx.x; o < cw * rows; o += static_cast<int>(blockDim.x)) {
            const int col = rank * cw + (o % cw);
            const int tok = o / cw;
            const int nn = nt * kCols + col;
            if (nn < p.N && !aborted) {
                if constexpr (GATED) {
                    float gate[8], up[8];
#pragma unroll
                    for (int src = 0; src < 8; ++src) {
                        const bool in = src < S;
                        gate[src] = in ? ld_dsmem_f32(&red[tok * kTileN + col], static_cast<uint32_t>(src)) : 0.f;
                        up[src] = in ? ld_dsmem_f32(&red[tok * kTileN + kCols + col], static_cast<uint32_t>(src)) : 0.f;
                    }
                    float gv = 0.f, uv = 0.f;
#pragma unroll
                    for (int src = 0; src < 8; ++src) {  // rank order
                        gv += gate[src];
                        uv += up[src];
                    }
                    const int64_t o2 = static_cast<int64_t>(m0 + tok) * p.N + nn;
                    p.C[o2] = __float2half_rn(gate_value(gv, p.act) * uv);
                    if (p.Pg) {
                        p.Pg[o2] = __float2half_rn(gv);
                        p.Pu[o2] = __float2half_rn(uv);
                    }
                } else {
                    float part[8];
#pragma unroll
                    for (int src = 0; src < 8; ++src)
                        part[src] = src < S ? ld_dsmem_f32(&red[tok * kTileN + col], static_cast<uint32_t>(src)) : 0.f;
                    float acc = 0.f;
#pragma unroll
                    for (int src = 0; src < 8; ++src) acc += part[src];  // rank order
                    p.C[static_cast<int64_t>(m0 + tok) * p.N + nn] = __float2half_rn(acc);
                }
            }
        }
        cluster_sync_all();
    }
}

template <int BN, int LS, int TC, int MINB, int DQ, bool OG, int BITS, int FORM>
int launch_variant(const CUtensorMap& map, const Params& p, dim3 grid, int cluster_x, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads_for(DQ), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    if (cluster_x > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = static_cast<unsigned>(cluster_x);
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    cudaError_t e = cudaLaunchKernelEx(&cfg, w4a16_gemm_kernel<BN, LS, TC, MINB, DQ, OG, BITS, FORM>, map, p);
    return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

template <int BN, int LS, int TC, int MINB, int DQ, bool OG, int BITS, int FORM>
GemmKernel make_kernel() {
    return GemmKernel{reinterpret_cast<const void*>(&w4a16_gemm_kernel<BN, LS, TC, MINB, DQ, OG, BITS, FORM>),
                      &launch_variant<BN, LS, TC, MINB, DQ, OG, BITS, FORM>};
}

// The kernels of one form, by token tile and kind of group size.
template <int BITS, int FORM>
GemmKernel kernel_of(int variant, int any_group) {
#define W4A16_PAIR(BN, LS, TC, MINB, DQ) \
    {make_kernel<BN, LS, TC, MINB, DQ, true, BITS, FORM>(), make_kernel<BN, LS, TC, MINB, DQ, false, BITS, FORM>()},
    static const GemmKernel table[][2] = {W4A16_TOKEN_TILES(W4A16_PAIR)};
#undef W4A16_PAIR
    return table[variant][any_group];
}

// This file's status word: its value, or -1 if it could not be read.
inline int read_gemm_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace

}  // namespace w4a16
