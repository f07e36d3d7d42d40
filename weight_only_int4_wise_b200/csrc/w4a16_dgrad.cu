// Products with the transposed 4-bit weights, for backward passes with the
// weights frozen:
//     dA[m, k] = sum_n dC[m, n] * W[k, n],   W[k, n] = fp16(q[k, n] * s[k / G, n]),
// and the backward pass of the gated projections, whose two products share one
// accumulator: dA = dG x W_gate^T + dU x W_up^T with
//     dG = dH * u * act'(g),  dU = dH * act(g).
// (The Int4GroupwiseGemmPluginV2 page describes the forward product only.)
//
// The tiled weight layout is the forward product's: 16 bytes hold 32 consecutive
// k of one column n. Here k is the output and n the contraction, so a decoded
// chunk is a run along the MMA's M extent: it is written to shared memory as it
// comes, as an M-major operand tile (128-byte swizzle), and no transposed copy of
// the weights is needed. Each CTA owns 128 values of k (the MMA M extent) and a
// tile of BN gradient rows (the MMA N extent), and walks the contraction in
// 64-deep stages:
//   warp 0      producer: one TMA tile load of the gradient rows per stage
//               (128-byte swizzle, zero fill past M and N) into a ring of LB
//               stages, and an L2 prefetch of the code tiles ahead of use;
//   warp 1      TMEM allocation and the MMA-issuing thread (tcgen05.mma
//               kind::f16, both operands in shared memory, fp32 accumulator in
//               TMEM);
//   warps 2..   decoding, in groups of four warps (group g takes stages g, g +
//               groups, ...): a thread takes one column n and 64 of the 128 k
//               (two 16-byte chunks), multiplies by the group scales and writes
//               eight 16-byte runs into a ring of LA operand tiles, rotated by
//               the column so that eight neighbouring lanes hit distinct banks;
//               then the epilogue (tcgen05.ld -> fp16 tile in shared memory ->
//               16-byte row stores).
// The two rings are separate because their costs are: a gradient tile (BN x 128
// bytes) needs time to arrive, a decoded tile (16 KB) is made on the spot.
// What bounds it is shared memory: per stage the decoded tile is written and read
// (2 x 16 KB), the gradient tile too (2 x 32 KB at 256 rows), 768 cycles at 128
// bytes per clock for 512 cycles of MMAs (measured: 800). So where the grid stays
// full enough a CTA takes KM = 2 neighbouring blocks of 128 k (both accumulators fill
// TMEM): the gradient tile is brought in once for both, 1280 cycles for 1024.
// Few tiles split the contraction over a cluster of up to 8 CTAs; the fp32
// partial tiles are summed in rank order (deterministic).
//
// The gated projections of many rows use the same pipeline (GATED): H = act(A W_gate)
// * (A W_up) with the contraction over k. A CTA's two blocks are the 128 gate columns
// and the same 128 up columns, which share the activation tile; a thread decodes 64 k
// of one column, a row of a K-major operand tile, and in the epilogue a TMEM lane
// holds both projections of its column. Against one 128-lane MMA tile of 64 gate and
// 64 up columns from TMEM (w4a16_gemm_kernel.cuh), which brings the activations in twice as
// often, 2048 x 4096 -> 14336 takes 417 instead of 470 us (with SiLU). Each row tile
// reads both weight matrices again (332 MB from DRAM there, for inputs of 77 MB): at 15 %
// of DRAM's rate that does not bound it.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/w4a16.h"
#include "dequant.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"
#include "roles.h"
#include "w4a16_internal.h"
#include "waits.cuh"

namespace w4a16 {

namespace {

__device__ int g_dgrad_status;  // latched device-side error (0 = none)

constexpr int kOutK = 128;         // k per CTA (MMA M)
constexpr int kDepth = 64;         // contraction per stage
constexpr int kTile = 4096;        // bytes of one 128-column x 64-row code tile
constexpr int kABytes = kOutK * kDepth * 2;
constexpr int kPrefetchStages = 12;  // code tiles the producer pulls into L2 ahead of use

__host__ __device__ constexpr int dgrad_threads(int dq) { return (2 + kGroupWarps * dq) * 32; }

struct DgradParams {
    const uint8_t* wt[2];   // tiled weights of the sources (gated: gate, up)
    const __half* sc[2];    // scales [ceil(K/G), N]
    __half* out;            // dA [rows, K] (gated: H [rows, N])
    __half* Pg;             // gated: the projections to keep (both or neither)
    __half* Pu;
    int32_t act;            // gated: W4A16_ACT_*
    int32_t rows, N, K, G;
    int32_t tile_rows;      // gradient rows per CTA (a multiple of 16 up to BN)
    int32_t ngroups, KT;    // ceil(K/G), ceil(K/64)
    int32_t NS;             // stages of one source: ceil(N/64)
    int32_t stages;         // all stages: sources * NS
    int32_t splits;         // CTAs along the contraction (cluster size along x)
    int32_t prefetch;       // weights/scales may be read before the previous kernel finishes
    int32_t vec_out;        // output rows start on 16-byte boundaries
    long long wait_limit;
    int32_t stall_stage;    // test aid: withhold the ready signal of this stage of each CTA's range (< 0: never)
};

template <int BN, int LB, int LA, int KM>
struct DgradLayout {
    static constexpr int kBBytes = BN * kDepth * 2;
    static constexpr int kSlotA = KM * kABytes;  // the decoded tiles of one stage
    static constexpr int kB = 0;
    static constexpr int kA = kB + LB * kBBytes;
    static constexpr int kBar = kA + LA * kSlotA;
    static constexpr int kNumBars = LB + LA + LA + LB + 1;  // full, ready, done (per ring), accfull
    static constexpr int kMisc = kBar + kNumBars * 8;
    static constexpr int kTotal = kMisc + 32;
    static constexpr int kAlloc = kTotal + 1024;  // slack for aligning the base to 1024
    static constexpr int kTmemCols = KM * (BN < 32 ? 32 : BN);
    static_assert(kAlloc <= 227 * 1024, "the rings fit a CTA's shared memory");
    static_assert(kBBytes % 1024 == 0, "swizzled tiles need 1024-byte alignment");
    static_assert(BN * kOutK * 4 <= LB * kBBytes, "the split partials or the output tiles fit the gradient ring");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 512, "TMEM allocations are powers of two");
};

// Shared-memory descriptor of an M-major operand tile with the 128-byte swizzle:
// rows (one contraction index each) of 64 consecutive M values, 8-row atoms of
// 1024 bytes along the contraction, blocks of 64 M values `block_bytes` apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>(block_bytes >> 4) << 16;  // leading byte offset: next 64 M values
    d |= static_cast<uint64_t>(1024 >> 4) << 32;          // stride byte offset: next 8 contraction rows
    d |= static_cast<uint64_t>(1) << 46;                  // descriptor version for sm_100
    d |= static_cast<uint64_t>(2) << 61;                  // swizzle mode: 128 B
    return d;
}

// OG: G is a multiple of 64, so a thread's 64 k lie inside one scale group;
// otherwise one scale per 16 k (G is a multiple of 16).
template <int BN, int LB, int LA, int DQ, int MINB, int KM, bool OG, bool GATED>
__global__ void __launch_bounds__(dgrad_threads(DQ), MINB)
    w4a16_dgrad_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                       const __grid_constant__ DgradParams p) {
    using L = DgradLayout<BN, LB, LA, KM>;
    static_assert(DQ % KM == 0, "each group decodes one of the CTA's blocks of k");
    constexpr int kTurn = DQ / KM;  // a group takes every kTurn-th stage
    constexpr int kScales = OG ? 1 : 4;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base_addr = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (base_addr & 1023u)) & 1023u);

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);  // gradient tile landed
    uint64_t* ready = full + LB;                                    // decoded tile written, gradient tile seen
    uint64_t* doneA = ready + LA;                                   // MMAs that read the decoded tile completed
    uint64_t* doneB = doneA + LA;                                   // MMAs that read the gradient tile completed
    uint64_t* accfull = doneB + LB;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
    volatile int* tile_ok = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int m0 = blockIdx.z * p.tile_rows;
    const int rows = min(p.tile_rows, p.rows - m0);
    const int split = blockIdx.x;
    const int ib = static_cast<int>((static_cast<int64_t>(split) * p.stages) / p.splits);
    const int ie = static_cast<int>((static_cast<int64_t>(split + 1) * p.stages) / p.splits);
    const int nst = ie - ib;
    const int n_mma = min(BN, (rows + 15) & ~15);

    // ---- decoding threads' state; the first loads go out before the setup below
    const int dw = warp - kFirstDecodeWarp;
    const int kb = block_of_warp(warp, KM);   // which of the CTA's blocks of k this group decodes
    const int grp = stage_of_warp(warp, KM);  // its first stage
    const int kblk = GATED ? blockIdx.y : blockIdx.y * KM + kb;  // block of the output
    const int t = static_cast<int>(threadIdx.x - 64) & 127;  // thread inside its group
    // Transposed: column r of the stage (contraction index) and 64 of the block's 128 k.
    // Gated: column t of the block's 128, the stage's 64 k.
    const int r = GATED ? t : t & 63;
    const int mb = GATED ? 0 : t >> 6;
    const int kt = 2 * kblk + mb;
    const bool kt_ok = kt < p.KT;
    // Element offsets of this thread's scale rows: its k do not change from stage to stage.
    int64_t soff[kScales];
#pragma unroll
    for (int q = 0; q < kScales; ++q)
        soff[q] = static_cast<int64_t>(min((kt * kDepth + 16 * q) / p.G, p.ngroups - 1)) * p.N;
    int li = grp;  // next local stage to load
    const int gn = kblk * kOutK + t;  // gated: this thread's column (codes past N are 0)
    const uint8_t* gw = p.wt[kb] + static_cast<int64_t>(kblk) * p.KT * kTile + t * 16;
    const __half* gs = p.sc[kb] + (gn < p.N ? gn : 0);
    auto load_next = [&](uint4 (&c)[2], __half (&sv)[kScales]) {
        const int i = ib + li;
        if constexpr (GATED) {
            if (li < nst) {
                c[0] = ld_cg_v4(gw + static_cast<int64_t>(i) * kTile);
                c[1] = ld_cg_v4(gw + static_cast<int64_t>(i) * kTile + 2048);
#pragma unroll
                for (int q = 0; q < kScales; ++q)
                    sv[q] = __ushort_as_half(
                        ld_cg_u16(gs + static_cast<int64_t>(min((i * kDepth + 16 * q) / p.G, p.ngroups - 1)) * p.N));
            }
            li += kTurn;
            return;
        }
        const int src = i >= p.NS ? 1 : 0;
        const int ns = i - (src ? p.NS : 0);
        const int n = ns * kDepth + r;
        if (li < nst && kt_ok && n < p.N) {
            const uint8_t* w = p.wt[src] + (static_cast<int64_t>(ns >> 1) * p.KT + kt) * kTile + ((ns & 1) * 64 + r) * 16;
            c[0] = ld_cg_v4(w);
            c[1] = ld_cg_v4(w + 2048);
#pragma unroll
            for (int q = 0; q < kScales; ++q) sv[q] = __ushort_as_half(ld_cg_u16(p.sc[src] + soff[q] + n));
        } else {
            // Past N the weights must be exact zeros: they meet the gradient's zero
            // fill, and a clamped scale could be an infinity.
            c[0] = c[1] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int q = 0; q < kScales; ++q) sv[q] = __float2half(0.f);
        }
        li += kTurn;
    };
    uint4 c0[2], c1[2];
    __half s0[kScales], s1[kScales];
    if (warp >= 2) {
        if (!p.prefetch) grid_dependency_wait();  // weights and scales may come from the previous kernel
        load_next(c0, s0);
        load_next(c1, s1);
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < LB; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&doneB[s], 1);
        }
        for (int s = 0; s < LA; ++s) {
            mbar_init(&ready[s], kGroupWarps * KM);
            mbar_init(&doneA[s], 1);
        }
        mbar_init(accfull, 1);
        *abort_flag = 0;
        *tile_ok = 1;
        fence_mbar_init();
        prefetch_tensor_map(&tm0);
        prefetch_tensor_map(&tm1);
        grid_launch_dependents();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_acc = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            grid_dependency_wait();  // the gradients may be written by the previous kernel
            auto issue = [&](int l) {
                const int i = ib + l, s = l % LB;
                const int src = !GATED && i >= p.NS ? 1 : 0;
                mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(p.tile_rows * kDepth * 2));
                tma_load_2d(smem + L::kB + s * L::kBBytes, src ? &tm1 : &tm0, (i - (src ? p.NS : 0)) * kDepth, m0,
                            &full[s]);
            };
            // A pair of stages shares one run of 2 KM code tiles (fewer at the end of
            // K): fetched once, on the pair's first stage.
            const uint32_t pair_bytes = static_cast<uint32_t>(min(2 * KM, p.KT - 2 * kblk)) * kTile;
            auto prefetch = [&](int l) {
                const int i = ib + l;
                if (GATED) {
                    if (l < nst) {
                        const int64_t off = (static_cast<int64_t>(kblk) * p.KT + i) * kTile;
                        bulk_prefetch_l2(p.wt[0] + off, kTile);
                        bulk_prefetch_l2(p.wt[1] + off, kTile);
                    }
                    return;
                }
                const int src = i >= p.NS ? 1 : 0;
                const int ns = i - (src ? p.NS : 0);
                if (l < nst && ((ns & 1) == 0 || l == 0))
                    bulk_prefetch_l2(p.wt[src] + (static_cast<int64_t>(ns >> 1) * p.KT + 2 * kblk) * kTile, pair_bytes);
            };
            const int first = min(nst, LB);
            for (int l = 0; l < first; ++l) issue(l);
            for (int l = 0; l < kPrefetchStages + first; ++l) prefetch(l);
            int issued = first;
            for (; issued < nst; ++issued) {
                if (!wait_phase(&doneB[issued % LB], static_cast<uint32_t>((issued / LB) - 1) & 1u, abort_flag,
                                p.wait_limit, &g_dgrad_status))
                    break;
                issue(issued);
                prefetch(issued + kPrefetchStages);
            }
            // Every issued copy must land before the CTA's shared memory is released.
            for (int l = max(0, issued - LB); l < issued; ++l)
                drain_phase(&full[l % LB], static_cast<uint32_t>(l / LB) & 1u, &g_dgrad_status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = idesc_f16_f32(128, static_cast<uint32_t>(n_mma)) | (GATED ? 0u : 1u << 15);  // (A is M-major)
            const uint64_t adesc0 = GATED ? smem_desc_k_sw128(smem_addr(smem + L::kA))
                                          : smem_desc_mn_sw128(smem_addr(smem + L::kA), kABytes / 2);
            constexpr uint64_t kStepA = GATED ? 2 : 2048 >> 4;
            const uint64_t bdesc0 = smem_desc_k_sw128(smem_addr(smem + L::kB));
            int sa = 0, sb = 0;
            uint32_t par = 0;
            for (int l = 0; l < nst; ++l) {
                if (!wait_phase(&ready[sa], par, abort_flag, p.wait_limit, &g_dgrad_status)) break;
                tc_fence_after_sync();
                const uint64_t a = adesc0 + static_cast<uint64_t>(sa) * (L::kSlotA >> 4);
                const uint64_t b = bdesc0 + static_cast<uint64_t>(sb) * (L::kBBytes >> 4);
                // 16 of the contraction per MMA: two 1024-byte atoms of the M-major
                // tile (32 bytes of every row of the K-major one), 32 bytes of every
                // gradient row.
#pragma unroll
                for (int h = 0; h < KM; ++h) {
                    const uint64_t ah = a + h * (kABytes >> 4);
                    const uint32_t acc = tmem_acc + h * BN;
                    mma_f16_ss(acc, ah, b, idesc, l > 0 ? 1u : 0u);
                    mma_f16_ss(acc, ah + kStepA, b + 2, idesc, 1u);
                    mma_f16_ss(acc, ah + 2 * kStepA, b + 4, idesc, 1u);
                    mma_f16_ss(acc, ah + 3 * kStepA, b + 6, idesc, 1u);
                }
                mma_commit(&doneA[sa]);
                mma_commit(&doneB[sb]);
                if (++sa == LA) {
                    sa = 0;
                    par ^= 1u;
                }
                if (++sb == LB) sb = 0;
            }
            mma_commit(accfull);  // fires once every MMA issued above has completed
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ decode + epilogue
        const uint32_t row_addr =
            smem_addr(smem + L::kA) + static_cast<uint32_t>(kb * kABytes + mb * (kABytes / 2) + (r >> 3) * 1024 + (r & 7) * 128);
        auto stage = [&](int l, uint4 (&c)[2], __half (&sv)[kScales]) -> bool {
            const int sa = l % LA;
            const uint32_t raw[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = dequant_word(raw[q], __half2half2(sv[OG ? 0 : q >> 1]));
            load_next(c, sv);
            if (l >= LA && !warp_wait_phase(&doneA[sa], static_cast<uint32_t>((l / LA) - 1) & 1u, abort_flag,
                                            p.wait_limit, &g_dgrad_status))
                return false;
            const uint32_t dst = row_addr + static_cast<uint32_t>(sa * L::kSlotA);
#pragma unroll
            for (int q = 0; q < 8; ++q) sts128(dst + ((q ^ (r & 7)) << 4), v[q]);
            fence_proxy_async_smem();
            // The group's first warp also sees the stage's gradient tile land, so
            // that the MMA thread waits on one barrier per stage.
            if ((dw & 3) == 0 && !warp_wait_phase(&full[l % LB], static_cast<uint32_t>(l / LB) & 1u, abort_flag,
                                                  p.wait_limit, &g_dgrad_status))
                return false;
            __syncwarp();
            if (lane == 0 && l != p.stall_stage) mbar_arrive(&ready[sa]);
            return true;
        };
        // Two register slots, used alternately: codes stay in the registers they were loaded into.
        for (int l = grp; l < nst; l += 2 * kTurn) {
            if (!stage(l, c0, s0)) break;
            if (l + kTurn < nst && !stage(l + kTurn, c1, s1)) break;
        }

        // -------------------------------------------------- epilogue
        const int quad = warp & 3;       // TMEM lane quadrant this warp may access
        const int j = quad * 32 + lane;  // k inside the tile = TMEM lane
        const uint32_t tlane = static_cast<uint32_t>(quad * 32) << 16;
        const bool drained = warp_drain_phase(accfull, 0, &g_dgrad_status);
        tc_fence_after_sync();
        grid_dependency_wait();  // the output may still be read by the previous kernel
        const int aborted = __shfl_sync(0xffffffffu, *abort_flag, 0);
        const bool have_acc = drained && !aborted && nst > 0;
        if (lane == 0 && !have_acc) *tile_ok = 0;
        if constexpr (GATED) {
            // H, and the projections if they are kept: three [row][128] tiles of which
            // the gradient ring holds two at 256 rows; the third goes over the decoded tiles.
            if (have_acc) {
                __half* tiles = reinterpret_cast<__half*>(smem + L::kB);
                static_assert(3 * BN * kOutK * 2 <= LB * L::kBBytes + LA * L::kSlotA, "output tiles");
                const int group = dw >> 2;
                for (int c = group; c < n_mma / 16; c += DQ) {
                    uint32_t gv[16], uv[16];
                    tmem_ld_32x32b_x16(tmem_acc + tlane + c * 16, gv);
                    tmem_ld_32x32b_x16(tmem_acc + BN + tlane + c * 16, uv);
                    tmem_ld_wait();
                    const int act = p.act;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float a = __uint_as_float(gv[x]), b = __uint_as_float(uv[x]);
                        const int o = (c * 16 + x) * kOutK + j;
                        tiles[o] = __float2half_rn(gate_value(a, act) * b);
                        if (p.Pg) {
                            tiles[BN * kOutK + o] = __float2half_rn(a);
                            tiles[2 * BN * kOutK + o] = __float2half_rn(b);
                        }
                    }
                }
            }
        } else if (p.splits == 1) {
            if (have_acc) {
                __half* stile = reinterpret_cast<__half*>(smem + L::kB) + kb * BN * kOutK;  // [block of k][row][128]
                for (int c = grp; c < n_mma / 16; c += kTurn) {
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(tmem_acc + kb * BN + tlane + c * 16, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        stile[(c * 16 + x) * kOutK + j] = __float2half_rn(__uint_as_float(v[x]));
                }
            }
        } else {
            float* red = reinterpret_cast<float*>(smem + L::kB);
            for (int c = grp; c < BN / 16; c += kTurn) {  // (KM = 1)
                uint32_t v[16];
                if (have_acc && c * 16 < n_mma) {
                    tmem_ld_32x32b_x16(tmem_acc + tlane + c * 16, v);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] = 0u;
                }
#pragma unroll
                for (int x = 0; x < 16; ++x) red[(c * 16 + x) * kOutK + j] = __uint_as_float(v[x]);
            }
        }
        tc_fence_before_sync();
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_acc, L::kTmemCols);
    }

    if constexpr (GATED) {
        if (*tile_ok) {
            const __half* tiles = reinterpret_cast<const __half*>(smem + L::kB);
            const int n0 = blockIdx.y * kOutK;
            for (int w = 0; w < (p.Pg ? 3 : 1); ++w) {
                __half* out = w == 0 ? p.out : (w == 1 ? p.Pg : p.Pu);
                const __half* tile = tiles + w * BN * kOutK;
                for (int o = threadIdx.x; o < rows * 16; o += static_cast<int>(blockDim.x)) {
                    const int rr = o >> 4;
                    const int cc = (o & 15) * 8;
                    __half* dst = out + static_cast<int64_t>(m0 + rr) * p.N + n0 + cc;
                    if (p.vec_out && n0 + cc + 8 <= p.N) {
                        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(tile + rr * kOutK + cc);
                    } else {
                        for (int e = 0; e < 8 && n0 + cc + e < p.N; ++e) dst[e] = tile[rr * kOutK + cc + e];
                    }
                }
            }
        }
        return;
    }
    const int k0 = blockIdx.y * KM * kOutK;
    if (KM > 1 || p.splits == 1) {
        if (*tile_ok) {
            const __half* stile = reinterpret_cast<const __half*>(smem + L::kB);
            for (int o = threadIdx.x; o < rows * 16 * KM; o += static_cast<int>(blockDim.x)) {
                const int rr = o / (16 * KM);
                const int cc = (o % (16 * KM)) * 8;
                const __half* src = stile + (cc / kOutK) * BN * kOutK + rr * kOutK + cc % kOutK;
                __half* dst = p.out + static_cast<int64_t>(m0 + rr) * p.K + k0 + cc;
                if (p.vec_out && k0 + cc + 8 <= p.K) {
                    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
                } else {
                    for (int e = 0; e < 8 && k0 + cc + e < p.K; ++e) dst[e] = src[e];
                }
            }
        }
        return;
    }
    // Sum the cluster's partial tiles in rank order; rank r writes k [r*128/S, (r+1)*128/S) of the tile.
    cluster_sync_all();
    const int S = p.splits;
    const int cw = kOutK / S;
    const int rank = static_cast<int>(cluster_ctarank());
    const float* red = reinterpret_cast<const float*>(smem + L::kB);
    // If any CTA of the cluster stopped early, none writes the tile.
    bool whole = true;
    for (int src = 0; src < S; ++src)
        whole &= __float_as_int(ld_dsmem_f32(const_cast<int*>(tile_ok), static_cast<uint32_t>(src))) != 0;
    for (int o = threadIdx.x; o < cw * rows; o += static_cast<int>(blockDim.x)) {
        const int col = rank * cw + (o % cw);
        const int tok = o / cw;
        if (k0 + col < p.K && whole) {
            float part[8];
#pragma unroll
            for (int src = 0; src < 8; ++src)
                part[src] = src < S ? ld_dsmem_f32(&red[tok * kOutK + col], static_cast<uint32_t>(src)) : 0.f;
            float acc = 0.f;
#pragma unroll
            for (int src = 0; src < 8; ++src) acc += part[src];  // rank order
            p.out[static_cast<int64_t>(m0 + tok) * p.K + k0 + col] = __float2half_rn(acc);
        }
    }
    cluster_sync_all();
}

// dG = dH * u * act'(g), dU = dH * act(g): one pass, eight elements per thread,
// fp32 arithmetic with one rounding of each gradient. Bound by HBM (10 bytes per
// element).
constexpr int kSlopeThreads = 256;

__global__ void __launch_bounds__(kSlopeThreads)
    gated_slopes_kernel(const __half* dH, const __half* g, const __half* u, __half* dG, __half* dU, int64_t vecs,
                        int act) {
    grid_dependency_wait();  // the inputs come from the previous kernels
    grid_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSlopeThreads + threadIdx.x; i < vecs;
         i += static_cast<int64_t>(gridDim.x) * kSlopeThreads) {
        const uint4 vh = ld_v4(dH + 8 * i);
        const uint4 vg = ld_v4(g + 8 * i);
        const uint4 vu = ld_v4(u + 8 * i);
        uint4 og, ou;
        const __half2* h2 = reinterpret_cast<const __half2*>(&vh);
        const __half2* g2 = reinterpret_cast<const __half2*>(&vg);
        const __half2* u2 = reinterpret_cast<const __half2*>(&vu);
        __half2* og2 = reinterpret_cast<__half2*>(&og);
        __half2* ou2 = reinterpret_cast<__half2*>(&ou);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 h = __half22float2(h2[e]), a = __half22float2(g2[e]), b = __half22float2(u2[e]);
            float vx, vy;
            const float dx = gate_slope(a.x, act, &vx), dy = gate_slope(a.y, act, &vy);
            og2[e] = __floats2half2_rn(h.x * b.x * dx, h.y * b.y * dy);
            ou2[e] = __floats2half2_rn(h.x * vx, h.y * vy);
        }
        reinterpret_cast<uint4*>(dG)[i] = og;
        reinterpret_cast<uint4*>(dU)[i] = ou;
    }
}

// ====================================================================== host

struct DgradVariant {
    int bn, km, per_sm, smem;
    const void* fn[2];  // G a multiple of 64, any G
    int (*launch[2])(const CUtensorMap&, const CUtensorMap&, const DgradParams&, dim3, int, cudaStream_t);
};

template <int BN, int LB, int LA, int DQ, int MINB, int KM, bool OG, bool GATED>
int launch_dgrad(const CUtensorMap& m0, const CUtensorMap& m1, const DgradParams& p, dim3 grid, int cluster_x,
                 cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(dgrad_threads(DQ), 1, 1);
    cfg.dynamicSmemBytes = DgradLayout<BN, LB, LA, KM>::kAlloc;
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
    return cudaLaunchKernelEx(&cfg, w4a16_dgrad_kernel<BN, LB, LA, DQ, MINB, KM, OG, GATED>, m0, m1, p) == cudaSuccess
               ? W4A16_OK
               : W4A16_ERR_CUDA;
}

template <int BN, int LB, int LA, int DQ, int MINB, int KM, bool GATED = false>
DgradVariant make_dgrad() {
    return DgradVariant{BN,
                        KM,
                        MINB,
                        DgradLayout<BN, LB, LA, KM>::kAlloc,
                        {reinterpret_cast<const void*>(&w4a16_dgrad_kernel<BN, LB, LA, DQ, MINB, KM, true, GATED>),
                         reinterpret_cast<const void*>(&w4a16_dgrad_kernel<BN, LB, LA, DQ, MINB, KM, false, GATED>)},
                        {&launch_dgrad<BN, LB, LA, DQ, MINB, KM, true, GATED>,
                         &launch_dgrad<BN, LB, LA, DQ, MINB, KM, false, GATED>}};
}

// <gradient rows, gradient stages, decoded stages, decoding groups, CTAs per SM, blocks of k per CTA>;
// the last one is the gated forward pass.
constexpr int kGatedForm = 5;
const DgradVariant kDgrad[] = {make_dgrad<32, 4, 4, 2, 2, 1>(), make_dgrad<64, 4, 4, 2, 2, 1>(),
                               make_dgrad<128, 6, 4, 4, 1, 1>(), make_dgrad<256, 5, 4, 4, 1, 1>(),
                               make_dgrad<256, 4, 3, 4, 1, 2>(), make_dgrad<256, 4, 3, 4, 1, 2, true>()};

int prepare_dgrad_device() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W4A16_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return W4A16_OK;
    for (const DgradVariant& v : kDgrad)
        for (const void* fn : v.fn)
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess ||
                cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared) != cudaSuccess)
                return W4A16_ERR_CUDA;
    // (The slopes kernel runs in front of the product: with the same carve-out the SMs
    // need not drain in between.)
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(&gated_slopes_kernel),
                             cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
        cudaSuccess)
        return W4A16_ERR_CUDA;
    done[dev] = true;
    return W4A16_OK;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows spread evenly over MT tiles, in whole MMA steps.
int64_t rows_of_tile(int64_t M, int64_t MT) { return ((M + MT - 1) / MT + 15) / 16 * 16; }

// The cost of a stage times the rounds over the SMs for `blocks` output blocks of
// km * 128, with the best number of row tiles (*mt): shared-memory traffic at 128
// bytes per clock (decoded tiles written and read, gradient tile written once and
// read per block). A few rows less per tile can save a whole round.
int64_t wide_cost(int64_t M, int64_t blocks, int64_t km, int64_t sms, int64_t* mt) {
    int64_t best = 0;
    const int64_t first = (M + 255) / 256;
    for (int64_t t = first; t <= first + 2; ++t) {
        const int64_t rows = rows_of_tile(M, t);
        if ((t - 1) * rows >= M) continue;  // (an empty tile)
        const int64_t cost = ((blocks * t + sms - 1) / sms) * (256 * km + rows * (1 + km));
        if (best == 0 || cost < best) {
            best = cost;
            *mt = t;
        }
    }
    return best;
}

// The grid's limits: at most 65535 output blocks and row tiles of the launch forms below.
bool dgrad_grid_fits(int64_t M, int64_t K) { return K <= 65535 * int64_t(kOutK) && M <= 65533 * int64_t(256); }

// dA = sum over the sources of dC_i x W_i^T.
int dgrad(int sources, const w4a16_half* const* dC, const uint8_t* const* Wt, const w4a16_half* const* S,
          w4a16_half* dA, int64_t M, int64_t N, int64_t K, int64_t G, cudaStream_t stream) {
    int rc = prepare_dgrad_device();
    if (rc) return rc;
    const int64_t sms = sm_count() > 0 ? sm_count() : 148;
    int vi = M <= 32 ? 0 : (M <= 64 ? 1 : (M <= 128 ? 2 : 3));
    int64_t MT = (M + kDgrad[vi].bn - 1) / kDgrad[vi].bn;
    const int64_t NS = (N + kDepth - 1) / kDepth;
    if (vi == 3) {  // one or two blocks of k per CTA
        int64_t mt1 = 0, mt2 = 0;
        const int64_t one = wide_cost(M, (K + kOutK - 1) / kOutK, 1, sms, &mt1);
        const int64_t two = wide_cost(M, (K + 2 * kOutK - 1) / (2 * kOutK), 2, sms, &mt2);
        vi = two < one ? 4 : 3;
        MT = two < one ? mt2 : mt1;
    }
    const int64_t tile_rows = rows_of_tile(M, MT);
    const DgradVariant& v = kDgrad[vi];
    const int64_t KB = (K + kOutK * v.km - 1) / (kOutK * v.km);
    if (!dgrad_grid_fits(M, K)) return W4A16_ERR_UNSUPPORTED;
    DgradParams p;
    std::memset(&p, 0, sizeof(p));
    for (int i = 0; i < 2; ++i) {
        p.wt[i] = Wt[i < sources ? i : 0];
        p.sc[i] = reinterpret_cast<const __half*>(S[i < sources ? i : 0]);
    }
    p.out = reinterpret_cast<__half*>(dA);
    p.rows = static_cast<int32_t>(M);
    p.tile_rows = static_cast<int32_t>(tile_rows);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + 63) / 64);
    p.NS = static_cast<int32_t>(NS);
    p.stages = static_cast<int32_t>(NS * sources);
    // Few tiles: split the contraction over a cluster while every rank keeps at
    // least eight stages and all CTAs are resident at once.
    int splits = 1;
    const int64_t slots = sms * v.per_sm;
    while (v.km == 1 && splits < 8 && KB * MT * splits * 2 <= slots && p.stages >= splits * 16) splits *= 2;
    p.splits = splits;
    p.prefetch = static_weights_enabled() ? 1 : 0;
    p.vec_out = aligned(dA, 16) ? 1 : 0;
    p.wait_limit = device_wait_limit();
    p.stall_stage = injected_stall_stage();
    CUtensorMap maps[2];
    for (int i = 0; i < 2; ++i) {
        rc = encode_activation_map(&maps[i], dC[i < sources ? i : 0], M, N, static_cast<int>(tile_rows));
        if (rc) return rc;
    }
    const dim3 grid(static_cast<unsigned>(splits), static_cast<unsigned>(KB), static_cast<unsigned>(MT));
    return v.launch[(G % kDepth) ? 1 : 0](maps[0], maps[1], p, grid, splits, stream);
}

}  // namespace

// Whether the gated projections run here rather than on the form with 64 output
// columns per CTA (half the work per CTA and stage, twice the CTAs, and a K split for
// one row tile). Cycles of a launch on either side, fitted to measured launches: a
// CTA's start and epilogue, then its stages (decoding bounds a stage here from below
// at 820), and the exchange of a K split. Measured, this form against the other (calls
// through the Python helper): 2048 x 4096 -> 14336 417 / 470 us, 449 / 499 with the
// projections kept; 700 x 800 -> 9000 27.3 / 39.6; 333 x 1112 -> 2856 (G = 48) 18.5 / 21.6;
// 96 x 4096 -> 14336 39.5 / 41.6; 150 x 4096 -> 4096 36.5 / 19.4; 500 x 2048 -> 4096
// 22.4 / 20.3.
bool wide_gated_takes(int64_t M, int64_t N, int64_t K, int64_t G, int64_t row_tile, int64_t splits,
                      int64_t ctas_per_sm) {
    const int64_t sms = sm_count() > 0 ? sm_count() : 148;
    const int64_t blocks = (N + kOutK - 1) / kOutK, KT = (K + kDepth - 1) / kDepth;
    if (M <= 64 || blocks > 65535) return false;
    int64_t mt = 0;
    wide_cost(M, blocks, 2, sms, &mt);
    const int64_t wide = ((blocks * mt + sms - 1) / sms) *
                         (15000 + KT * std::max<int64_t>(820, 4 * rows_of_tile(M, mt) + 200));
    const int64_t ctas = ((N + 63) / 64) * ((M + row_tile - 1) / row_tile) * splits;
    int64_t stage = row_tile <= 128 ? 1170 : 750;  // (small row tiles: two CTAs per SM)
    if (G % kDepth) stage += stage / 4;            // eight scales per stage and thread
    const int64_t other = ((ctas + sms * ctas_per_sm - 1) / (sms * ctas_per_sm)) * (16000 + (KT / splits) * stage) +
                          (splits > 1 ? 12000 : 0);
    return wide < other;
}

int wide_gated_launch(const w4a16_half* A, const uint8_t* Wt_gate, const w4a16_half* S_gate, const uint8_t* Wt_up,
                      const w4a16_half* S_up, w4a16_half* H, w4a16_half* Pg, w4a16_half* Pu, int64_t M, int64_t N,
                      int64_t K, int64_t G, int act, cudaStream_t stream) {
    int rc = prepare_dgrad_device();
    if (rc) return rc;
    const DgradVariant& v = kDgrad[kGatedForm];
    const int64_t blocks = (N + kOutK - 1) / kOutK;
    int64_t MT = 0;
    wide_cost(M, blocks, 2, sm_count() > 0 ? sm_count() : 148, &MT);
    if (MT > 65535) return W4A16_ERR_UNSUPPORTED;
    DgradParams p;
    std::memset(&p, 0, sizeof(p));
    p.wt[0] = Wt_gate;
    p.wt[1] = Wt_up;
    p.sc[0] = reinterpret_cast<const __half*>(S_gate);
    p.sc[1] = reinterpret_cast<const __half*>(S_up);
    p.out = reinterpret_cast<__half*>(H);
    p.Pg = reinterpret_cast<__half*>(Pg);
    p.Pu = reinterpret_cast<__half*>(Pu);
    p.act = act;
    p.rows = static_cast<int32_t>(M);
    p.tile_rows = static_cast<int32_t>(rows_of_tile(M, MT));
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + 63) / 64);
    p.NS = p.stages = p.KT;
    p.splits = 1;
    p.prefetch = static_weights_enabled() ? 1 : 0;
    p.vec_out = aligned(H, 16) && aligned(Pg, 16) && aligned(Pu, 16) ? 1 : 0;
    p.wait_limit = device_wait_limit();
    p.stall_stage = injected_stall_stage();
    CUtensorMap map;
    rc = encode_activation_map(&map, A, M, K, p.tile_rows);
    if (rc) return rc;
    const dim3 grid(1, static_cast<unsigned>(blocks), static_cast<unsigned>(MT));
    return v.launch[(G % kDepth) ? 1 : 0](map, map, p, grid, 1, stream);
}

namespace {

int gated_slopes(const w4a16_half* dH, const w4a16_half* Pg, const w4a16_half* Pu, w4a16_half* dPg, w4a16_half* dPu,
                 int64_t elements, int act, cudaStream_t stream) {
    const int rc = prepare_dgrad_device();
    if (rc) return rc;
    const int64_t vecs = elements / 8;
    const int64_t cap = static_cast<int64_t>(sm_count() > 0 ? sm_count() : 148) * 8;
    const int64_t blocks = std::min<int64_t>(cap, (vecs + kSlopeThreads - 1) / kSlopeThreads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kSlopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gated_slopes_kernel, reinterpret_cast<const __half*>(dH),
                              reinterpret_cast<const __half*>(Pg), reinterpret_cast<const __half*>(Pu),
                              reinterpret_cast<__half*>(dPg), reinterpret_cast<__half*>(dPu), vecs,
                              act) == cudaSuccess
               ? W4A16_OK
               : W4A16_ERR_CUDA;
}

}  // namespace

int dgrad_device_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_dgrad_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_dgrad_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" int w4a16_gemm_dgrad(const w4a16_half* dC_dev, const uint8_t* Wt_dev, const w4a16_half* S_dev,
                                w4a16_half* dA_dev, int64_t M, int64_t N, int64_t K, int64_t G, uint32_t flags,
                                void* stream) {
    if (!dC_dev || !Wt_dev || !S_dev || !dA_dev || M < 0) return W4A16_ERR_INVALID_ARG;
    if (flags & ~static_cast<uint32_t>(W4A16_FLAG_STATIC_WEIGHTS)) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    if (!aligned(dC_dev, 16) || !aligned(Wt_dev, 16) || !aligned(S_dev, 16) || !aligned(dA_dev, 2))
        return W4A16_ERR_MISALIGNED;
    if (M == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    const CallStaticWeights scope((flags & W4A16_FLAG_STATIC_WEIGHTS) != 0);
    return dgrad(1, &dC_dev, &Wt_dev, &S_dev, dA_dev, M, N, K, G, static_cast<cudaStream_t>(stream));
}

extern "C" int w4a16_gated_gemm_backward(const w4a16_half* dH_dev, const w4a16_half* Pg_dev, const w4a16_half* Pu_dev,
                                         const uint8_t* Wt_gate_dev, const w4a16_half* S_gate_dev,
                                         const uint8_t* Wt_up_dev, const w4a16_half* S_up_dev, w4a16_half* dPg_dev,
                                         w4a16_half* dPu_dev, w4a16_half* dA_dev, int64_t M, int64_t N, int64_t K,
                                         int64_t G, int act, uint32_t flags, void* stream) {
    if (!dH_dev || !Pg_dev || !Pu_dev || !Wt_gate_dev || !S_gate_dev || !Wt_up_dev || !S_up_dev || !dPg_dev ||
        !dPu_dev || !dA_dev || M < 0)
        return W4A16_ERR_INVALID_ARG;
    if (act < W4A16_ACT_IDENTITY || act > W4A16_ACT_SILU) return W4A16_ERR_INVALID_ARG;
    if (flags & ~static_cast<uint32_t>(W4A16_FLAG_STATIC_WEIGHTS)) return W4A16_ERR_INVALID_ARG;
    int rc = check_shape(N, K, G);
    if (rc) return rc;
    if (M >= (int64_t(1) << 31)) return W4A16_ERR_UNSUPPORTED;
    for (const void* q : {static_cast<const void*>(dH_dev), static_cast<const void*>(Pg_dev),
                          static_cast<const void*>(Pu_dev), static_cast<const void*>(Wt_gate_dev),
                          static_cast<const void*>(S_gate_dev), static_cast<const void*>(Wt_up_dev),
                          static_cast<const void*>(S_up_dev), static_cast<const void*>(dPg_dev),
                          static_cast<const void*>(dPu_dev)})
        if (!aligned(q, 16)) return W4A16_ERR_MISALIGNED;
    if (!aligned(dA_dev, 2)) return W4A16_ERR_MISALIGNED;
    if (M == 0) return W4A16_OK;
    rc = check_device();
    if (rc) return rc;
    if (!dgrad_grid_fits(M, K)) return W4A16_ERR_UNSUPPORTED;  // (before the slopes are enqueued)
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = gated_slopes(dH_dev, Pg_dev, Pu_dev, dPg_dev, dPu_dev, M * N, act, s);
    if (rc) return rc;
    const CallStaticWeights scope((flags & W4A16_FLAG_STATIC_WEIGHTS) != 0);
    const w4a16_half* dC[2] = {dPg_dev, dPu_dev};
    const uint8_t* Wt[2] = {Wt_gate_dev, Wt_up_dev};
    const w4a16_half* S[2] = {S_gate_dev, S_up_dev};
    return dgrad(2, dC, Wt, S, dA_dev, M, N, K, G, s);
}
