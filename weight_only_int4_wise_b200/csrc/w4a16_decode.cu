// Decode-sized (M = 1..16) forms of the gated projections and of the product
// with low-rank adapters on 4-bit weights (include/w4a16.h: w4a16_gated_gemm,
// w4a16_lora_gemm; the Int4GroupwiseGemmPluginV2 page describes the plain product
// that both contain).
//
// The floor is the stream of the codes: to keep up with HBM an SM would have to
// decode about 21 bytes (42 weights) per clock. So the kernel is laid out around
// the instructions per weight and an even share of the weights per SM:
//   - one CTA per SM; a warp owns 16 rows of the MMA's A operand (weights: 8 gate
//     and the same 8 up columns, or 16 columns of the plain product) for every
//     KS-th 128-deep block of K, a CTA P such warp tiles times KS warps each, with P
//     the smallest number of tiles that covers N on all SMs in one wave;
//   - each thread loads its 16-byte chunks (32 k of one column) and scales straight
//     into registers, kAhead of its blocks ahead (no shared-memory ring and no
//     barrier on the weight path), decodes them to fp16(q * s) and feeds them to
//     m16n8k16 MMAs with the tokens as the 8-column operand;
//   - the activations are staged once (or in pieces, when K is long) with only M
//     rows, one bulk copy per row (16 copies of 8 KB arrive in about 2 us; 16-byte
//     copies by the threads took 7): the operand columns past M read row M - 1, and
//     their results are dropped;
//   - the KS partial tiles are added in order through shared memory.
// Measured (gated, 4096 -> 14336, 60.6 MB): 21.6 us at M = 1..8 (2.8 TB/s), 30.2 at M =
// 9..16. No unit is full: DRAM 22-29 %, issue slots 47-52 %, tensor pipe 13-20 %. The
// largest stall is the wait for global loads (4.7-5.2 cycles per issue): what a warp has
// in flight lives in its registers, kAhead blocks of about ten. Between K = 4096 and 8192
// a block of 2048 weights takes a sub-partition 308 cycles with one token tile and 510
// with two; the difference is eight more MMAs, four more shared loads, and the spills of
// the two-tile forms (24 to 44 bytes stored at 72 registers; the one-tile forms have
// none). 1792 warp tiles in CTAs of 13 leave 10 of 148 SMs without work.
// A chunk of 32 k is four words of 8 codes; inside an MMA the order of k is free as
// long as both operands use it, so thread t of a quad takes k = 32t + 8v .. + 7 of
// a block for step w, with v = w for t = 0, 1 and v = w ^ 1 for t = 2, 3: with rows
// 32 bytes (mod 128) apart, the eight lanes of one shared-memory phase then read
// eight distinct 16-byte banks.
//
// Adapters (FORM kLora): after its blocks of K a warp goes on with the adapter
// ranks as more k: for each token m (every KS-th) the rows of LB[ids[m]] of its 16
// columns are the A operand, and V[m] in fp16 is the token's column of the B
// operand, zeros the other seven. An infinity or NaN of LB would turn those zeros
// into NaN: it is left out of the MMA, and the epilogue adds its terms to the
// tokens that use that adapter.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/w4a16.h"
#include "dequant.cuh"
#include "epilogue.cuh"
#include "once.h"
#include "ptx.cuh"
#include "w4a16_internal.h"
#include "waits.cuh"

namespace w4a16 {

namespace {

constexpr int kMaxWarps = 28;  // 896 threads: 72 registers each, one CTA per SM
constexpr int kAhead = 3;      // blocks a thread has in flight
constexpr int kBlockK = 128;
constexpr int kMaxSmem = 224 * 1024;

enum DecodeForm { kGated = 0, kLora = 1 };

struct DecodeParams {
    const uint8_t* wt[2];  // tiled weights: gate and up, or the shared matrix twice
    const __half* sc[2];
    const __half* A;
    __half* C;             // H, or C
    __half* Pg;            // gated: the projections to keep (both or neither)
    __half* Pu;
    int32_t M, N, K, G;
    int32_t ngroups, KT, KB;  // groups, 64-deep tiles, 128-deep blocks
    int32_t tiles;            // warp tiles of all of N
    int32_t P, KS;            // warp tiles per CTA, warps per tile
    int32_t iters;            // blocks of a warp: ceil(KB / KS)
    int32_t piece;            // iterations whose activations are staged together (a multiple of kAhead)
    int32_t row_bytes;        // staged activation row
    uint32_t g_magic;         // floor(k / G) == (k * g_magic) >> 32
    int32_t act, prefetch;
    long long wait_limit;
    LoraOperands lora;
};

__device__ int g_decode_status;  // latched device-side error (0 = none)

// 16 bytes of codes, read once, without a place in L1.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Nonzero if a half of x is an infinity or NaN (all-ones exponent field).
__device__ __forceinline__ uint32_t nonfinite(uint32_t x) { return ((x & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }

__device__ __forceinline__ uint32_t keep_finite(uint32_t x) { return x & ~((nonfinite(x) >> 15) * 0xFFFFu); }

// FINE: G is not a multiple of 32, so a chunk may touch two scale groups (one per 16 k).
template <int MT, int FORM, bool FINE>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) w4a16_decode_kernel(const __grid_constant__ DecodeParams p) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int fix;     // adapters: an infinity or NaN was left out
    __shared__ int failed;  // the wait for the activations ran out
    __shared__ __align__(8) uint64_t landed;
    constexpr bool LORA = FORM == kLora;
    constexpr int kNS = FINE ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = warp % p.P, kh = warp / p.P;
    const int gt = blockIdx.x * p.P + tile;
    const bool active = gt < p.tiles;
    // The columns of this thread's two MMA rows (g and g + 8).
    const int na = LORA ? gt * 16 + g : gt * 8 + g;
    const int nb = LORA ? na + 8 : na;
    float4* red = reinterpret_cast<float4*>(sm + p.M * p.row_bytes);

    struct Block {
        uint4 a, b;
        uint16_t sa[kNS], sb[kNS];
    };
    // Running state of the loads, in 32 bits (the weights are below 4 GB): the next
    // block's byte offset, the same for both rows but for a constant, its first k,
    // and how many blocks are left. (The loads are volatile: left free, the compiler
    // moves the scale loads down to their use and waits there for each of them.)
    uint32_t w_off = static_cast<uint32_t>(((na >> 7) * static_cast<int64_t>(p.KT) + 2 * kh + (t >> 1)) * 4096 +
                                           (t & 1) * 2048 + (na & 127) * 16);
    const uint32_t w_step = static_cast<uint32_t>(p.KS) * 8192u;
    uint32_t k_next = static_cast<uint32_t>(kh * kBlockK + 32 * t);
    const uint32_t row_step = 2u * static_cast<uint32_t>(p.N);  // bytes of a scale row
    const uint32_t s_off = 2u * static_cast<uint32_t>(na);
    const uint32_t sb_more = LORA && nb < p.N ? 16u : 0u;       // (a row past N reads row g's scales; it is not written)
    const uint8_t* wa = p.wt[0];
    const uint8_t* wb = LORA ? wa + 128 : p.wt[1];
    const uint8_t* sa = reinterpret_cast<const uint8_t*>(p.sc[0]);
    const uint8_t* sb = LORA ? sa : reinterpret_cast<const uint8_t*>(p.sc[1]);
    const int blocks = active && kh < p.KB ? (p.KB - kh + p.KS - 1) / p.KS : 0;  // this warp's
    int to_load = blocks;
    constexpr bool early = LORA;  // (its loads are not behind the dependency wait)
    auto load = [&](Block& x) {
        if (to_load > 0) {  // (the same for the whole warp)
            --to_load;
            // K may end in the middle of the last block: a chunk that does not exist
            // reads the block's first tile, with scales of zero.
            const bool missing = k_next >= static_cast<uint32_t>(p.KT) * 64u;
            const uint32_t off = missing ? w_off - 4096u : w_off;
            x.a = early ? ld_cg_v4(wa + off) : ld_once_v4(wa + off);
            x.b = early ? ld_cg_v4(wb + off) : ld_once_v4(wb + off);
#pragma unroll
            for (int q = 0; q < kNS; ++q) {
                const uint32_t gi = min(__umulhi(k_next + 16 * q, p.g_magic), static_cast<uint32_t>(p.ngroups - 1));
                const uint32_t so = gi * row_step + s_off;
                x.sa[q] = early ? ld_cg_u16(sa + so) : ld_u16(sa + so);
                x.sb[q] = early ? ld_cg_u16(sb + (so + sb_more)) : ld_u16(sb + (so + sb_more));
                if (missing) x.sa[q] = x.sb[q] = 0;
            }
            w_off += w_step;
            k_next += p.KS * kBlockK;
        }
    };

    Block blk[kAhead];
    if (threadIdx.x == 0) {
        fix = 0;
        failed = 0;
        mbar_init(&landed, 1);
        fence_mbar_init();
    }
    // (Adapters: this launch follows the kernel that makes V, which lets it start only
    // once everything before it is complete; weights, scales and activations are read
    // at once, not through L1, and it waits for that kernel just before it reads V.)
    if (LORA || p.prefetch) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) load(blk[d]);
    }
    grid_launch_dependents();
    if (!LORA) grid_dependency_wait();
    if (!LORA && !p.prefetch) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) load(blk[d]);
    }

    float acc[2][MT][4];  // two chains: the even and the odd 16-deep steps
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[u][j][0] = acc[u][j][1] = acc[u][j][2] = acc[u][j][3] = 0.f;
    // Where this thread's units of a row start, for even and odd steps.
    uint32_t aeven[MT], aodd[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const uint32_t base = smem_addr(sm) + static_cast<uint32_t>(min(8 * j + g, p.M - 1) * p.row_bytes + 64 * t);
        aeven[j] = base + 16 * (t >> 1);
        aodd[j] = base - 16 * (t >> 1);
    }

    for (int i0 = 0; i0 < p.iters; i0 += p.piece) {
        // Stage the activations of blocks [i0 * KS, (i0 + piece) * KS): zero past K.
        {
            const int k0 = i0 * p.KS * kBlockK;
            const int blocks = min(p.KB - i0 * p.KS, p.piece * p.KS);
            const int have = min(p.K - k0, blocks * kBlockK);  // (a multiple of 8)
            __syncthreads();  // the barrier is set up, or the piece before is consumed
            if (threadIdx.x == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(&landed, static_cast<uint32_t>(p.M * have * 2));
                for (int m = 0; m < p.M; ++m)
                    bulk_g2s(sm + m * p.row_bytes, p.A + static_cast<int64_t>(m) * p.K + k0,
                             static_cast<uint32_t>(have * 2), &landed);
            }
            const int tail = (blocks * kBlockK - have) / 8;  // 16-byte units past K
            for (int c = threadIdx.x; c < p.M * tail; c += static_cast<int>(blockDim.x))
                *reinterpret_cast<uint4*>(sm + (c / tail) * p.row_bytes + have * 2 + (c % tail) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            const uint32_t par = static_cast<uint32_t>(i0 / p.piece) & 1u;
            if (!warp_wait_phase(&landed, par, &failed, p.wait_limit, &g_decode_status))
                warp_drain_phase(&landed, par, &g_decode_status);  // (no copy may outlive the CTA)
            if (tail > 0) __syncthreads();  // (the zeros)
        }
        const int iend = min(p.iters, i0 + p.piece);
        uint32_t off = static_cast<uint32_t>(kh) * 256;  // this warp's block in the staged piece
        int left = min(iend, blocks) - i0;               // its blocks of the piece
        for (int i = i0; i < iend; i += kAhead) {
#pragma unroll
            for (int d = 0; d < kAhead; ++d) {
                Block& x = blk[d];
                if (left > 0) {  // (the same for the whole warp)
                    // (steps in this thread's order)
                    const bool odd = t & 2;
                    const uint32_t aw[4] = {odd ? x.a.y : x.a.x, odd ? x.a.x : x.a.y, odd ? x.a.w : x.a.z,
                                            odd ? x.a.z : x.a.w};
                    const uint32_t bw[4] = {odd ? x.b.y : x.b.x, odd ? x.b.x : x.b.y, odd ? x.b.w : x.b.z,
                                            odd ? x.b.z : x.b.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint4 qa = dequant_word(aw[w], __half2half2(__ushort_as_half(x.sa[FINE ? w >> 1 : 0])));
                        const uint4 qb = dequant_word(bw[w], __half2half2(__ushort_as_half(x.sb[FINE ? w >> 1 : 0])));
                        const uint32_t f0[4] = {qa.x, qb.x, qa.y, qb.y};
                        const uint32_t f1[4] = {qa.z, qb.z, qa.w, qb.w};
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            const uint4 y = lds128((w & 1 ? aodd[j] : aeven[j]) + off + 16 * w);
                            mma_m16n8k16(acc[0][j], f0, y.x, y.y);
                            mma_m16n8k16(acc[1][j], f1, y.z, y.w);
                        }
                    }
                    load(x);
                    off += static_cast<uint32_t>(p.KS) * 256;
                    --left;
                }
            }
        }
    }

    if constexpr (LORA) {
        grid_dependency_wait();  // V is complete (and the output may be written)
        const int R = p.lora.R;
        bool bad = false;
        for (int m = kh; m < p.M; m += p.KS) {
            const int id = __ldcg(p.lora.ids + m);
            if (id < 0 || id >= p.lora.L || !active) continue;
            const __half* la = p.lora.LB + (static_cast<int64_t>(id) * p.N + na) * R + 8 * t;
            const __half* lb = p.lora.LB + (static_cast<int64_t>(id) * p.N + (nb < p.N ? nb : na)) * R + 8 * t;
            const __half* v = p.lora.V + static_cast<int64_t>(m) * R + 8 * t;
#pragma unroll 2
            for (int r = 0; r < R; r += 32) {
                uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa, y = xa;
                if (r + 8 * t < R) {
                    xa = __ldcg(reinterpret_cast<const uint4*>(la + r));
                    xb = __ldcg(reinterpret_cast<const uint4*>(lb + r));
                    if (g == (m & 7)) y = __ldcg(reinterpret_cast<const uint4*>(v + r));
                }
                if (nonfinite(xa.x) | nonfinite(xa.y) | nonfinite(xa.z) | nonfinite(xa.w) | nonfinite(xb.x) |
                    nonfinite(xb.y) | nonfinite(xb.z) | nonfinite(xb.w)) {
                    bad = true;
                    xa = make_uint4(keep_finite(xa.x), keep_finite(xa.y), keep_finite(xa.z), keep_finite(xa.w));
                    xb = make_uint4(keep_finite(xb.x), keep_finite(xb.y), keep_finite(xb.z), keep_finite(xb.w));
                }
                __syncwarp();
                const uint32_t f0[4] = {xa.x, xb.x, xa.y, xb.y};
                const uint32_t f1[4] = {xa.z, xb.z, xa.w, xb.w};
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    if (j == (m >> 3)) {
                        mma_m16n8k16(acc[0][j], f0, y.x, y.y);
                        mma_m16n8k16(acc[1][j], f1, y.z, y.w);
                    }
                }
            }
        }
        if (bad) fix = 1;
    }

#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][j][e] += acc[1][j][e];
    if (kh > 0) {
#pragma unroll
        for (int j = 0; j < MT; ++j)
            red[(((kh - 1) * p.P + tile) * MT + j) * 32 + lane] =
                make_float4(acc[0][j][0], acc[0][j][1], acc[0][j][2], acc[0][j][3]);
    }
    __syncthreads();
    if (kh > 0 || !active || *const_cast<volatile int*>(&failed)) return;
    for (int s = 1; s < p.KS; ++s) {  // in order: deterministic
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const float4 v = red[(((s - 1) * p.P + tile) * MT + j) * 32 + lane];
            acc[0][j][0] += v.x;
            acc[0][j][1] += v.y;
            acc[0][j][2] += v.z;
            acc[0][j][3] += v.w;
        }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = 8 * j + 2 * t + e;
            if (m >= p.M) continue;
            const int64_t o = static_cast<int64_t>(m) * p.N;
            float x = acc[0][j][e], y = acc[0][j][2 + e];
            if constexpr (LORA) {
                if (fix) {
                    const int id = __ldcg(p.lora.ids + m);
                    if (id >= 0 && id < p.lora.L) {
                        for (int r = 0; r < p.lora.R; ++r) {
                            const float v = __half2float(__ldcg(p.lora.V + static_cast<int64_t>(m) * p.lora.R + r));
                            const __half* col = p.lora.LB + (static_cast<int64_t>(id) * p.N + na) * p.lora.R + r;
                            const float l0 = __half2float(__ldcg(col));
                            if (!isfinite(l0)) x += v * l0;
                            if (nb < p.N) {
                                const float l1 = __half2float(__ldcg(col + static_cast<int64_t>(8) * p.lora.R));
                                if (!isfinite(l1)) y += v * l1;
                            }
                        }
                    }
                }
                p.C[o + na] = __float2half_rn(x);
                if (nb < p.N) p.C[o + nb] = __float2half_rn(y);
            } else {
                p.C[o + na] = __float2half_rn(gate_value(x, p.act) * y);
                if (p.Pg) {
                    p.Pg[o + na] = __float2half_rn(x);
                    p.Pu[o + na] = __float2half_rn(y);
                }
            }
        }
    }
}

// ====================================================================== host

// floor(k / G) as a multiply-shift for every k < kend: with magic = (2^32 + e) / G,
// 0 <= e < G, k * magic / 2^32 = k / G + k * e / (G * 2^32) floors to floor(k / G)
// whenever k * e < 2^32 (the fractional part of k / G is at most (G - 1) / G). One
// group needs no multiplier. False if some k might come out wrong (K above 2^32 / G).
bool group_magic(int64_t G, int64_t kend, uint32_t* magic) {
    *magic = 0;
    if (G >= kend) return true;
    const uint64_t g = static_cast<uint64_t>(G);
    const uint64_t m = ((uint64_t(1) << 32) + g - 1) / g;
    const uint64_t e = m * g - (uint64_t(1) << 32);
    if (e != 0 && static_cast<uint64_t>(kend) > ((uint64_t(1) << 32) - 1) / e) return false;
    *magic = static_cast<uint32_t>(m);
    return true;
}

typedef void (*DecodeKernel)(DecodeParams);

int decode_launch(DecodeParams& p, DecodeForm form, int64_t M, int64_t N, int64_t K, int64_t G, cudaStream_t stream) {
    static const DecodeKernel kernels[8] = {
        w4a16_decode_kernel<1, kGated, false>, w4a16_decode_kernel<1, kGated, true>,
        w4a16_decode_kernel<2, kGated, false>, w4a16_decode_kernel<2, kGated, true>,
        w4a16_decode_kernel<1, kLora, false>,  w4a16_decode_kernel<1, kLora, true>,
        w4a16_decode_kernel<2, kLora, false>,  w4a16_decode_kernel<2, kLora, true>};
    static OncePerDevice prepared[8];
    const int mt = M <= 8 ? 1 : 2;
    const int vi = 4 * form + 2 * (mt - 1) + (G % 32 ? 1 : 0);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W4A16_ERR_CUDA;
    const int rc = prepared[vi].run(dev, [&] {
        const void* fn = reinterpret_cast<const void*>(kernels[vi]);
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) == cudaSuccess &&
                       cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                            cudaSharedmemCarveoutMaxShared) == cudaSuccess
                   ? W4A16_OK
                   : W4A16_ERR_CUDA;
    });
    if (rc) return rc;
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.G = static_cast<int32_t>(G);
    p.ngroups = static_cast<int32_t>((K + G - 1) / G);
    p.KT = static_cast<int32_t>((K + 63) / 64);
    p.KB = (p.KT + 1) / 2;
    const int64_t tiles = form == kGated ? N / 8 : (N + 15) / 16;
    const int sms = sm_count() > 0 ? sm_count() : 148;
    // One wave of one CTA per SM if the warps suffice; then as many warps per tile
    // as fit, but no more than its blocks need in the fewest rounds.
    const int64_t P = std::min<int64_t>(kMaxWarps, (tiles + sms - 1) / sms);
    const int ks = static_cast<int>(std::min<int64_t>(kMaxWarps / P, p.KB));
    p.iters = (p.KB + ks - 1) / ks;
    p.KS = (p.KB + p.iters - 1) / p.iters;
    p.P = static_cast<int32_t>(P);
    p.tiles = static_cast<int32_t>(tiles);
    // Activations staged together: all of K if it fits beside the partial tiles,
    // else pieces of whole rounds of the block buffers (with fewer warps per tile
    // if one such piece would not fit either).
    int red = 0, blocks = 0;  // bytes of the partial tiles; 128-deep blocks of activations that fit
    for (;; --p.KS) {
        red = (p.KS - 1) * p.P * mt * 512;
        blocks = ((kMaxSmem - red) / p.M - 32) / 256;
        if (blocks >= p.KB || blocks >= p.KS * kAhead || p.KS == 1) break;
    }
    p.iters = (p.KB + p.KS - 1) / p.KS;
    p.piece = blocks >= p.KB ? (p.iters + kAhead - 1) / kAhead * kAhead : blocks / p.KS / kAhead * kAhead;
    p.row_bytes = std::min(p.piece * p.KS, p.KB) * 256 + 32;
    if (!group_magic(G, static_cast<int64_t>(p.KB) * kBlockK, &p.g_magic)) return W4A16_ERR_UNSUPPORTED;
    p.wait_limit = device_wait_limit();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((tiles + P - 1) / P), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(p.P * p.KS * 32), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.M * p.row_bytes + red);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernels[vi], p) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

}  // namespace

bool decode_takes(int64_t M, int64_t N, int64_t K, int64_t G) {
    uint32_t magic;
    return M <= kSkinnyMaxM && w4a16_tiled_bytes(K, N) < (int64_t(1) << 32) &&
           group_magic(G, (K + 127) / 128 * 128, &magic);
}

int decode_device_status(bool clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_decode_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

int decode_gated_launch(const void* A, const uint8_t* Wt_gate, const void* S_gate, const uint8_t* Wt_up,
                        const void* S_up, void* H, void* Pg, void* Pu, int64_t M, int64_t N, int64_t K, int64_t G,
                        int act, cudaStream_t stream) {
    DecodeParams p;
    std::memset(&p, 0, sizeof(p));
    p.wt[0] = Wt_gate;
    p.wt[1] = Wt_up;
    p.sc[0] = reinterpret_cast<const __half*>(S_gate);
    p.sc[1] = reinterpret_cast<const __half*>(S_up);
    p.A = reinterpret_cast<const __half*>(A);
    p.C = reinterpret_cast<__half*>(H);
    p.Pg = reinterpret_cast<__half*>(Pg);
    p.Pu = reinterpret_cast<__half*>(Pu);
    p.act = act;
    p.prefetch = static_weights_enabled() ? 1 : 0;
    return decode_launch(p, kGated, M, N, K, G, stream);
}

int decode_lora_launch(const LoraOperands& lora, const void* A, const uint8_t* Wt, const void* S, void* C, int64_t M,
                       int64_t N, int64_t K, int64_t G, cudaStream_t stream) {
    DecodeParams p;
    std::memset(&p, 0, sizeof(p));
    p.wt[0] = p.wt[1] = Wt;
    p.sc[0] = p.sc[1] = reinterpret_cast<const __half*>(S);
    p.A = reinterpret_cast<const __half*>(A);
    p.C = reinterpret_cast<__half*>(C);
    p.lora = lora;
    return decode_launch(p, kLora, M, N, K, G, stream);
}

}  // namespace w4a16
