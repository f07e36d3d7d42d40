// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w4a16.h"

namespace w4a16 {

// W4A16_OK if the current device is an sm_100 part this library was built for,
// W4A16_ERR_UNSUPPORTED otherwise (including "no CUDA device").
int check_device();

// Streaming multiprocessors of the current device (0 if unknown).
int sm_count();

// Whether the caller declared weights and scales static (w4a16_set_static_weights).
bool static_weights_enabled();

// W4A16_FLAG_STATIC_WEIGHTS for the duration of one call on this host thread.
extern thread_local int t_call_static_weights;
struct CallStaticWeights {
    explicit CallStaticWeights(bool on) { t_call_static_weights = on ? 1 : 0; }
    ~CallStaticWeights() { t_call_static_weights = 0; }
};

// A tiled tensor map over fp16 elements [outer, inner] (row stride in bytes),
// box [box_outer, box_inner], no swizzle, zero fill outside the tensor.
// W4A16_OK, or W4A16_ERR_CUDA if the driver's encoder is missing or refuses.
int make_half_map_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes,
                     uint32_t box_inner, uint32_t box_outer);

// A tiled tensor map over activations A [rows, K] fp16 with a {64, box_rows}
// box, the 128-byte swizzle and zero fill past the tensor, as the tensor-core
// kernels stage them. Encoded maps are kept in a small per-thread cache keyed
// by (device, address, rows, K, box_rows), so repeated calls on the same
// buffers skip the encoder.
// encode_activation_map is the encoder alone.
int encode_activation_map(CUtensorMap* map, const void* A, int64_t rows, int64_t K, int box_rows);
int activation_map(CUtensorMap* map, const void* A, int64_t rows, int64_t K, int box_rows);

// The grouped-expert GEMM with an activation epilogue (w4a16_grouped_gemm_act).
int grouped_gemm_act(const w4a16_half* A_dev, const uint8_t* const* Wt, const w4a16_half* const* S,
                     const int32_t* offsets_dev, w4a16_half* C_dev, int64_t E, int64_t total_rows, int64_t N,
                     int64_t K, int64_t G, int act, cudaStream_t stream);

// The expert-layer kernels' latched device status (0 = none, -1 if it could not be read).
int moe_device_status(bool clear);

// The quantiser kernel's latched device status (0 = none, -1 if it could not be read).
int quant_device_status(bool clear);

// The adapter kernel's latched device status (0 = none, -1 if it could not be read).
int lora_device_status(bool clear);

// What the shared product adds for low-rank adapters: V [M, R] fp16 (scaled
// down-projections), LB [L, N, R], and for the tensor-core form the distinct
// adapters of each token tile.
struct LoraOperands {
    const __half* LB;
    const int32_t* ids;   // [M], negative or >= L: no adapter
    const __half* V;
    const int32_t* list;  // [tiles][tile rows]
    const int32_t* count; // [tiles]
    int32_t L, R;
};

// The transposed product's latched device status (0 = none, -1 if it could not be read).
int dgrad_device_status(bool clear);

// The bound of every device wait in SM clock cycles, and the stage whose ready
// signal is withheld (-1: none): w4a16_set_fault_injection.
long long device_wait_limit();
int injected_stall_stage();

// Argument checks that the products share: sizes of a weight matrix, alignment.
int check_shape(int64_t N, int64_t K, int64_t G);

// Decode-sized products (M <= kSkinnyMaxM) run on the skinny kernel.
constexpr int kSkinnyMaxM = 16;

struct SkinnyPlan {
    int mt;             // token tiles of 8 rows (1 or 2)
    int threads;        // threads per CTA (256 per K half)
    int splits;         // CTAs along K in one cluster
    int depth;          // 128-deep K blocks in flight per thread (2 to 8)
    int grid_x, grid_y;
    int act_stride;     // staged activation row, in halves
    int scale_rows;     // staged scale rows
    int smem;           // dynamic shared memory per CTA
    uint32_t g_magic;   // multiply-shift constant for floor(k / G)
    int post_scale;     // 1 when every 128-deep K block lies in one scale group
};

// W4A16_OK and a plan, or W4A16_ERR_UNSUPPORTED if the shape needs the general kernel.
int skinny_plan(int64_t M, int64_t N, int64_t K, int64_t G, SkinnyPlan* plan);

// The skinny plan for a given K split (1..8 CTAs per cluster), K halves per CTA
// (1 or 2; 2 only for one token tile) and ring depth (deep = 0: four blocks in
// flight per CTA, 1: eight). W4A16_ERR_UNSUPPORTED when that form does not
// exist for the shape (more splits than 128-deep K blocks, shared memory).
int skinny_plan_fill(int64_t M, int64_t N, int64_t K, int64_t G, int splits, int kh, int deep, SkinnyPlan* plan);

// The skinny kernel's latched device status (0 = none, -1 if it could not be read).
int skinny_device_status(bool clear);

int skinny_launch(const SkinnyPlan& plan, const void* A, const uint8_t* Wt, const void* S, void* C, int64_t M,
                  int64_t N, int64_t K, int64_t G, cudaStream_t stream);

// The skinny plan of the grouped form: the smallest K split whose staged
// activations fit (the experts' column tiles already fill the grid).
int skinny_plan_grouped(int64_t total_rows, int64_t N, int64_t K, int64_t G, SkinnyPlan* plan);

// The decode-sized forms (M <= kSkinnyMaxM) of the gated projections (H [M, N],
// and the projections Pg and Pu if not null) and of the product with adapters
// (right after the kernel that makes V, on the same stream).
int decode_gated_launch(const void* A, const uint8_t* Wt_gate, const void* S_gate, const uint8_t* Wt_up,
                        const void* S_up, void* H, void* Pg, void* Pu, int64_t M, int64_t N, int64_t K, int64_t G,
                        int act, cudaStream_t stream);
int decode_lora_launch(const LoraOperands& lora, const void* A, const uint8_t* Wt, const void* S, void* C, int64_t M,
                       int64_t N, int64_t K, int64_t G, cudaStream_t stream);

// The gated projections of many rows, 128 output columns per CTA, and whether that
// form is the faster one for the shape, given the other form's launch.
bool wide_gated_takes(int64_t M, int64_t N, int64_t K, int64_t G, int64_t row_tile, int64_t splits,
                      int64_t ctas_per_sm);
int wide_gated_launch(const w4a16_half* A, const uint8_t* Wt_gate, const w4a16_half* S_gate, const uint8_t* Wt_up,
                      const w4a16_half* S_up, w4a16_half* H, w4a16_half* Pg, w4a16_half* Pu, int64_t M, int64_t N,
                      int64_t K, int64_t G, int act, cudaStream_t stream);

int decode_device_status(bool clear);

// Whether they take the shape (a scale group's index must fit their multiply-shift,
// the weights' offsets 32 bits); the tensor-core kernel takes any.
bool decode_takes(int64_t M, int64_t N, int64_t K, int64_t G);

// Grouped-expert form of the skinny kernel (grid z = expert) for at most 16
// gathered rows in total (plan from skinny_plan_grouped): rows
// [off[e], off[e+1]) of A and C use Wt[e] and S[e] (host arrays of E device
// pointers); the activation act (W4A16_ACT_*) applies to the fp16 result.
// Malformed offsets (or a segment longer than the plan's token tiles) latch
// W4A16_ERR_BAD_OFFSETS in the skinny status word and write nothing.
int skinny_grouped_launch(const SkinnyPlan& plan, const void* A, const uint8_t* const* Wt, const void* const* S,
                          const int32_t* offsets, void* C, int64_t E, int64_t total_rows, int64_t N, int64_t K,
                          int64_t G, int act, cudaStream_t stream);

// How the product with adapters will launch, and the launch itself (right after
// the kernel that makes V, on the same stream).
struct LoraPlan {
    int tile_rows;  // token tile of the tensor-core form; 0 for the decode-sized form
    int splits;
    int grid_y, grid_z;
};
int lora_plan(int64_t M, int64_t N, int64_t K, int64_t G, LoraPlan* plan);
int lora_product(const LoraPlan& plan, const LoraOperands& lora, const w4a16_half* A, const uint8_t* Wt,
                 const w4a16_half* S, w4a16_half* C, int64_t M, int64_t N, int64_t K, int64_t G, cudaStream_t stream);

}  // namespace w4a16
