// The gated and adapter forms of the tensor-core product (w4a16_gemm_kernel.cuh) in
// a module of their own: it is loaded at the first call of one of them, and the
// plain products load as fast as without it (first call 6 ms; 26 with all forms in
// one module).
#include "w4a16_gemm_kernel.cuh"

namespace w4a16 {

GemmKernel gated_kernel(int variant, int any_group) { return kernel_of<4, kGated>(variant, any_group); }

GemmKernel lora_kernel(int variant, int any_group) { return kernel_of<4, kLora>(variant, any_group); }

int forms_device_status(bool clear) { return read_gemm_status(clear); }

}  // namespace w4a16
