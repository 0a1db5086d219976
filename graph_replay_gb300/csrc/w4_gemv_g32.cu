// w4_gemv_g32.cu -- the few-token kernels for groups of 32 columns (w4_gemv.cuh).
#include "w4_gemv.cuh"

namespace gd {
const void* w4_gemv_kernel_32(int parts, int nb, int kind) { return w4_gemv_kernel<32>(parts, nb, kind); }
}  // namespace gd
