// w4_gemv_g128.cu -- the few-token kernels for groups of 128 columns (w4_gemv.cuh).
#include "w4_gemv.cuh"

namespace gd {
const void* w4_gemv_kernel_128(int parts, int nb, int kind) { return w4_gemv_kernel<128>(parts, nb, kind); }
}  // namespace gd
