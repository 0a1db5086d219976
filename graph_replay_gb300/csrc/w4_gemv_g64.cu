// w4_gemv_g64.cu -- the few-token kernels for groups of 64 columns (w4_gemv.cuh).
#include "w4_gemv.cuh"

namespace gd {
const void* w4_gemv_kernel_64(int parts, int nb, int kind) { return w4_gemv_kernel<64>(parts, nb, kind); }
}  // namespace gd
