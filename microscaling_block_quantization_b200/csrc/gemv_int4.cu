// mx_gemv kernels of two's complement INT4 weights.
#include "gemv_kernel.cuh"

namespace mxk {

GvKernel gv_kernel_int4(int mode, int bc, int nt) { return gv_pick_mode<GE_INT4>(mode, bc, nt); }

}  // namespace mxk
