// mx_gemv kernels of unsigned INT4 weights.
#include "gemv_kernel.cuh"

namespace mxk {

GvKernel gv_kernel_uint4(int mode, int bc, int nt) { return gv_pick_mode<GE_UINT4>(mode, bc, nt); }

}  // namespace mxk
