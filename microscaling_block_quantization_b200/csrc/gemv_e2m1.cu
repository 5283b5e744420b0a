// mx_gemv kernels of E2M1 weights.
#include "gemv_kernel.cuh"

namespace mxk {

GvKernel gv_kernel_e2m1(int mode, int bc, int nt) { return gv_pick_mode<GE_E2M1>(mode, bc, nt); }

}  // namespace mxk
