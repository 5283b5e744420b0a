// mx_gemv kernels of E3M0 weights.
#include "gemv_kernel.cuh"

namespace mxk {

GvKernel gv_kernel_e3m0(int mode, int bc, int nt) { return gv_pick_mode<GE_E3M0>(mode, bc, nt); }

}  // namespace mxk
