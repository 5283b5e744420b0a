// mx_attn_decode kernels of E2M1 caches, heads of 128.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_E2M1, 128)

}  // namespace mxk
