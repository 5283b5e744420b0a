// mx_attn_decode kernels of E2M3 caches, heads of 128.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(AE_E2M3, 128)

}  // namespace mxk
