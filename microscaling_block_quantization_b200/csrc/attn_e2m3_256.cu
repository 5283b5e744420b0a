// mx_attn_decode kernels of E2M3 caches, heads of 256.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(AE_E2M3, 256)

}  // namespace mxk
