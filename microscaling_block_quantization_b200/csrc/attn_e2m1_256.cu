// mx_attn_decode kernels of E2M1 caches, heads of 256.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_E2M1, 256)

}  // namespace mxk
