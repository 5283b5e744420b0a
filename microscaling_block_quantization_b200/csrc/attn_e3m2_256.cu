// mx_attn_decode kernels of E3M2 caches, heads of 256.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(AE_E3M2, 256)

}  // namespace mxk
