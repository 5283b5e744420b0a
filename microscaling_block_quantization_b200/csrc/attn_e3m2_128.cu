// mx_attn_decode kernels of E3M2 caches, heads of 128.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(AE_E3M2, 128)

}  // namespace mxk
