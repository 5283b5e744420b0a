// mx_attn_decode kernels of INT4 caches, heads of 256.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_INT4, 256)

}  // namespace mxk
