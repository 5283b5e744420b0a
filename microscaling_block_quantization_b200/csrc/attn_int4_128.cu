// mx_attn_decode kernels of INT4 caches, heads of 128.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_INT4, 128)

}  // namespace mxk
