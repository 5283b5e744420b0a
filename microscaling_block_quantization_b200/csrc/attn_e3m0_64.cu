// mx_attn_decode kernels of E3M0 caches, heads of 64.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_E3M0, 64)

}  // namespace mxk
