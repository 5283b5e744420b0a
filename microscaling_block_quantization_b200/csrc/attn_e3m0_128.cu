// mx_attn_decode kernels of E3M0 caches, heads of 128.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_E3M0, 128)

}  // namespace mxk
