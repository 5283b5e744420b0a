// mx_attn_decode kernels of E3M0 caches, heads of 256.
#include "attn_kernel.cuh"

namespace mxk {

AT_DEFINE(GE_E3M0, 256)

}  // namespace mxk
