// The attention's kernels for layers with a window (a translation unit of their own, so that
// they compile beside the others).
#include "tree_attn_kernel.cuh"

namespace dfl2 {

cudaError_t launch_window_attn(const AttnArgs& a, const dfl2_cache* c, cudaStream_t s) {
  return c->dtype == DFL2_F16 ? launch_attn_d<__half, true>(a, c, s)
                              : launch_attn_d<__nv_bfloat16, true>(a, c, s);
}

}  // namespace dfl2
