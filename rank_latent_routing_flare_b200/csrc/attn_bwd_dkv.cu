// The dK/dV pass of the attention's backward.
#include "attn_bwd_kernel.cuh"

namespace flare {

cudaError_t launch_attn_bwd_dkv(const AttnMaps& m, const AttnBwdParams& p, cudaStream_t s) {
  return launch_attn_bwd_pass<true>(m.k, m.v, m.q, m.dy, p, s);
}

}  // namespace flare
