// ua_latent_l256.cu -- instantiations of the absorbed latent-attention kernel for 256 latent elements.
#include "ua_latent.cuh"

namespace ua {

cudaError_t launch_latent_l256(const LatentParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? launch_latent_t<256, true>(p, s) : launch_latent_t<256, false>(p, s);
}

}  // namespace ua
