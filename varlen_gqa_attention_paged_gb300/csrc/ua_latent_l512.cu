// ua_latent_l512.cu -- instantiations of the absorbed latent-attention kernel for 512 latent elements.
#include "ua_latent.cuh"

namespace ua {

cudaError_t launch_latent_l512(const LatentParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? launch_latent_t<512, true>(p, s) : launch_latent_t<512, false>(p, s);
}

}  // namespace ua
