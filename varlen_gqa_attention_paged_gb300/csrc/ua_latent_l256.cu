// ua_latent_l256.cu -- instantiations of the absorbed latent-attention kernel for 256 latent elements.
#include "ua_latent.cuh"

namespace ua {

cudaError_t launch_latent_l256(const LatentParams& p, bool bf16, cudaStream_t s) {
  return launch_latent_any<256>(p, bf16, s);
}

}  // namespace ua
