// ua_latent_l512.cu -- instantiations of the absorbed latent-attention kernel for 512 latent elements.
#include "ua_latent.cuh"

namespace ua {

cudaError_t launch_latent_l512(const LatentParams& p, bool bf16, cudaStream_t s) {
  return launch_latent_any<512>(p, bf16, s);
}

}  // namespace ua
