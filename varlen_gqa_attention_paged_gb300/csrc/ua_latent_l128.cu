// ua_latent_l128.cu -- instantiations of the absorbed latent-attention kernel for 128 latent elements.
#include "ua_latent.cuh"

namespace ua {

cudaError_t launch_latent_l128(const LatentParams& p, bool bf16, cudaStream_t s) {
  return launch_latent_any<128>(p, bf16, s);
}

}  // namespace ua
