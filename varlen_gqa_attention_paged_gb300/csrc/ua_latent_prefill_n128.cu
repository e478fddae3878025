// ua_latent_prefill_n128.cu -- instantiations of the expanded latent-attention kernel for keys of 128
// elements beside the rope part.
#include "ua_latent_prefill.cuh"

namespace ua {

cudaError_t launch_latent_prefill_n128(const LatentPrefillParams& p, int value, bool bf16,
                                     cudaStream_t s) {
  if (value == 64)
    return bf16 ? launch_latent_prefill_t<128, 64, true>(p, s)
                : launch_latent_prefill_t<128, 64, false>(p, s);
  return bf16 ? launch_latent_prefill_t<128, 128, true>(p, s)
              : launch_latent_prefill_t<128, 128, false>(p, s);
}

}  // namespace ua
