// ua_latent_prefill_n64.cu -- instantiations of the expanded latent-attention kernel for keys of 64
// elements beside the rope part.
#include "ua_latent_prefill.cuh"

namespace ua {

cudaError_t launch_latent_prefill_n64(const LatentPrefillParams& p, int value, bool bf16,
                                     cudaStream_t s) {
  return value == 64 ? launch_latent_prefill_any<64, 64>(p, bf16, s)
                     : launch_latent_prefill_any<64, 128>(p, bf16, s);
}

}  // namespace ua
