// ua_prefill_blk_d256.cu -- instantiations of the tensor-memory prefill kernel for head_dim
// 256 and block-scaled caches.
#include "ua_prefill_wide.cuh"

namespace ua {

cudaError_t launch_prefill_blk_d256(const PrefillParams& pp, dim3 grid, int kv, bool feat, int nq,
                                    cudaStream_t s) {
  if (nq != 1) return cudaErrorInvalidValue;
  if (kv == KV_E4M3B)
    return feat ? launch_prefill_wide_t<256, false, true, true, 1>(pp, grid, s)
                : launch_prefill_wide_t<256, false, false, true, 1>(pp, grid, s);
  if (kv == KV_I8B)
    return feat ? launch_prefill_wide_t<256, false, true, true, 2>(pp, grid, s)
                : launch_prefill_wide_t<256, false, false, true, 2>(pp, grid, s);
  return cudaErrorInvalidValue;
}

}  // namespace ua
