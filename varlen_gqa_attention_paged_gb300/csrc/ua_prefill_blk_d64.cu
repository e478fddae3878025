// ua_prefill_blk_d64.cu -- instantiations of the tensor-memory prefill kernel for head_dim
// 64 and block-scaled caches.
#include "ua_prefill_tm.cuh"

namespace ua {

cudaError_t launch_prefill_blk_d64(const PrefillParams& pp, dim3 grid, int kv, bool feat, int nq,
                                  cudaStream_t s) {
  return nq == 2 ? launch_prefill_tm_blk<64, 2>(pp, grid, kv, feat, s)
                 : launch_prefill_tm_blk<64, 1>(pp, grid, kv, feat, s);
}

}  // namespace ua
