// ua_prefill_blk_d256.cu -- instantiations of the tensor-memory prefill kernel for head_dim
// 256 and block-scaled caches.
#include "ua_prefill_wide.cuh"

namespace ua {

// With score features two softmax warps share a lane quarter: softcap, 24/4 heads, two chunks of
// 4096 behind 4096 (e4m3) 1384 us against 1598 with one, three ragged ones of up to 1501 (int8)
// 250 against 302.  Without them one does, in one pass; the halves' exchange of row maxima cost
// 3 % there (1.32 against 1.36 ms, both in two passes).
cudaError_t launch_prefill_blk_d256(const PrefillParams& pp, dim3 grid, int kv, bool feat, int nq,
                                    cudaStream_t s) {
  if (nq != 1) return cudaErrorInvalidValue;
  if (kv == KV_E4M3B)
    return feat ? launch_prefill_wide_t<256, false, true, true, 1, 2>(pp, grid, s)
                : launch_prefill_wide_t<256, false, false, true, 1, 1>(pp, grid, s);
  if (kv == KV_I8B)
    return feat ? launch_prefill_wide_t<256, false, true, true, 2, 2>(pp, grid, s)
                : launch_prefill_wide_t<256, false, false, true, 2, 1>(pp, grid, s);
  return cudaErrorInvalidValue;
}

}  // namespace ua
