// ua_decode_blk_pair.cu -- instantiations of the key-major decode tile kernel for block-scaled
// caches, two kv-heads a CTA.
#include "ua_decode.cuh"

namespace ua {

cudaError_t launch_decode_blk_pair_d64(const TileParams& tp, dim3 grid, int kv, bool feat,
                                       int cluster_y, int cluster_z, cudaStream_t s) {
  return launch_decode_blk<64, 4, 2>(tp, grid, kv, feat, cluster_y, cluster_z, s);
}

cudaError_t launch_decode_blk_pair_d128(const TileParams& tp, dim3 grid, int kv, bool feat,
                                       int cluster_y, int cluster_z, cudaStream_t s) {
  return launch_decode_blk<128, 4, 2>(tp, grid, kv, feat, cluster_y, cluster_z, s);
}

int decode_cluster_capacity_blk_pair(int head_dim, int kv, int cluster_y, int cluster_z) {
  if (kv == KV_I8B)
    return head_dim == 64 ? decode_cluster_capacity_t<64, KV_I8B, 4, 2>(cluster_y, cluster_z)
                          : decode_cluster_capacity_t<128, KV_I8B, 4, 2>(cluster_y, cluster_z);
  return head_dim == 64 ? decode_cluster_capacity_t<64, KV_E4M3B, 4, 2>(cluster_y, cluster_z)
                        : decode_cluster_capacity_t<128, KV_E4M3B, 4, 2>(cluster_y, cluster_z);
}

}  // namespace ua
