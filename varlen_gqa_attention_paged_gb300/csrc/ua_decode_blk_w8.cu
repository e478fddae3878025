// ua_decode_blk_w8.cu -- instantiations of the key-major decode tile kernel for block-scaled
// caches, eight consumer warps.
#include "ua_decode.cuh"

namespace ua {

cudaError_t launch_decode_blk_w8_d64(const TileParams& tp, dim3 grid, int kv, bool feat,
                                       int cluster_y, int cluster_z, cudaStream_t s) {
  return launch_decode_blk<64, 8, 1>(tp, grid, kv, feat, cluster_y, cluster_z, s);
}

cudaError_t launch_decode_blk_w8_d128(const TileParams& tp, dim3 grid, int kv, bool feat,
                                       int cluster_y, int cluster_z, cudaStream_t s) {
  return launch_decode_blk<128, 8, 1>(tp, grid, kv, feat, cluster_y, cluster_z, s);
}

cudaError_t launch_decode_blk_w8_d256(const TileParams& tp, dim3 grid, int kv, bool feat,
                                        int cluster_y, int cluster_z, cudaStream_t s) {
  return launch_decode_blk<256, 8, 1>(tp, grid, kv, feat, cluster_y, cluster_z, s);
}

int decode_cluster_capacity_blk_w8(int head_dim, int kv, int cluster_y, int cluster_z) {
  if (kv == KV_I8B)
    return head_dim == 64    ? decode_cluster_capacity_t<64, KV_I8B, 8, 1>(cluster_y, cluster_z)
           : head_dim == 128 ? decode_cluster_capacity_t<128, KV_I8B, 8, 1>(cluster_y, cluster_z)
                             : decode_cluster_capacity_t<256, KV_I8B, 8, 1>(cluster_y, cluster_z);
  return head_dim == 64    ? decode_cluster_capacity_t<64, KV_E4M3B, 8, 1>(cluster_y, cluster_z)
         : head_dim == 128 ? decode_cluster_capacity_t<128, KV_E4M3B, 8, 1>(cluster_y, cluster_z)
                           : decode_cluster_capacity_t<256, KV_E4M3B, 8, 1>(cluster_y, cluster_z);
}

}  // namespace ua
