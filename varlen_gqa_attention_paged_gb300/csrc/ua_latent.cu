// ua_latent.cu -- latent attention, absorbed form: argument checks and launches, the merge of
// row tiles that several workers shared, and the masks of drafted trees.
#include <algorithm>
#include <climits>
#include <cmath>

#include "ua_device.cuh"
#include "ua_latent.h"

#include "ua.h"

namespace ua {

// One warp a partial row: with m_k, l_k and acc_k of part k
//   M = max m_k,  L = sum l_k 2^(m_k - M),  out = sum acc_k 2^(m_k - M) / L
// in the order of the parts.  Block (x, y) takes rows y, y + 8, .. (a warp each 8) of the tile that
// CTA x began.
template <int L>
__global__ void __launch_bounds__(256) ua_latent_merge_kernel(
    const __grid_constant__ LatentMergeParams p) {
  constexpr int kPer = L / 128;  // float4s of a lane
  grid_dependency_wait();
  grid_launch_dependents();
  const int cta = blockIdx.x;
  const int4 meta = p.ws_meta[cta];
  const int parts = min(meta.z, p.ctas / p.cl - cta / p.cl);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= min(meta.y, kLatRows) || parts <= 0) return;
  const long long row = static_cast<long long>(meta.x) + r;
  if (row < 0 || row >= p.rows) return;
  auto at = [&](int k) -> size_t {  // part k's row
    const int slot = k == 0 ? 2 * cta + 1 : 2 * (cta + k * p.cl);
    return static_cast<size_t>(slot) * kLatRows + r;
  };
  float M = -INFINITY;
  for (int k = lane; k < parts; k += 32) M = fmaxf(M, p.ws_m[at(k)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const int k = k0 + lane;
    const float l = k < parts ? p.ws_l[at(k)] : 0.f;
    // (a part that saw no key has no elements either)
    const float f = l == 0.f ? 0.f : fast_exp2(p.ws_m[at(k)] - M);
    sum += l == 0.f ? 0.f : l * f;
    const int n = min(32, parts - k0);
#pragma unroll 4
    for (int e = 0; e < n; ++e) {
      const float fe = __shfl_sync(0xffffffffu, f, e);
      const float le = __shfl_sync(0xffffffffu, l, e);
      if (le == 0.f) continue;
      const float4* a = reinterpret_cast<const float4*>(p.ws_acc + at(k0 + e) * L) + lane;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float4 v = a[32 * i];
        acc[i].x += v.x * fe;
        acc[i].y += v.y * fe;
        acc[i].z += v.z * fe;
        acc[i].w += v.w * fe;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float4 v = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    const size_t e = static_cast<size_t>(row) * L + 4 * (lane + 32 * i);
    if (p.out_dtype == UA_DT_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + e) = v;
    } else {
      const bool bf = p.out_dtype == UA_DT_BF16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + e) =
          make_uint2(bf ? pack_bf16(v.x, v.y) : pack_f16(v.x, v.y),
                     bf ? pack_bf16(v.z, v.w) : pack_f16(v.z, v.w));
    }
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

cudaError_t launch_latent_merge(const LatentMergeParams& p, int latent, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.ctas), kLatRows / 8);
  const auto kern = latent == 512   ? ua_latent_merge_kernel<512>
                    : latent == 256 ? ua_latent_merge_kernel<256>
                                    : ua_latent_merge_kernel<128>;
  return launch_pdl(kern, grid, dim3(256), 0, s, 1, p);
}

}  // namespace ua

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check(const ua_latent_t& a) {
  if (a.num_seqs < 0 || a.total_q < 0 || a.max_seqlen_q < 0 || a.max_seqlen_k < 0 ||
      a.max_blocks_per_seq < 0 || a.num_blocks < 0 || a.block_size < 1 || a.num_heads < 1)
    return UA_ERR_INVALID_ARG;
  if (a.latent_dim != 128 && a.latent_dim != 256 && a.latent_dim != 512) return UA_ERR_INVALID_ARG;
  if (a.rope_dim < 16 || a.rope_dim > 64 || a.rope_dim % 16 != 0) return UA_ERR_INVALID_ARG;
  if (a.dtype != UA_DT_F16 && a.dtype != UA_DT_BF16) return UA_ERR_INVALID_ARG;
  if (a.out_dtype != UA_DT_F16 && a.out_dtype != UA_DT_BF16 && a.out_dtype != UA_DT_F32)
    return UA_ERR_INVALID_ARG;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return UA_ERR_INVALID_ARG;
  if (a.tree_mask != nullptr &&
      (a.tree_words < 1 || a.tree_mask_stride < 0 || !aligned(a.tree_mask, 4) ||
       static_cast<long long>(a.tree_words) * 32 < a.max_seqlen_q))
    return UA_ERR_INVALID_ARG;
  // row numbers of q and of the cache are 32-bit coordinates of the copies
  if (static_cast<long long>(a.total_q) * a.num_heads > INT_MAX - 2 * ua::kLatRows * 2 ||
      static_cast<long long>(a.num_blocks) * a.block_size > INT_MAX - 64)
    return UA_ERR_UNSUPPORTED;
  return UA_OK;
}

// CTAs of a worker and workers of a call on `sms` SMs, from the host's sizes (a bound of the work:
// the kernel takes its shares from the lengths themselves).
constexpr int kMinShare = 4;
void shape(const ua_latent_t& a, int sms, int* workers, int* cl) {
  *cl = static_cast<long long>(a.max_seqlen_q) * a.num_heads > ua::kLatRows ? 2 : 1;
  const long long tiles =
      static_cast<long long>(a.total_q) * a.num_heads / (ua::kLatRows * *cl) + a.num_seqs;
  const long long keys = std::max(1, (a.max_seqlen_k + ua::kLatKeys - 1) / ua::kLatKeys);
  const long long most = std::max(1, sms / *cl);
  *workers = static_cast<int>(
      std::max(1LL, std::min(most, (tiles * keys + kMinShare - 1) / kMinShare)));
}

// Rows [width] in boxes of 64 elements x `box_rows`.
bool row_map(CUtensorMap* map, const void* base, bool bf16, long long rows, int width,
             int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  return ua::encode_half_map(map, base, bf16, 2, dims, strides, box);
}

int attend(const ua_latent_t& a, cudaStream_t st) {
  int rc = check(a);
  if (rc != UA_OK) return rc;
  if (a.total_q == 0 || a.num_seqs == 0) return UA_OK;
  if (!a.q || !a.cache || !a.out || !a.cu_seqlens_q || !a.seq_lens_k || !a.block_table)
    return UA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.cache, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4))
    return UA_ERR_INVALID_ARG;
  if (a.max_blocks_per_seq < 1 || a.num_blocks < 1) return UA_ERR_INVALID_ARG;

  int sms = 0;
  if ((rc = ua::device_sm_count(&sms)) != UA_OK) return rc;
  ua::LatentParams p{};
  shape(a, sms, &p.workers, &p.cl);
  const int ctas = p.workers * p.cl;
  const size_t need = ua::latent_scratch_bytes(ctas, a.latent_dim);
  void* ws = a.workspace;
  if (ws != nullptr) {
    if (a.workspace_bytes < need || !aligned(ws, 16)) return UA_ERR_WORKSPACE;
  } else if ((rc = ua::library_workspace(st, need, &ws)) != UA_OK) {
    return rc;
  }
  const bool bf16 = a.dtype == UA_DT_BF16;
  p.box_rows = std::min(ua::kLatKeys, a.block_size & -a.block_size);
  const int width = a.latent_dim + a.rope_dim;
  if (!row_map(&p.q_map, a.q, bf16, static_cast<long long>(a.total_q) * a.num_heads, width,
               ua::kLatRows) ||
      !row_map(&p.k_map, a.cache, bf16, static_cast<long long>(a.num_blocks) * a.block_size, width,
               p.box_rows))
    return UA_ERR_CUDA;
  p.out = a.out;
  p.lse = a.lse;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens_k = a.seq_lens_k;
  p.block_table = a.block_table;
  p.tree = a.tree_mask;
  p.tree_stride = a.tree_mask_stride;
  p.tree_words = a.tree_words;
  const size_t slots = static_cast<size_t>(ctas) * 2 * ua::kLatRows;
  p.ws_acc = static_cast<float*>(ws);
  p.ws_meta = reinterpret_cast<int4*>(p.ws_acc + slots * a.latent_dim);
  p.ws_m = reinterpret_cast<float*>(p.ws_meta + ctas);
  p.ws_l = p.ws_m + slots;
  if ((rc = ua::status_word(&p.status)) != UA_OK) return rc;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.num_blocks;
  p.block_size = a.block_size;
  p.heads = a.num_heads;
  p.rope_dim = a.rope_dim;
  p.out_dtype = a.out_dtype;
  p.min_share = kMinShare;
  p.scale = a.scale;
  const auto launch = a.latent_dim == 512   ? ua::launch_latent_l512
                      : a.latent_dim == 256 ? ua::launch_latent_l256
                                            : ua::launch_latent_l128;
  if (launch(p, bf16, st) != cudaSuccess) return UA_ERR_CUDA;
  if (p.workers == 1) return UA_OK;  // no tile is shared
  ua::LatentMergeParams m{};
  m.out = a.out;
  m.lse = a.lse;
  m.ws_acc = p.ws_acc;
  m.ws_m = p.ws_m;
  m.ws_l = p.ws_l;
  m.ws_meta = p.ws_meta;
  m.rows = static_cast<long long>(a.total_q) * a.num_heads;
  m.ctas = ctas;
  m.cl = p.cl;
  m.out_dtype = a.out_dtype;
  return ua::launch_latent_merge(m, a.latent_dim, st) == cudaSuccess ? UA_OK : UA_ERR_CUDA;
}

}  // namespace

extern "C" int ua_latent_attention(const ua_latent_t* call, void* stream) {
  try {
    if (call == nullptr) return UA_ERR_INVALID_ARG;
    return attend(*call, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return UA_ERR_CUDA;
  }
}

extern "C" size_t ua_latent_workspace_bytes(const ua_latent_t* call) {
  int sms = 0, workers = 0, cl = 0;
  if (call == nullptr || check(*call) != UA_OK || ua::device_sm_count(&sms) != UA_OK) return 0;
  shape(*call, sms, &workers, &cl);
  return ua::latent_scratch_bytes(workers * cl, call->latent_dim);
}
