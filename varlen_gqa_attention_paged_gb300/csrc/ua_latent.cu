// ua_latent.cu -- latent attention, absorbed form: argument checks and launches, and the merge of
// row tiles that several workers shared.
#include <algorithm>
#include <climits>
#include <cmath>

#include "ua_device.cuh"
#include "ua_latent.h"

#include "ua.h"

namespace ua {

// Four neighbouring elements of the output.
__device__ __forceinline__ void store_four(void* out, size_t at, float4 v, int dtype) {
  if (dtype == UA_DT_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  } else {
    const bool bf = dtype == UA_DT_BF16;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(bf ? pack_bf16(v.x, v.y) : pack_f16(v.x, v.y),
                   bf ? pack_bf16(v.z, v.w) : pack_f16(v.z, v.w));
  }
}

// One output row from its partial rows: with m_k, l_k and acc_k of part k
//   M = max m_k,  L = sum l_k 2^(m_k - M),  out = sum acc_k 2^(m_k - M) / L
// Blocks (x, y) share the rows of the tile that CTA x began: two warps a row, half of its elements
// each, or, with many parts of few rows (152 parts of 2 KB a row), a block a row, an eighth of the parts
// a warp, joined in shared memory.  About 3.5 us of a call of 64 sequences of up to 8191 keys, latency
// of its loads.  Sums run in a fixed order.
constexpr int kMergeMany = 16;
constexpr int kMergeFewBlocks = 1024;

template <int L>
__global__ void __launch_bounds__(256) ua_latent_merge_kernel(
    const __grid_constant__ LatentMergeParams p) {
  constexpr int kVec = L / 4;             // float4s of a row
  constexpr int kPer = (kVec + 31) / 32;  // of a lane, a warp a row
  __shared__ float4 s_acc[8][kVec];
  __shared__ float s_sum[8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 meta = p.ws_meta[cta];
  const int parts = min(meta.z, p.ctas / p.cl - cta / p.cl);
  const int rows = static_cast<int>(
      min(static_cast<long long>(min(meta.y, kLatRows)), p.rows - meta.x));
  if (parts <= 0 || meta.x < 0) return;
  auto at = [&](int k, int r) -> size_t {  // part k of row r
    const int slot = k == 0 ? 2 * cta + 1 : 2 * (cta + k * p.cl);
    return static_cast<size_t>(slot) * kLatRows + r;
  };
  auto store = [&](int r, int v4, float4 v) {
    store_four(p.out, (static_cast<size_t>(meta.x) + r) * L + 4 * v4, v, p.out_dtype);
  };
  // max over the row's parts; the lane's first part with it
  auto top_of = [&](int r, float& m0, float& l0) -> float {
    m0 = lane < parts ? p.ws_m[at(lane, r)] : -INFINITY;
    l0 = lane < parts ? p.ws_l[at(lane, r)] : 0.f;
    float M = m0;
    for (int k = lane + 32; k < parts; k += 32) M = fmaxf(M, p.ws_m[at(k, r)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    return M;
  };
  if (parts <= kMergeMany || rows > kLatRows / 2) {
    constexpr int kHalf = (kPer + 1) / 2;
    const int half = warp & 1;
    for (int r = blockIdx.y * 4 + (warp >> 1); r < rows; r += gridDim.y * 4) {
      float m, l;
      const float M = top_of(r, m, l);
      float sum = 0.f;
      float4 acc[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < parts; k0 += 32) {
        if (k0 > 0) {
          m = k0 + lane < parts ? p.ws_m[at(k0 + lane, r)] : -INFINITY;
          l = k0 + lane < parts ? p.ws_l[at(k0 + lane, r)] : 0.f;
        }
        // (a part that saw no key has no elements either)
        const float f = l == 0.f ? 0.f : fast_exp2(m - M);
        sum += l == 0.f ? 0.f : l * f;
        for (int k = 0; k < min(32, parts - k0); k += 4) {
          float4 v[4][kHalf];
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // (lanes past the parts have l = 0)
            const float le = __shfl_sync(0xffffffffu, l, k + e);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
              const int v4 = (half * kHalf + i) * 32 + lane;
              v[e][i] = le != 0.f && v4 < kVec
                            ? reinterpret_cast<const float4*>(p.ws_acc + at(k0 + k + e, r) * L)[v4]
                            : make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float fe = __shfl_sync(0xffffffffu, f, k + e);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
              acc[i].x += v[e][i].x * fe;
              acc[i].y += v[e][i].y * fe;
              acc[i].z += v[e][i].z * fe;
              acc[i].w += v[e][i].w * fe;
            }
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        const int v4 = (half * kHalf + i) * 32 + lane;
        if (v4 < kVec)
          store(r, v4, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
      }
      if (p.lse != nullptr && lane == 0 && half == 0)
        p.lse[meta.x + r] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
    }
    return;
  }
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float m0, l0;
    const float M = top_of(r, m0, l0);
    float4 acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int k = warp; k < parts; k += 8) {
      const float l = p.ws_l[at(k, r)], f = l == 0.f ? 0.f : fast_exp2(p.ws_m[at(k, r)] - M);
      sum += l == 0.f ? 0.f : l * f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float4 v = l != 0.f && 32 * i + lane < kVec
                             ? reinterpret_cast<const float4*>(p.ws_acc + at(k, r) * L)[32 * i + lane]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        acc[i].x += v.x * f;
        acc[i].y += v.y * f;
        acc[i].z += v.z * f;
        acc[i].w += v.w * f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i + lane < kVec) s_acc[warp][32 * i + lane] = acc[i];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += s_sum[w];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int v4 = threadIdx.x; v4 < kVec; v4 += 256) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float4 v = s_acc[w][v4];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      store(r, v4, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
    }
    if (p.lse != nullptr && threadIdx.x == 0)
      p.lse[meta.x + r] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
    __syncthreads();
  }
}

// The same for few row tiles of many parts (one long sequence): x counts the tiles that have parts, a
// block takes 128 elements of a row, an eighth of the parts a warp, joined in shared memory.  (A kernel
// of its own: in the one above its code cost every other call 0.5 us.)
template <int L>
__global__ void __launch_bounds__(256) ua_latent_merge_few_kernel(
    const __grid_constant__ LatentMergeParams p) {
  constexpr int kPieces = L / 128;
  __shared__ float4 s_acc[8][32];
  __shared__ float s_sum[8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int cta = -1, seen = 0;  // the CTA that began the tile
#pragma unroll 4
  for (int base = 0; base < p.ctas; base += 32) {
    const bool begun = base + lane < p.ctas && p.ws_meta[base + lane].z > 0;
    const unsigned m = __ballot_sync(0xffffffffu, begun);
    const unsigned mine = __ballot_sync(
        0xffffffffu,
        begun && seen + __popc(m & ((1u << lane) - 1u)) == static_cast<int>(blockIdx.x));
    if (mine != 0u) cta = base + __ffs(mine) - 1;
    seen += __popc(m);
  }
  if (cta < 0) return;
  const int4 meta = p.ws_meta[cta];
  const int parts = min(meta.z, p.ctas / p.cl - cta / p.cl);
  const int rows = static_cast<int>(
      min(static_cast<long long>(min(meta.y, kLatRows)), p.rows - meta.x));
  if (parts <= 0 || meta.x < 0) return;
  for (int e = blockIdx.y; e < rows * kPieces; e += gridDim.y) {
    const int r = e / kPieces, v4 = e % kPieces * 32 + lane;
    auto at = [&](int k) -> size_t {  // part k of the row
      const int slot = k == 0 ? 2 * cta + 1 : 2 * (cta + k * p.cl);
      return static_cast<size_t>(slot) * kLatRows + r;
    };
    float M = -INFINITY;
    for (int k = lane; k < parts; k += 32) M = fmaxf(M, p.ws_m[at(k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int k0 = warp; k0 < parts; k0 += 64) {
      float l[8], m[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // eight parts' loads in flight
        const int k = min(k0 + 8 * u, parts - 1);
        l[u] = p.ws_l[at(k)];
        m[u] = p.ws_m[at(k)];
        v[u] = reinterpret_cast<const float4*>(p.ws_acc + at(k) * L)[v4];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        // (a part that saw no key has no elements)
        if (k0 + 8 * u >= parts || l[u] == 0.f) continue;
        const float f = fast_exp2(m[u] - M);
        sum += l[u] * f;
        acc.x += v[u].x * f;
        acc.y += v[u].y * f;
        acc.z += v[u].z * f;
        acc.w += v[u].w * f;
      }
    }
    s_acc[warp][lane] = acc;
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      sum = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float4 v = s_acc[w][lane];
        sum += s_sum[w];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      store_four(p.out, (static_cast<size_t>(meta.x) + r) * L + 4 * v4,
                 make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv), p.out_dtype);
      if (p.lse != nullptr && lane == 0 && e % kPieces == 0)
        p.lse[meta.x + r] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

cudaError_t launch_latent_merge(const LatentMergeParams& p, int latent, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.few ? p.few : p.ctas),
                  static_cast<unsigned>(p.grid_rows));
  const auto kern = latent == 512   ? p.few ? ua_latent_merge_few_kernel<512>
                                            : ua_latent_merge_kernel<512>
                    : latent == 256 ? p.few ? ua_latent_merge_few_kernel<256>
                                            : ua_latent_merge_kernel<256>
                    : p.few         ? ua_latent_merge_few_kernel<128>
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
// the kernel takes its shares from the lengths themselves).  Workers of two CTAs are one choice for the
// batch, made by its longest sequence of new tokens: a sequence of an odd number of row tiles leaves
// the second CTA of a pair without rows on its walk, single tokens among chunks above all (a chunk of
// 64 tokens behind 2,496 and 63 single tokens over 4,000 keys, 16 heads: 114.8 us, where the two as
// calls of their own take 22.2 and 64.2; a chunk of 512: 163.0, 75.3 and 64.5).
constexpr int kMinShare = 2;
// Few row tiles over few keys take a cluster of up to kSpread CTAs each instead (`spread` CTAs; 0: even
// shares), with an even part of the keys a CTA: that saves the merge kernel and the second row tile
// that a share may reach into, but the longest sequence sets the time.  So a part may be longer than a
// share by one tile where there is one sequence, and otherwise longer by three (five, where a worker
// is two CTAs) than half a share, which is what shares come to where lengths are spread from 0 up to
// the longest.  Clusters of eight are placed onto seven eighths of the SMs at most (17 of them took
// 12.4 us where 17 of four took 10.7).  In us, parts against even shares (tiles of each):
//   16 heads:   1 x 700 keys 10.6 : 12.2 (2 : 2), 1 x 1500 13.1 : 13.1 (3 : 2), 1 x 2500 16.2 : 13.4 (5 : 2),
//               28 x 1000 15.6 : 19.2 (4 : 3), 28 x 2500 25.2 : 25.3 (10 : 8), 50 x 300 13.5 : 18.4 (3 : 2),
//               50 x 2500 43.4 : 42.2 (20 : 14), 100 x 300 16.2 : 25.0 (5 : 4)
//   128 heads:  1 x 700 14.1 : 13.6 (2 : 2), 1 x 2500 20.2 : 17.0 (5 : 2), 12 x 300 14.6 : 20.8 (2 : 2),
//               25 x 1000 24.4 : 30.6 (8 : 6)
constexpr int kSpread = 8;
void shape(const ua_latent_t& a, int sms, int* workers, int* cl, int* spread) {
  *cl = static_cast<long long>(a.max_seqlen_q) * a.num_heads > ua::kLatRows ? 2 : 1;
  const long long rows = static_cast<long long>(a.total_q) * a.num_heads;
  const long long tiles = rows / (ua::kLatRows * *cl) + a.num_seqs;
  const long long keys = (std::max<long long>(a.max_seqlen_k, 1) + ua::kLatKeys - 1) / ua::kLatKeys;
  const long long most = std::max(1, sms / *cl);
  *workers = static_cast<int>(
      std::max(1LL, std::min(most, (tiles * keys + kMinShare - 1) / kMinShare)));
  *spread = 0;
  const long long slots = rows / ua::kLatRows + a.num_seqs;  // row tiles at most
  int parts = 1;
  while (parts < kSpread && parts < keys && slots * 2 * parts <= (parts < 4 ? sms : sms * 7 / 8))
    parts *= 2;
  const long long share = std::max<long long>(kMinShare, (tiles * keys + most - 1) / most);
  const long long longest = a.num_seqs > 1 ? share / 2 + 1 + 2 * *cl : share + 1;
  if (slots * parts > sms || (keys + parts - 1) / parts > longest) return;
  *spread = parts;
  *workers = static_cast<int>(slots);
  *cl = 1;
}

// Rows [width] in boxes of 64 elements x `box_rows`.
bool row_map(CUtensorMap* map, const void* base, bool bf16, long long rows, int width,
             int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  return ua::encode_half_map(map, base, bf16, 2, dims, strides, box);
}

// The rows' latent parts as [blocks][rows][64]: boxes of 64 rows x `box_blocks`.
bool block_map(CUtensorMap* map, const void* base, bool bf16, long long rows, int width, int latent,
               int box_blocks) {
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(latent) / 64};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width) * 2, 128};
  const cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(box_blocks)};
  return ua::encode_half_map(map, base, bf16, 3, dims, strides, box);
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
  shape(a, sms, &p.workers, &p.cl, &p.spread);
  const int ctas = p.spread > 0 ? 0 : p.workers * p.cl;  // that need scratch
  void* ws = a.workspace;
  if (ctas > 0) {
    const size_t need = ua::latent_scratch_bytes(ctas, a.latent_dim);
    if (ws != nullptr) {
      if (a.workspace_bytes < need || !aligned(ws, 16)) return UA_ERR_WORKSPACE;
    } else if ((rc = ua::library_workspace(st, need, &ws)) != UA_OK) {
      return rc;
    }
  }
  const bool bf16 = a.dtype == UA_DT_BF16;
  p.box_rows = std::min(ua::kLatKeys, a.block_size & -a.block_size);
  const int width = a.latent_dim + a.rope_dim;
  const long long q_rows = static_cast<long long>(a.total_q) * a.num_heads;
  const long long k_rows = static_cast<long long>(a.num_blocks) * a.block_size;
  const int half = a.latent_dim / (a.latent_dim > 128 ? 128 : 64);  // column blocks of a half
  if (!row_map(&p.q_map, a.q, bf16, q_rows, width, ua::kLatRows) ||
      !block_map(&p.q_lat, a.q, bf16, q_rows, width, a.latent_dim, a.latent_dim / 64) ||
      !row_map(&p.k_map, a.cache, bf16, k_rows, width, p.box_rows) ||
      !block_map(&p.k_half, a.cache, bf16, k_rows, width, a.latent_dim, half))
    return UA_ERR_CUDA;
  p.out = a.out;
  p.lse = a.lse;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens_k = a.seq_lens_k;
  p.block_table = a.block_table;
  p.tree = a.tree_mask;
  p.tree_stride = a.tree_mask_stride;
  p.tree_words = a.tree_words;
  if (ctas > 0) {
    const size_t slots = static_cast<size_t>(ctas) * 2 * ua::kLatRows;
    p.ws_acc = static_cast<float*>(ws);
    p.ws_meta = reinterpret_cast<int4*>(p.ws_acc + slots * a.latent_dim);
    p.ws_m = reinterpret_cast<float*>(p.ws_meta + ctas);
    p.ws_l = p.ws_m + slots;
  }
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
  if (p.workers == 1 || p.spread > 0) return UA_OK;  // no tile is shared through scratch
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
  const long long rows = std::max(
      1LL, std::min<long long>(ua::kLatRows, static_cast<long long>(a.max_seqlen_q) * a.num_heads));
  // (pairs of) row tiles at most; few of them, of many parts: in us, against the other kernel: 16 heads,
  // one sequence of 2500 keys 12.9 : 13.5, 16000 17.3 : 21.6, 128000 44.2 : 47.1, 4 of 8000 (30 parts)
  // 21.0 : 22.2, 12 of 8000 (10 parts) 36.4 : 33.7; 128 heads, one of 16000 23.4 : 29.4, 4 of 5000
  // (4096 blocks) 39.4 : 28.2
  const long long begun = m.rows / (ua::kLatRows * p.cl) + a.num_seqs;
  const long long pieces = rows * (a.latent_dim / 128);
  if (begun * ua::kMergeMany <= p.workers && p.cl * begun * pieces <= ua::kMergeFewBlocks)
    m.few = static_cast<int>(p.cl * begun);
  // blocks of a tile: one for each 128 elements; or one for each row, sixteen at most (they walk the
  // others)
  m.grid_rows = static_cast<int>(m.few ? pieces : std::min(16LL, rows));
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
  int sms = 0, workers = 0, cl = 0, spread = 0;
  if (call == nullptr || check(*call) != UA_OK || ua::device_sm_count(&sms) != UA_OK) return 0;
  shape(*call, sms, &workers, &cl, &spread);
  return spread > 0 ? 0 : ua::latent_scratch_bytes(workers * cl, call->latent_dim);
}
