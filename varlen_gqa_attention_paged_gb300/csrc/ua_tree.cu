// ua_tree.cu -- ua_tree_mask: masks and positions of drafted trees from their parents.
//
// A new token sees itself and what its parent sees:
//   mask_i = bit i | mask_parent(i),   depth_i = depth_parent(i) + 1,   position = context + depth.
// One thread a token and word of its mask walks up the parents, which a block keeps in shared
// memory; parents lie before their children, so a walk ends after at most i steps.  A batch of 8
// trees of 60 tokens is bound by the launch and one walk's chain (4.7 us alone and cold; 1.2 us of a
// step with its attention), one deep tree of 1000 tokens by the walks (37 us; a thread a token that
// writes all its words in one walk took 43, its stores diverging).
#include <climits>

#include "ua_device.cuh"
#include "ua_internal.h"

#include "ua.h"

namespace {

constexpr int kMaxTree = 4096;  // new tokens of a sequence

struct TreeParams {
  const int32_t* parents;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;
  int32_t* mask;
  int32_t* positions;
  long long mask_stride;
  unsigned int* status;
  int total_q, words, max_q;
};

__global__ void __launch_bounds__(256) ua_tree_mask_kernel(const TreeParams p) {
  extern __shared__ int32_t up[];
  ua::grid_dependency_wait();
  ua::grid_launch_dependents();
  const int b = blockIdx.x;
  const int q0 = __ldg(p.cu_seqlens_q + b), q1 = __ldg(p.cu_seqlens_q + b + 1);
  const int kv = __ldg(p.seq_lens_k + b);
  if (q0 < 0) return;
  const int all = min(q1, p.total_q) - q0;
  const int n = min(all, p.max_q);
  bool bad = all > n;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int v = __ldg(p.parents + q0 + i);
    if (v < -1 || v >= i) {
      v = -1;
      bad = true;
    }
    up[i] = v;
  }
  if (bad && blockIdx.y == 0) atomicOr(p.status, ua::DEV_BAD_SHAPE);
  __syncthreads();
  const long long tasks = static_cast<long long>(max(n, 0)) * p.words;
  for (long long e = blockIdx.y * blockDim.x + threadIdx.x; e < tasks;
       e += static_cast<long long>(gridDim.y) * blockDim.x) {
    const int i = static_cast<int>(e / p.words), w = static_cast<int>(e % p.words);
    uint32_t bits = 0;
    int depth = -1;
    for (int a = i; a >= 0; a = up[a]) {
      if ((a >> 5) == w) bits |= 1u << (a & 31);
      ++depth;
    }
    if (p.mask != nullptr) p.mask[(q0 + i) * p.mask_stride + w] = static_cast<int32_t>(bits);
    if (p.positions != nullptr && w == 0) p.positions[q0 + i] = kv - (q1 - q0) + depth;
  }
}

int tree(const ua_tree_t& a, cudaStream_t st) {
  if (a.num_seqs < 0 || a.total_q < 0 || a.max_seqlen_q < 0 || a.max_seqlen_q > kMaxTree ||
      a.mask_words < 1 || static_cast<long long>(a.mask_words) * 32 < a.max_seqlen_q ||
      a.mask_stride < a.mask_words)
    return UA_ERR_INVALID_ARG;
  if (a.total_q == 0 || a.num_seqs == 0) return UA_OK;
  if (!a.parents || !a.cu_seqlens_q || !a.seq_lens_k || (!a.mask && !a.positions))
    return UA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(a.parents), static_cast<const void*>(a.mask),
                        static_cast<const void*>(a.positions)})
    if ((reinterpret_cast<uintptr_t>(x) & 3) != 0) return UA_ERR_INVALID_ARG;
  TreeParams p{a.parents, a.cu_seqlens_q, a.seq_lens_k, a.mask, a.positions, a.mask_stride,
               nullptr,   a.total_q,      a.mask_words, a.max_seqlen_q};
  const int rc = ua::status_word(&p.status);
  if (rc != UA_OK) return rc;
  const long long tasks = static_cast<long long>(a.max_seqlen_q) * a.mask_words;
  const unsigned y = static_cast<unsigned>(tasks <= 256 ? 1 : tasks >= 16 * 256 ? 16 : (tasks + 255) / 256);
  const cudaError_t err =
      ua::launch_pdl(ua_tree_mask_kernel, dim3(static_cast<unsigned>(a.num_seqs), y), dim3(256),
                     static_cast<size_t>(a.max_seqlen_q) * 4, st, 1, p);
  return err == cudaSuccess ? UA_OK : UA_ERR_CUDA;
}

}  // namespace

extern "C" int ua_tree_mask(const ua_tree_t* call, void* stream) {
  try {
    if (call == nullptr) return UA_ERR_INVALID_ARG;
    return tree(*call, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return UA_ERR_CUDA;
  }
}
