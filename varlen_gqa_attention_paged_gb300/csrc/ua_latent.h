// ua_latent.h -- launch arguments of the latent-attention kernels of libua.so.
#pragma once

#include "ua_internal.h"

namespace ua {

// The library's own scratch on the current device for work on `stream`: grow-only, one for each
// stream and one for each capture.
int library_workspace(cudaStream_t stream, size_t bytes, void** out);
// A tensor map of f16 or bf16 elements, boxes in the 128-byte swizzle, zeros outside the tensor.
bool encode_half_map(CUtensorMap* map, const void* base, bool bf16, int rank,
                     const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box);

// Rows (query token x head) of one CTA's tile, and keys of one tile.
constexpr int kLatRows = 64;
constexpr int kLatKeys = 64;

// One launch of the absorbed form's kernel.  q is mapped as rows [total_q * heads][L + R] in boxes of
// 64 elements x 64 rows, the cache as rows [num_blocks * block_size][L + R] in boxes of 64 elements x
// box_rows (elements past L + R read as zero); and the latent parts as column blocks of 64 elements,
// in boxes of 64 rows of all of them (q) or of a half (the cache).
struct LatentParams {
  CUtensorMap q_map, q_lat, k_map, k_half;
  void* out;                    // [total_q, heads, L]
  float* lse;                   // [total_q, heads] or null
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;
  const int32_t* block_table;
  const int32_t* tree;          // [total_q][tree_stride] words of bits, or null: causal
  long long tree_stride;
  int tree_words;
  // partial rows of a tile that several workers share: slot 2 * cta (the worker entered the tile
  // at a later key) or 2 * cta + 1 (it began the tile and did not end it), kLatRows rows each
  float* ws_acc;
  float* ws_m;
  float* ws_l;
  int4* ws_meta;                // [ctas] of the tile that a CTA began: first row, rows, parts
  unsigned int* status;
  int num_seqs, total_q, max_blocks_per_seq, num_blocks, block_size, heads, rope_dim, out_dtype;
  int workers;                  // groups of `cl` CTAs that share a tile's keys; or (spread) row tiles
  int cl;                       // CTAs (tiles of kLatRows rows) of a worker: 1 or 2
  int spread;                   // > 0: a cluster of that many CTAs a row tile, a part of its keys each
  int box_rows;                 // cache rows of a box: a power of two that divides the block size
  int min_share;                // key tiles that a worker takes at least
  float scale;
};

// One launch of the expanded form's kernel: maps of q [total_q][heads][N + R], k_nope
// [total_k][heads][N] and v [total_k][heads][V] (boxes of 64 elements x one head x 128 tokens) and
// of k_rope [total_k][R] (64 elements x 128 tokens; elements past R read as zero).
constexpr int kLatentParts = 4;

struct LatentPrefillParams {
  CUtensorMap q, k, k_rope, v;
  void* out;                    // [total_q, heads, V]
  float* lse;                   // [total_q, heads] or null
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  unsigned int* status;
  int num_seqs, total_q, total_k, heads, rope_dim, out_dtype, slots;
  int parts;                    // CTAs (a cluster) that share a q-block's keys: 1 .. kLatentParts
  int by_length;                // 1: q-blocks start by the length of their walks (at most 64 slots)
  float scale;
};

struct LatentMergeParams {
  void* out;
  float* lse;
  const float* ws_acc;
  const float* ws_m;
  const float* ws_l;
  const int4* ws_meta;
  long long rows;               // total_q * heads
  int ctas, cl, out_dtype, grid_rows;
  int few;                      // > 0: row tiles at most, which the grid's x counts
};

cudaError_t launch_latent_l128(const LatentParams& p, bool bf16, cudaStream_t s);
cudaError_t launch_latent_l256(const LatentParams& p, bool bf16, cudaStream_t s);
cudaError_t launch_latent_l512(const LatentParams& p, bool bf16, cudaStream_t s);
cudaError_t launch_latent_prefill_n64(const LatentPrefillParams& p, int value, bool bf16,
                                      cudaStream_t s);
cudaError_t launch_latent_prefill_n128(const LatentPrefillParams& p, int value, bool bf16,
                                       cudaStream_t s);
cudaError_t launch_latent_merge(const LatentMergeParams& p, int latent, cudaStream_t s);

// Scratch of a launch of `ctas` CTAs.
constexpr size_t latent_scratch_bytes(int ctas, int latent) {
  return static_cast<size_t>(ctas) * (2 * kLatRows * (static_cast<size_t>(latent) + 2) * 4 + 16);
}

}  // namespace ua
