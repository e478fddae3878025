// ua_latent_prefill.cu -- ua_latent_prefill: argument checks and the launch.
#include <algorithm>
#include <climits>
#include <cmath>

#include "ua_latent.h"

#include "ua.h"

namespace {

constexpr int kBlockTokens = 256;  // query tokens of a CTA

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides that a copy's tensor map takes: multiples of 16 bytes below 2^40, not zero (a dim of one
// element may have any: it is replaced).
bool stride(int64_t s, int64_t n) { return n <= 1 || (s > 0 && s % 8 == 0 && s < (1ll << 38)); }

// [tokens][heads][width] rows of `width` elements.
bool head_map(CUtensorMap* map, const void* base, bool bf16, int tokens, int heads, int width,
              const int64_t* st) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t any = static_cast<cuuint64_t>(width) * 2;
  const cuuint64_t strides[2] = {heads > 1 ? static_cast<cuuint64_t>(st[1]) * 2 : any,
                                 tokens > 1 ? static_cast<cuuint64_t>(st[0]) * 2 : any};
  const cuuint32_t box[3] = {64, 1, 128};
  return ua::encode_half_map(map, base, bf16, 3, dims, strides, box);
}

// CTAs (a cluster) that share a q-block's keys: 2 or 4, if all q-blocks still start at once and the
// longest walk becomes shorter by four key tiles of 128 or more, which is what joining the parts
// costs.  In us, 4 | 2 | 1 CTAs a q-block of 256 tokens, 16 heads unless said: 64 tokens behind 3,936
// 19.1 | 31.4 | 54.4; 256 behind 7,744 37.7 | 66.8 | 115.3; 1,000 of 8 heads 13.7 | 18.1 | 20.4; 1,000
// (256 CTAs if of four) 25.0 | 18.3 | 20.6; 600 (5 key tiles) - | 15.1 | 13.4; 2,000 (256 CTAs if of
// two) - | 37.4 | 34.3.  Parts of eight were slower than of four wherever they fitted.
int parts(const ua_latent_prefill_t& a, long long slots, int sms) {
  const long long blocks =
      std::min(slots, static_cast<long long>(a.num_seqs) *
                          ((static_cast<long long>(a.max_seqlen_q) + kBlockTokens - 1) / kBlockTokens)) *
      a.num_heads;
  const int tiles = static_cast<int>((static_cast<long long>(a.max_seqlen_k) + 127) / 128);
  for (int n = ua::kLatentParts; n > 1; n /= 2)
    if (blocks * n <= (n > 2 ? sms * 7 / 8 : sms) && tiles - (tiles + n - 1) / n >= 4) return n;
  return 1;
}

int prefill(const ua_latent_prefill_t& a, cudaStream_t st) {
  if (a.num_seqs < 0 || a.total_q < 0 || a.total_k < 0 || a.max_seqlen_q < 0 || a.max_seqlen_k < 0 ||
      a.num_heads < 1)
    return UA_ERR_INVALID_ARG;
  if ((a.nope_dim != 64 && a.nope_dim != 128) || (a.value_dim != 64 && a.value_dim != 128) ||
      a.rope_dim < 16 || a.rope_dim > 64 || a.rope_dim % 16 != 0)
    return UA_ERR_INVALID_ARG;
  if (a.dtype != UA_DT_F16 && a.dtype != UA_DT_BF16) return UA_ERR_INVALID_ARG;
  if (a.out_dtype != UA_DT_F16 && a.out_dtype != UA_DT_BF16 && a.out_dtype != UA_DT_F32)
    return UA_ERR_INVALID_ARG;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return UA_ERR_INVALID_ARG;
  if (a.total_q == 0 || a.num_seqs == 0) return UA_OK;
  if (!a.q || !a.out || !a.cu_seqlens_q || !a.cu_seqlens_k ||
      (a.total_k > 0 && (!a.k_nope || !a.k_rope || !a.v)))
    return UA_ERR_INVALID_ARG;
  for (const void* x : {a.q, a.k_nope, a.k_rope, a.v, static_cast<const void*>(a.out)})
    if (!aligned(x, 16)) return UA_ERR_INVALID_ARG;
  if (!aligned(a.lse, 4)) return UA_ERR_INVALID_ARG;
  if (!stride(a.q_stride[0], a.total_q) || !stride(a.q_stride[1], a.num_heads) ||
      !stride(a.k_nope_stride[0], a.total_k) || !stride(a.k_nope_stride[1], a.num_heads) ||
      !stride(a.v_stride[0], a.total_k) || !stride(a.v_stride[1], a.num_heads) ||
      !stride(a.k_rope_stride, a.total_k))
    return UA_ERR_INVALID_ARG;
  const long long slots = static_cast<long long>(a.total_q) / kBlockTokens + a.num_seqs;
  if (slots > 65535) return UA_ERR_UNSUPPORTED;  // (of a grid's second dimension)

  const bool bf16 = a.dtype == UA_DT_BF16;
  ua::LatentPrefillParams p{};
  // (without keys the maps are not used: they describe q)
  const bool keys = a.total_k > 0;
  const int tk = keys ? a.total_k : a.total_q;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.rope_dim), static_cast<cuuint64_t>(tk)};
  const cuuint64_t strides[1] = {
      static_cast<cuuint64_t>(keys && tk > 1 ? a.k_rope_stride : a.rope_dim) * 2};
  const cuuint32_t box[2] = {64, 128};
  if (!head_map(&p.q, a.q, bf16, a.total_q, a.num_heads, a.nope_dim + a.rope_dim, a.q_stride) ||
      !head_map(&p.k, keys ? a.k_nope : a.q, bf16, tk, a.num_heads, a.nope_dim,
                keys ? a.k_nope_stride : a.q_stride) ||
      !ua::encode_half_map(&p.k_rope, keys ? a.k_rope : a.q, bf16, 2, dims, strides, box) ||
      !head_map(&p.v, keys ? a.v : a.q, bf16, tk, a.num_heads, a.value_dim,
                keys ? a.v_stride : a.q_stride))
    return UA_ERR_CUDA;
  p.out = a.out;
  p.lse = a.lse;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.cu_seqlens_k = a.cu_seqlens_k;
  int rc, sms = 0;
  if ((rc = ua::status_word(&p.status)) != UA_OK) return rc;
  if ((rc = ua::device_sm_count(&sms)) != UA_OK) return rc;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.heads = a.num_heads;
  p.rope_dim = a.rope_dim;
  p.out_dtype = a.out_dtype;
  p.slots = static_cast<int>(slots);
  p.scale = a.scale;
  p.parts = parts(a, slots, sms);
  // (where all start at once, or all are short, the order is nothing: it costs 500 cycles.  A lane ranks
  // two slots; past 64 they start in reverse order of the batch: 118 slots of 4 heads, prompts of 3,000
  // and 2,000 tokens and 70 of 100, take 52.6 us with the long ones last in it and 64.7 with them first)
  p.by_length = slots <= 64 && slots * a.num_heads > sms && a.max_seqlen_k > 2 * kBlockTokens;
  const auto launch =
      a.nope_dim == 64 ? ua::launch_latent_prefill_n64 : ua::launch_latent_prefill_n128;
  return launch(p, a.value_dim, bf16, st) == cudaSuccess ? UA_OK : UA_ERR_CUDA;
}

}  // namespace

extern "C" int ua_latent_prefill(const ua_latent_prefill_t* call, void* stream) {
  try {
    if (call == nullptr) return UA_ERR_INVALID_ARG;
    return prefill(*call, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return UA_ERR_CUDA;
  }
}
