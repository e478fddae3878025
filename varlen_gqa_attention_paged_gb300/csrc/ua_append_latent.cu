// ua_append_latent.cu -- ua_append_latent: new tokens' latents, normalised, and rope keys, rotated,
// into a paged latent cache; the queries' rope parts rotated beside them.
//
//   c_j = x_j (mean(x^2) + eps)^(-1/2) w_j,    a' = a cos - b sin,   b' = b cos + a sin
//
// Moves each byte once and computes little: bound by HBM for many tokens, by the chain of
// dependent loads (sequence search, block table, rotation table) for few.  A warp takes a token's
// latent and rope key, or some of its query heads: rope_dim / 16 lanes a head, each with both
// 16-byte chunks of its eight pairs, 32 / (rope_dim / 16) heads a pass.
//
// Measured (one GB300): 4 prompts of 2048 tokens, L 512, R 64, 64 query heads, bf16: 29.4 us for 153
// MB, 5.2 TB/s (0.77 of a copy; six blocks of four warps an SM, of 80 registers; seven 29.2, eight,
// which spill, 35.4); one token of each of 32 sequences 2.4 us in a captured graph.
#include <algorithm>
#include <climits>

#include "ua_append.cuh"

namespace {

struct AppendLatentParams {
  const uint16_t* latent;
  const uint16_t* k_rope;
  const uint16_t* q_rope;
  uint16_t* q_rope_out;
  uint16_t* cache;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;
  const int32_t* block_table;
  const void* weight;
  const float* cos_sin;
  const int32_t* positions;
  long long latent_stride, k_rope_stride, q_stride[2], q_out_stride[2];
  unsigned int* status;
  int num_seqs, total_q, max_blocks_per_seq, num_blocks, block_size, heads, rope_dim;
  int max_position, interleaved, weight_f32;
  int lanes, heads_per_pass;      // lanes of a head's rope part, heads of a pass
  int pass_group, warps_per_token;  // passes of a query warp, warps of a token
  float eps;
};

constexpr int kWarps = 4, kBlocks = 6;  // warps of a block, blocks of an SM

template <int L, bool BF>
__global__ void __launch_bounds__(32 * kWarps, kBlocks)
    ua_append_latent_kernel(const __grid_constant__ AppendLatentParams p) {
  constexpr int kPer = (L + 255) / 256;  // 16-byte chunks of the latent that a lane takes
  constexpr int U = 4;                   // passes whose loads are in flight together
  ua::grid_dependency_wait();
  ua::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long task = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(task / p.warps_per_token);
  const int part = static_cast<int>(task % p.warps_per_token);
  if (t >= p.total_q) return;
  const int c = lane % p.lanes, slot = lane / p.lanes;
  const bool inter = p.interleaved != 0;
  // the lane's two chunks of a rope row, half a row apart: halves apart they are the two sides of its
  // eight pairs, interleaved four pairs each (so that an access covers whole sectors)
  struct {
    int lo, hi;
  } const ch = {8 * c, p.rope_dim / 2 + 8 * c};
  // What does not need the token's place is loaded first: the search, the table and the block table
  // are a chain of three loads.
  uint4 x[kPer], lo[U], hi[U];
  const uint16_t* const src = p.q_rope + t * p.q_stride[0];
  const int h0 = (part - 1) * p.pass_group * p.heads_per_pass;
  const int h1 = min(p.heads, h0 + p.pass_group * p.heads_per_pass);
  auto load_heads = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = base + u * p.heads_per_pass + slot;
      if (slot >= p.heads_per_pass || h >= h1) continue;
      lo[u] = *reinterpret_cast<const uint4*>(src + h * p.q_stride[1] + ch.lo);
      hi[u] = *reinterpret_cast<const uint4*>(src + h * p.q_stride[1] + ch.hi);
    }
  };
  if (part == 0) {
    const uint4* from = reinterpret_cast<const uint4*>(p.latent + t * p.latent_stride);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i + lane < L / 8) x[i] = __ldg(from + 32 * i + lane);
    if (slot == 0) {
      const uint16_t* k = p.k_rope + t * p.k_rope_stride;
      lo[0] = __ldg(reinterpret_cast<const uint4*>(k + ch.lo));
      hi[0] = __ldg(reinterpret_cast<const uint4*>(k + ch.hi));
    }
  } else {
    load_heads(h0);
  }
  const ua::SeqOf s = ua::seq_of(p.cu_seqlens_q, p.seq_lens_k, p.num_seqs, t,
                                 [](int c, int) -> long long { return c; });
  if (t < s.q0 || t >= s.end) return;
  const int at = s.kv_len - (s.end - t);
  if (at < 0) return;
  float cs[8], sn[8];
  if (p.cos_sin != nullptr) {
    const int pos = p.positions != nullptr ? __ldg(p.positions + t) : at;
    if (pos < 0 || pos >= p.max_position) {
      if (lane == 0) atomicOr(p.status, ua::DEV_BAD_POSITION);
      return;
    }
    const float* row = p.cos_sin + static_cast<size_t>(pos) * p.rope_dim;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = inter ? 4 * c + h * (p.rope_dim / 4) : 8 * c + 4 * h;
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + f));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + p.rope_dim / 2 + f));
      cs[4 * h] = a.x, cs[4 * h + 1] = a.y, cs[4 * h + 2] = a.z, cs[4 * h + 3] = a.w;
      sn[4 * h] = b.x, sn[4 * h + 1] = b.y, sn[4 * h + 2] = b.z, sn[4 * h + 3] = b.w;
    }
  }
  auto turned = [&](uint4& lo, uint4& hi) {
    if (p.cos_sin == nullptr) return;
    float a[8], b[8];
    ua::unpack16<BF>(lo, hi, inter, a, b);
    ua::turn(a, b, cs, sn);
    ua::pack16<BF>(a, b, inter, lo, hi);
  };

  if (part == 0) {
    const int col = at / p.block_size;
    const int blk = col < p.max_blocks_per_seq
                        ? __ldg(p.block_table + static_cast<size_t>(s.b) * p.max_blocks_per_seq + col)
                        : -1;
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
      if (lane == 0) atomicOr(p.status, ua::DEV_BAD_BLOCK);
      return;
    }
    uint16_t* const row = p.cache + (static_cast<size_t>(blk) * p.block_size + at % p.block_size) *
                                        static_cast<size_t>(L + p.rope_dim);
    if (p.weight != nullptr) {
      float v[kPer][8], sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool in = 32 * i + lane < L / 8;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = in ? ua::unpack2<BF>(w[e]) : make_float2(0.f, 0.f);
          v[i][2 * e] = f.x;
          v[i][2 * e + 1] = f.y;
          sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float rs = rsqrtf(sum * (1.f / L) + p.eps);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (32 * i + lane >= L / 8) continue;
        float g[8];
        if (p.weight_f32) {
          const float4* w = static_cast<const float4*>(p.weight) + 2 * (32 * i + lane);
          const float4 a = __ldg(w), b = __ldg(w + 1);
          g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
          g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
        } else {
          const uint4 w4 = __ldg(static_cast<const uint4*>(p.weight) + 32 * i + lane);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = ua::unpack2<BF>(w[e]);
            g[2 * e] = f.x;
            g[2 * e + 1] = f.y;
          }
        }
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = ua::pack2<BF>(v[i][2 * e] * rs * g[2 * e], v[i][2 * e + 1] * rs * g[2 * e + 1]);
        x[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i + lane < L / 8) reinterpret_cast<uint4*>(row)[32 * i + lane] = x[i];
    if (slot == 0) {
      turned(lo[0], hi[0]);
      *reinterpret_cast<uint4*>(row + L + ch.lo) = lo[0];
      *reinterpret_cast<uint4*>(row + L + ch.hi) = hi[0];
    }
    return;
  }

  // query heads: passes of heads_per_pass, U of them at a time
  uint16_t* const dst = p.q_rope_out + t * p.q_out_stride[0];
  for (int base = h0; base < h1; base += U * p.heads_per_pass) {
    if (base > h0) load_heads(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = base + u * p.heads_per_pass + slot;
      if (slot >= p.heads_per_pass || h >= h1) continue;
      turned(lo[u], hi[u]);
      *reinterpret_cast<uint4*>(dst + h * p.q_out_stride[1] + ch.lo) = lo[u];
      *reinterpret_cast<uint4*>(dst + h * p.q_out_stride[1] + ch.hi) = hi[u];
    }
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A stride between n rows that are read in 16-byte chunks (one row has none).
bool stride8(int64_t s, int64_t n) { return n <= 1 || (s >= 0 && s % 8 == 0); }

int append(const ua_append_latent_t& a, cudaStream_t st) {
  if (a.num_seqs < 0 || a.total_q < 0 || a.max_blocks_per_seq < 0 || a.num_blocks < 0 ||
      a.block_size < 1 || a.num_heads < 0)
    return UA_ERR_INVALID_ARG;
  if (a.latent_dim != 128 && a.latent_dim != 256 && a.latent_dim != 512) return UA_ERR_INVALID_ARG;
  if (a.rope_dim < 16 || a.rope_dim > 64 || a.rope_dim % 16 != 0) return UA_ERR_INVALID_ARG;
  if (a.dtype != UA_DT_F16 && a.dtype != UA_DT_BF16) return UA_ERR_INVALID_ARG;
  if (a.norm_weight != nullptr &&
      ((a.norm_dtype != a.dtype && a.norm_dtype != UA_DT_F32) || !aligned(a.norm_weight, 16) ||
       !(a.norm_eps >= 0.f)))
    return UA_ERR_INVALID_ARG;
  if (a.cos_sin != nullptr ? a.max_position < 1 || !aligned(a.cos_sin, 16) : a.positions != nullptr)
    return UA_ERR_INVALID_ARG;
  if (a.total_q == 0 || a.num_seqs == 0) return UA_OK;
  if (!a.latent || !a.k_rope || !a.cache || !a.cu_seqlens_q || !a.seq_lens_k || !a.block_table ||
      (a.q_rope != nullptr) != (a.num_heads > 0) || (a.q_rope && !a.q_rope_out))
    return UA_ERR_INVALID_ARG;
  for (const void* x : {a.latent, a.k_rope, a.q_rope, static_cast<const void*>(a.q_rope_out),
                        static_cast<const void*>(a.cache)})
    if (!aligned(x, 16)) return UA_ERR_INVALID_ARG;
  if (!aligned(a.positions, 4)) return UA_ERR_INVALID_ARG;
  if (!stride8(a.latent_stride, a.total_q) || !stride8(a.k_rope_stride, a.total_q))
    return UA_ERR_INVALID_ARG;
  if (a.q_rope) {
    for (int i = 0; i < 2; ++i) {
      const int64_t n = i == 0 ? a.total_q : a.num_heads;
      if (!stride8(a.q_rope_stride[i], n) || !stride8(a.q_rope_out_stride[i], n))
        return UA_ERR_INVALID_ARG;
      // in place, a row is read and written by the same lanes
      if (a.q_rope_out == a.q_rope && n > 1 && a.q_rope_out_stride[i] != a.q_rope_stride[i])
        return UA_ERR_INVALID_ARG;
    }
    // what is written may not overlap itself
    const bool head_in = a.q_rope_out_stride[1] <= a.q_rope_out_stride[0];
    const int64_t inner = a.q_rope_out_stride[head_in ? 1 : 0];
    const int64_t outer = a.q_rope_out_stride[head_in ? 0 : 1];
    const int64_t n_in = head_in ? a.num_heads : a.total_q, n_out = head_in ? a.total_q : a.num_heads;
    if ((n_in > 1 && inner < a.rope_dim) ||
        (n_out > 1 && outer < (n_in > 1 ? inner * (n_in - 1) : 0) + a.rope_dim))
      return UA_ERR_INVALID_ARG;
  }
  if (a.max_blocks_per_seq < 1 || a.num_blocks < 1) return UA_ERR_INVALID_ARG;

  AppendLatentParams p{};
  p.latent = static_cast<const uint16_t*>(a.latent);
  p.k_rope = static_cast<const uint16_t*>(a.k_rope);
  p.q_rope = static_cast<const uint16_t*>(a.q_rope);
  p.q_rope_out = static_cast<uint16_t*>(a.q_rope_out);
  p.cache = static_cast<uint16_t*>(a.cache);
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens_k = a.seq_lens_k;
  p.block_table = a.block_table;
  p.weight = a.norm_weight;
  p.weight_f32 = a.norm_dtype == UA_DT_F32;
  p.cos_sin = a.cos_sin;
  p.positions = a.positions;
  p.latent_stride = a.latent_stride;
  p.k_rope_stride = a.k_rope_stride;
  for (int i = 0; i < 2; ++i) {
    p.q_stride[i] = a.q_rope_stride[i];
    p.q_out_stride[i] = a.q_rope_out_stride[i];
  }
  int sms = 0, rc;
  if ((rc = ua::status_word(&p.status)) != UA_OK) return rc;
  if ((rc = ua::device_sm_count(&sms)) != UA_OK) return rc;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.num_blocks;
  p.block_size = a.block_size;
  p.heads = a.q_rope ? a.num_heads : 0;
  p.rope_dim = a.rope_dim;
  p.max_position = a.max_position;
  p.interleaved = a.interleaved != 0;
  p.eps = a.norm_eps;
  p.lanes = a.rope_dim / 16;
  p.heads_per_pass = 32 / p.lanes;
  const int passes = (p.heads + p.heads_per_pass - 1) / p.heads_per_pass;
  // A pass a warp while all warps fit the device at once, else four: in us, 64 heads (9 warps a token
  // if one pass each), 400 tokens (23.7 warps an SM) 3.3 with one; 416 (24.6) 3.1 with four, 4.2 with
  // one; 480 (28.4) 3.1, 4.5; 536 (31.7) 3.2, 4.7.
  const long long resident = static_cast<long long>(kWarps) * kBlocks * sms;
  p.pass_group = static_cast<long long>(a.total_q) * (1 + passes) <= resident ? 1 : 4;
  p.warps_per_token = 1 + (passes + p.pass_group - 1) / p.pass_group;
  const long long grid = (static_cast<long long>(a.total_q) * p.warps_per_token + kWarps - 1) / kWarps;
  if (grid > INT_MAX) return UA_ERR_INVALID_ARG;
  const dim3 g(static_cast<unsigned>(grid)), t(32 * kWarps);
  const bool bf = a.dtype == UA_DT_BF16;
  decltype(&ua_append_latent_kernel<512, true>) kern;
  switch (a.latent_dim) {
    case 128: kern = bf ? ua_append_latent_kernel<128, true> : ua_append_latent_kernel<128, false>; break;
    case 256: kern = bf ? ua_append_latent_kernel<256, true> : ua_append_latent_kernel<256, false>; break;
    default: kern = bf ? ua_append_latent_kernel<512, true> : ua_append_latent_kernel<512, false>; break;
  }
  return ua::launch_pdl(kern, g, t, 0, st, 1, p) == cudaSuccess ? UA_OK : UA_ERR_CUDA;
}

}  // namespace

extern "C" int ua_append_latent(const ua_append_latent_t* call, void* stream) {
  try {
    if (call == nullptr) return UA_ERR_INVALID_ARG;
    return append(*call, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return UA_ERR_CUDA;
  }
}
