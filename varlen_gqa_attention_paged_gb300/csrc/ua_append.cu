// ua_append.cu -- ua_append_kv: argument checks, launch shapes and instantiations of the
// cache-writing kernels.
#include <algorithm>
#include <climits>

#include "ua_append.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Row strides of a [tokens, heads, D] tensor whose rows are read in 16-byte chunks.
bool row_strides(const int64_t* s) {
  return s[0] >= 0 && s[1] >= 0 && s[0] % 8 == 0 && s[1] % 8 == 0;
}

// No two elements of a written array [s0][s1](..[inner contiguous]) share memory: each stride,
// from the smallest, clears what lies under it.  (Sizes of one have no stride.)
template <int N>
bool disjoint(const int64_t* stride, const int64_t (&size)[N], int64_t inner) {
  int order[N];
  for (int i = 0; i < N; ++i) order[i] = i;
  std::sort(order, order + N, [&](int a, int b) { return stride[a] < stride[b]; });
  __int128 reach = inner;
  for (int i : order) {
    if (size[i] <= 1) continue;
    if (stride[i] < reach) return false;
    reach = static_cast<__int128>(stride[i]) * size[i];
  }
  return true;
}

int check(const ua_append_t& a) {
  if (a.num_seqs < 0 || a.total_q < 0 || a.max_seqlen_q < 0 || a.max_blocks_per_seq < 0 ||
      a.num_blocks < 0 || a.block_size < 1 || a.num_kv_heads < 1 || a.num_q_heads < 0)
    return UA_ERR_INVALID_ARG;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return UA_ERR_INVALID_ARG;
  if (a.dtype != UA_DT_F16 && a.dtype != UA_DT_BF16) return UA_ERR_INVALID_ARG;
  const bool f8 = a.kv_dtype == UA_DT_F8E4M3, i8 = a.kv_dtype == UA_DT_I8;
  if (!f8 && !i8) {
    if (a.kv_dtype != UA_DT_F16 && a.kv_dtype != UA_DT_BF16) return UA_ERR_INVALID_ARG;
    if (a.kv_dtype != a.dtype) return UA_ERR_UNSUPPORTED;
  }
  if (a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 16 != 0) return UA_ERR_INVALID_ARG;
  if ((a.cos_sin == nullptr) != (a.rot_dim == 0)) return UA_ERR_INVALID_ARG;
  if (a.rot_dim > 0) {
    if (a.max_position < 1 || !aligned(a.cos_sin, 16)) return UA_ERR_INVALID_ARG;
    if (a.n_axes < 1 || a.n_axes > ua::kMaxAxes) return UA_ERR_INVALID_ARG;
    if (a.n_axes > 1) {
      if (a.positions == nullptr || a.axis_of == nullptr || a.positions_stride < 0)
        return UA_ERR_INVALID_ARG;
      for (int f = 0; f < a.rot_dim / 2; ++f)
        if (a.axis_of[f] >= a.n_axes) return UA_ERR_INVALID_ARG;
    }
  }
  // exactly one form of scales for an 8-bit cache (per block for int8), none for a 16-bit one
  const bool tok = a.k_scale_tok || a.v_scale_tok, blk = a.k_scale_blk || a.v_scale_blk;
  const int forms = (a.kv_scale ? 1 : 0) + (tok ? 1 : 0) + (blk ? 1 : 0);
  if ((f8 || i8) ? forms != 1 : forms != 0) return UA_ERR_INVALID_ARG;
  if (i8 && !blk) return UA_ERR_INVALID_ARG;
  if (tok && (!a.k_scale_tok || !a.v_scale_tok)) return UA_ERR_INVALID_ARG;
  if (blk && (!a.k_scale_blk || !a.v_scale_blk)) return UA_ERR_INVALID_ARG;
  return UA_OK;
}

template <int D, bool BF, bool I8>
cudaError_t launch_blk(const ua::AppendParams& p, dim3 g, dim3 t, bool filled, cudaStream_t st) {
  const bool one = p.block_size <= static_cast<int>(t.x) / (D / 16);
  const auto kern = !one     ? ua::ua_append_blk_kernel<D, BF, I8, false, 3>
                    : filled ? ua::ua_append_blk_kernel<D, BF, I8, true, 4>
                             : ua::ua_append_blk_kernel<D, BF, I8, true, 3>;
  return ua::launch_pdl(kern, g, t, 0, st, 1, p);
}

template <int D, bool BF>
cudaError_t launch(const ua::AppendParams& p, ua::AppendKind kind, unsigned grid, int threads,
                   bool filled, cudaStream_t st) {
  const dim3 g(grid), t(static_cast<unsigned>(threads));
  switch (kind) {
    case ua::APP_16:
      return ua::launch_pdl(ua::ua_append_rows_kernel<D, BF, ua::APP_16>, g, t, 0, st, 1, p);
    case ua::APP_E4M3:
      return ua::launch_pdl(ua::ua_append_rows_kernel<D, BF, ua::APP_E4M3>, g, t, 0, st, 1, p);
    case ua::APP_E4M3_TOK:
      return ua::launch_pdl(ua::ua_append_rows_kernel<D, BF, ua::APP_E4M3_TOK>, g, t, 0, st, 1, p);
    case ua::APP_E4M3_BLK: return launch_blk<D, BF, false>(p, g, t, filled, st);
    default: return launch_blk<D, BF, true>(p, g, t, filled, st);
  }
}

int append(const ua_append_t& a, cudaStream_t st) {
  int rc = check(a);
  if (rc != UA_OK) return rc;
  if (a.total_q == 0 || a.num_seqs == 0) return UA_OK;
  if (!a.k || !a.v || !a.k_cache || !a.v_cache || !a.cu_seqlens_q || !a.seq_lens_k ||
      !a.block_table || (a.q != nullptr) != (a.num_q_heads > 0) || (a.q && !a.q_out))
    return UA_ERR_INVALID_ARG;
  for (const void* x : {a.k, a.v, a.q, static_cast<const void*>(a.q_out),
                        static_cast<const void*>(a.k_cache), static_cast<const void*>(a.v_cache)})
    if (!aligned(x, 16)) return UA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(a.kv_scale),
                        static_cast<const void*>(a.k_scale_tok),
                        static_cast<const void*>(a.v_scale_tok),
                        static_cast<const void*>(a.k_scale_blk),
                        static_cast<const void*>(a.v_scale_blk),
                        static_cast<const void*>(a.positions)})
    if (!aligned(x, 4)) return UA_ERR_INVALID_ARG;
  if (!row_strides(a.k_stride) || !row_strides(a.v_stride)) return UA_ERR_INVALID_ARG;
  if (a.q && (!row_strides(a.q_stride) || !row_strides(a.q_out_stride))) return UA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (a.k_scale_tok && (a.k_scale_tok_stride[i] < 0 || a.v_scale_tok_stride[i] < 0))
      return UA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    if (a.k_scale_blk && (a.k_scale_blk_stride[i] < 0 || a.v_scale_blk_stride[i] < 0))
      return UA_ERR_INVALID_ARG;
  // what is written may not overlap itself
  const int64_t rows[2] = {a.total_q, a.num_q_heads};
  const int64_t tok[3] = {a.num_blocks, a.block_size, a.num_kv_heads};
  const int64_t blocks[2] = {a.num_blocks, a.num_kv_heads};
  if (a.q && !disjoint(a.q_out_stride, rows, a.head_dim)) return UA_ERR_INVALID_ARG;
  if (a.k_scale_tok &&
      !(disjoint(a.k_scale_tok_stride, tok, 1) && disjoint(a.v_scale_tok_stride, tok, 1)))
    return UA_ERR_INVALID_ARG;
  if (a.k_scale_blk &&
      !(disjoint(a.k_scale_blk_stride, blocks, 1) && disjoint(a.v_scale_blk_stride, blocks, 1)))
    return UA_ERR_INVALID_ARG;
  if (a.max_blocks_per_seq < 1 || a.num_blocks < 1) return UA_ERR_INVALID_ARG;

  int sms = 0;
  if ((rc = ua::device_sm_count(&sms)) != UA_OK) return rc;
  ua::AppendParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens_k = a.seq_lens_k;
  p.block_table = a.block_table;
  p.cos_sin = a.cos_sin;
  p.positions = a.positions;
  p.kv_scale = a.kv_scale;
  for (int i = 0; i < 2; ++i) {
    p.q_stride[i] = a.q_stride[i];
    p.k_stride[i] = a.k_stride[i];
    p.v_stride[i] = a.v_stride[i];
    p.q_out_stride[i] = a.q_out_stride[i];
  }
  const bool blk = a.k_scale_blk != nullptr;
  if (blk) {
    p.k_scale = a.k_scale_blk;
    p.v_scale = a.v_scale_blk;
    p.k_scale_stride[0] = a.k_scale_blk_stride[0];
    p.k_scale_stride[2] = a.k_scale_blk_stride[1];
    p.v_scale_stride[0] = a.v_scale_blk_stride[0];
    p.v_scale_stride[2] = a.v_scale_blk_stride[1];
  } else if (a.k_scale_tok) {
    p.k_scale = a.k_scale_tok;
    p.v_scale = a.v_scale_tok;
    for (int i = 0; i < 3; ++i) {
      p.k_scale_stride[i] = a.k_scale_tok_stride[i];
      p.v_scale_stride[i] = a.v_scale_tok_stride[i];
    }
  }
  p.pos_stride = a.positions_stride;
  if ((rc = ua::status_word(&p.status)) != UA_OK) return rc;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.num_blocks;
  p.block_size = a.block_size;
  p.hq = a.q ? a.num_q_heads : 0;
  p.hkv = a.num_kv_heads;
  p.rot_dim = a.rot_dim;
  p.max_position = a.max_position;
  p.interleaved = a.interleaved != 0;
  p.n_axes = a.rot_dim > 0 ? a.n_axes : 0;
  if (p.n_axes > 1) {
    std::copy(a.axis_of, a.axis_of + a.rot_dim / 2, p.axis_of);
    for (int i = 0; i < a.rot_dim / 8; ++i) {
      const uint8_t* f = a.axis_of + 4 * i;
      p.axis4[i] = f[0] == f[1] && f[0] == f[2] && f[0] == f[3] ? f[0] : 255;
    }
  }

  const ua::AppendKind kind = a.kv_dtype == UA_DT_I8         ? ua::APP_I8_BLK
                              : a.kv_dtype != UA_DT_F8E4M3   ? ua::APP_16
                              : blk                          ? ua::APP_E4M3_BLK
                              : a.k_scale_tok                ? ua::APP_E4M3_TOK
                                                             : ua::APP_E4M3;
  // Warps of the row kernel (and of the block kernel's query part): one takes a token's heads
  // in groups of passes, 512 / D heads each.  The group size is the one that is done first in
  // whole waves of resident warps, a warp costing its passes and about four more (its search
  // and the loads that wait for it): 28.7 against 31.9 us for ragged chunks of up to 1500
  // tokens at head_dim 256 with half the passes, 15.9 against 19.7 us for chunks of up to 700
  // with all of them.
  const int rpp = 512 / a.head_dim;
  p.passes = (p.hq + rpp - 1) / rpp + (blk ? 0 : 2 * ((p.hkv + rpp - 1) / rpp));
  p.pass_group = std::max(1, p.passes);
  long long best = LLONG_MAX;
  for (int groups = 1; groups <= p.passes; ++groups) {
    const int g = (p.passes + groups - 1) / groups;
    const long long warps = static_cast<long long>(a.total_q) * ((p.passes + g - 1) / g);
    const long long wave = 4LL * ua::kRowsMinBlocks * sms;
    const long long cost = (warps + wave - 1) / wave * (g + 4);
    if (cost < best) best = cost, p.pass_group = g;
  }
  const long long row_warps =
      p.passes == 0 ? 0
                    : static_cast<long long>(a.total_q) *
                          ((p.passes + p.pass_group - 1) / p.pass_group);
  int threads = 128;
  long long grid;
  bool filled = false;
  if (blk) {
    const int bs = a.block_size;
    const int lanes = (a.head_dim / 16) * std::min(bs, ua::kBlkThreads);
    threads = std::max(64, std::min(ua::kBlkThreads, (lanes + 31) / 32 * 32));
    p.slot_per_seq = a.max_seqlen_q <= 1;
    const long long slots = p.slot_per_seq ? a.num_seqs : a.total_q / bs + 2LL * a.num_seqs;
    if (slots > INT_MAX) return UA_ERR_INVALID_ARG;
    p.slots = static_cast<int>(slots);
    // a CTA walks kv-heads (its rows' cosines and sines stay in registers) while the grid
    // still has three CTAs an SM
    auto hgroups = [&] { return (p.hkv + p.heads_per_cta - 1) / p.heads_per_cta; };
    p.heads_per_cta = p.hkv;
    while (p.heads_per_cta > 1 && static_cast<long long>(p.slots) * hgroups() < 3LL * sms)
      p.heads_per_cta = (p.heads_per_cta + 1) / 2;
    const int warps = threads / 32;
    grid = static_cast<long long>(p.slots) * hgroups() + (row_warps + warps - 1) / warps;
    filled = grid * threads > 3LL * sms * ua::kBlkThreads;
  } else {
    grid = (row_warps + 3) / 4;
  }
  if (grid > INT_MAX) return UA_ERR_INVALID_ARG;
  const unsigned gx = static_cast<unsigned>(grid);
  const bool bf = a.dtype == UA_DT_BF16;
  decltype(&launch<64, true>) run;
  switch (a.head_dim) {
    case 64: run = bf ? launch<64, true> : launch<64, false>; break;
    case 128: run = bf ? launch<128, true> : launch<128, false>; break;
    default: run = bf ? launch<256, true> : launch<256, false>; break;
  }
  const cudaError_t err = run(p, kind, gx, threads, filled, st);
  return err == cudaSuccess ? UA_OK : UA_ERR_CUDA;
}

}  // namespace

extern "C" int ua_append_kv(const ua_append_t* call, void* stream) {
  try {
    if (call == nullptr) return UA_ERR_INVALID_ARG;
    return append(*call, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return UA_ERR_CUDA;
  }
}
