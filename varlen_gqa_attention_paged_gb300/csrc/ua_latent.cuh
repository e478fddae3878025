// ua_latent.cuh -- attention over a paged cache of latent vectors, absorbed form (included by
// ua_latent_l*.cu).
//
// A cache row is [c | r]: L latent elements, keys and values at once, and R rope elements, keys
// only.  Row i of a sequence (its query tokens' heads one after the other) attends with
//   s_j = scale q_i . [c_j | r_j],   o_i = sum_j 2^(s_j log2 e - m) c_j / sum_j 2^(s_j log2 e - m)
// so a key is read once for all heads: 2 H (2 L + R) flops on 2 (L + R) bytes, 30 flops a byte with
// 16 heads (bound by HBM) and 242 with 128 (by both).
//
// A CTA owns 64 rows.  S (64 rows x 64 keys) = Q K^T runs with the rows on the MMA's M side, O is
// kept transposed, O^T (L x 64 rows) += V^T P^T, in L / 128 accumulators of 128 x 64: with L = 512
// O takes 256 of tensor memory's 512 columns, which as rows x L it would take whole, with no
// room for S.  A key tile (64 keys x (L + R), 73.7 KB) is loaded once and read twice, as K and as
// V; two of them and Q fill the shared memory, so P has one buffer and the softmax of tile j + 1
// hands it over when P.V of tile j is done.
//
// Work split: all (row tile, key tile) pairs of the batch, row tile after row tile, are cut into
// equal shares for the workers (one CTA, or two that take neighbouring row tiles of a sequence over
// the same keys, so that the second read of a key hits L2).  A row tile that ends up with
// several workers leaves fp32 partial rows for the merge kernel.
#pragma once

#include <atomic>

#include "ua_latent.h"
#include "ua_prefill.cuh"

#include "ua.h"

namespace ua {

template <int L>
struct LatentCfg {
  static constexpr int kCB = L / 64;             // column blocks of the latent part
  static constexpr int kCH = kCB + 1;            // and the rope part's
  static constexpr int kMB = L / 128;            // accumulators of O^T
  static constexpr int kQCB = kLatRows * 128;    // one column block of Q
  static constexpr int kQBytes = kCH * kQCB;
  static constexpr int kGroup = kCH * 1024;      // eight keys: every column block's 8 x 128 bytes
  static constexpr int kTileBytes = kLatKeys / 8 * kGroup;
  static constexpr int kPBytes = kLatRows * 128;
  static constexpr int kSmallBytes = 1024;       // barriers, rescale factors
  static constexpr int kFit =
      (227 * 1024 - 1024 - kSmallBytes - kQBytes - kPBytes) / kTileBytes;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kSmemBytes =
      1024 + kQBytes + kStages * kTileBytes + kPBytes + kSmallBytes;
  static constexpr int kTmemO = 2 * kLatKeys;    // two S buffers, then O^T
  static constexpr int kTmemCols = kTmemO + kMB * kLatRows > 256 ? 512 : 256;
  static constexpr int kThreads = 192;           // four softmax warps, MMA issue, copies
  static_assert(L % 128 == 0 && L <= 512);
  static_assert(kStages >= 2 && kSmemBytes + 16 <= 227 * 1024);
};

// A worker's walk over its share: segments of consecutive key tiles of one row tile.  Every warp
// walks it for itself.
struct LatentWalk {
  long long pos, left, share;   // next unit, units left, units of a share
  int b, t, j;                  // sequence, row tile of the worker, key tile
  int q0, q_len, kv_len, rows, rt, kt;

  // Rows of the tokens [q0, q1) (those from total_q on have none).
  __device__ __forceinline__ static int rows_of(const LatentParams& p, int q0, int q1) {
    return q0 < 0 ? 0 : max(0, min(q1, p.total_q) - q0) * p.heads;
  }
  __device__ __forceinline__ static int row_tiles(const LatentParams& p, int rows) {
    return (rows + kLatRows * p.cl - 1) / (kLatRows * p.cl);
  }
  // (a sequence without keys has one empty tile, whose rows are written as 0)
  __device__ __forceinline__ static int key_tiles(int kv_len) {
    return max(1, (max(kv_len, 0) + kLatKeys - 1) / kLatKeys);
  }
  __device__ __forceinline__ void load(const LatentParams& p) {
    q0 = __ldg(p.cu_seqlens_q + b);
    const int q1 = __ldg(p.cu_seqlens_q + b + 1);
    q_len = q1 - q0;
    kv_len = max(0, __ldg(p.seq_lens_k + b));
    rows = rows_of(p, q0, q1);
    rt = row_tiles(p, rows);
    kt = key_tiles(kv_len);
  }

  // Called by a whole warp.
  __device__ __forceinline__ LatentWalk(const LatentParams& p, int worker) {
    const int lane = threadIdx.x & 31;
    auto units = [&](int i) -> long long {
      if (i >= p.num_seqs) return 0;
      const int n = rows_of(p, __ldg(p.cu_seqlens_q + i), __ldg(p.cu_seqlens_q + i + 1));
      return static_cast<long long>(row_tiles(p, n)) * key_tiles(__ldg(p.seq_lens_k + i));
    };
    const long long first = units(lane);
    long long total = first;
    for (int base = 32; base < p.num_seqs; base += 32) total += units(base + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    share = max(static_cast<long long>(p.min_share), (total + p.workers - 1) / p.workers);
    pos = worker * share;
    left = min(share, total - pos);
    b = t = j = 0;
    q0 = q_len = kv_len = rows = rt = kt = 0;
    if (left <= 0) return;
    long long before = 0;
    for (int base = 0; base < p.num_seqs; base += 32) {
      const long long u = base == 0 ? first : units(base + lane);
      long long end = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += x;
      }
      const unsigned m = __ballot_sync(0xffffffffu, before + end > pos);
      if (m != 0u) {
        const int src = __ffs(m) - 1;
        const long long off = pos - before - __shfl_sync(0xffffffffu, end - u, src);
        b = base + src;
        load(p);
        t = static_cast<int>(off / kt);
        j = static_cast<int>(off % kt);
        return;
      }
      before += __shfl_sync(0xffffffffu, end, 31);
    }
    left = 0;
  }

  __device__ __forceinline__ int length() const {
    return static_cast<int>(min(left, static_cast<long long>(kt - j)));
  }
  __device__ __forceinline__ void next(const LatentParams& p) {
    const int n = length();
    pos += n;
    left -= n;
    j += n;
    if (j < kt || left <= 0) return;
    j = 0;
    if (++t < rt) return;
    t = 0;
    do {
      ++b;
      load(p);
    } while (rt == 0 && b + 1 < p.num_seqs);
  }
};

// A segment as one CTA of the worker sees it.
struct LatentSeg {
  int row0;       // its first row within the sequence
  int rows;       // its rows (<= 0: none)
  int ctx, seen;  // cached tokens before the new ones; the keys that its last row sees
  int j0, nt;     // key tiles [j0, j0 + nt) that a row of it may see
  __device__ __forceinline__ LatentSeg(const LatentParams& p, const LatentWalk& w, int rank) {
    row0 = (w.t * p.cl + rank) * kLatRows;
    rows = min(kLatRows, w.rows - row0);
    ctx = w.kv_len - w.q_len;
    seen = w.kv_len;
    if (rows > 0 && p.tree == nullptr)
      seen = max(0, min(seen, ctx + (row0 + rows - 1) / p.heads + 1));
    j0 = w.j;
    nt = rows <= 0 ? 0 : max(0, min(w.j + w.length(), (seen + kLatKeys - 1) / kLatKeys) - w.j);
  }
};

// Whether `v` holds in any of the barrier's threads; a barrier too.
__device__ __forceinline__ bool named_bar_any(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Bits [at, at + 32) of a row of words (at may be negative; words past the row are 0).
__device__ __forceinline__ uint32_t mask_bits32(const int32_t* words, int n, int at) {
  const int w = at >> 5, s = at & 31;
  const uint32_t lo = w >= 0 && w < n ? static_cast<uint32_t>(__ldg(words + w)) : 0u;
  const uint32_t hi = w + 1 >= 0 && w + 1 < n ? static_cast<uint32_t>(__ldg(words + w + 1)) : 0u;
  return __funnelshift_r(lo, hi, s);
}
// The low n bits (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  return BF16 ? pack_bf16(a, b) : pack_f16(a, b);
}

__device__ __forceinline__ void store_as(void* out, size_t at, float v, int dtype) {
  if (dtype == UA_DT_F32) static_cast<float*>(out)[at] = v;
  else if (dtype == UA_DT_BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[at] = __float2half_rn(v);
}

// ln of a row's sum: m its running max in log2 units, l the sum of 2^(x - m).
__device__ __forceinline__ float latent_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int L, bool BF16>
__global__ void __launch_bounds__(LatentCfg<L>::kThreads, 1)
    ua_latent_kernel(const __grid_constant__ LatentParams p) {
  using C = LatentCfg<L>;
  constexpr int S = C::kStages;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sQ = smem;
  uint8_t* const sK = sQ + C::kQBytes;
  uint8_t* const sP = sK + S * C::kTileBytes;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sP + C::kPBytes);
  uint64_t* const q_full = bars + 0;
  uint64_t* const q_empty = bars + 1;
  uint64_t* const s_full = bars + 2;   // [2]
  uint64_t* const p_full = bars + 4;
  uint64_t* const pv_done = bars + 5;
  uint64_t* const o_empty = bars + 6;
  uint64_t* const fin = bars + 7;
  uint64_t* const k_full = bars + 8;   // [S]
  uint64_t* const k_empty = k_full + S;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(k_empty + S);
  float* const sF = reinterpret_cast<float*>(bars + 32);  // [2][64] factors of O's rows
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int worker = blockIdx.x / p.cl, rank = blockIdx.x % p.cl;
  constexpr int kMma = 4, kCopy = 5;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    mbar_init(o_empty, 4);
    mbar_init(fin, 1);
    for (int i = 0; i < S; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kCopy && lane == 0) {
    tma_prefetch_desc(&p.q_lat);
    tma_prefetch_desc(&p.q_row);
    tma_prefetch_desc(&p.k_lat);
    tma_prefetch_desc(&p.k_row);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  volatile int* abort_flag = &s_abort;
  grid_dependency_wait();
  grid_launch_dependents();

  LatentWalk w(p, worker);
  int it = 0;  // key tiles of all segments so far
  int sg = 0;  // segments with key tiles so far
  bool ok = true;

  if (warp == kCopy) {
    // ======================================================== copies
    const int bs = p.block_size;
    const int oob = p.num_blocks * bs;
    const int per_lane = p.box_rows == 8 ? 1 : 2;  // boxes of a tile that a lane loads
    for (; ok && w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      if (s.nt <= 0) continue;
      if (sg > 0 && !pf_wait_warp(q_empty, (sg - 1) & 1, abort_flag, p.status)) { ok = false; break; }
      if (lane == 0) {
        const int row = w.q0 * p.heads + s.row0;
        mbar_arrive_expect_tx(q_full, C::kQBytes);
        tma_load_3d_pf(sQ, &p.q_lat, 0, row, 0, q_full);
        tma_load_2d(sQ + C::kCB * C::kQCB, &p.q_row, L, row, q_full);
      }
      ++sg;
      const int32_t* bt = p.block_table + static_cast<size_t>(w.b) * p.max_blocks_per_seq;
      // the block of this lane's box i of key tile j, loaded two tiles ahead of its use
      auto key_of = [&](int j, int i) -> int {
        return j * kLatKeys + (p.box_rows == 8 ? 8 * lane : lane + 32 * i);
      };
      auto block_of = [&](int j, int i) -> int {
        if (j >= s.j0 + s.nt || i >= per_lane || (p.box_rows == 8 && lane >= 8)) return -1;
        const int key = key_of(j, i), col = key / bs;
        return key < w.kv_len && col < p.max_blocks_per_seq ? __ldg(bt + col) : -1;
      };
      // its cache row (past the cache, so that the copy fills zeros, where there is no key)
      auto row_of = [&](int j, int i, int blk) -> int {
        const int key = key_of(j, i);
        if (key >= w.kv_len) return oob;
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
          atomicOr(p.status, DEV_BAD_BLOCK);
          return oob;
        }
        return blk * bs + key % bs;
      };
      int blk0[2], blk1[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        blk0[i] = block_of(s.j0, i);
        blk1[i] = block_of(s.j0 + 1, i);
      }
      for (int n = 0; n < s.nt; ++n, ++it) {
        const int j = s.j0 + n, st = it % S;
        if (it >= S && !pf_wait_warp(&k_empty[st], ((it / S) - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], C::kTileBytes);
        __syncwarp();
        uint8_t* const tile = sK + st * C::kTileBytes;
        if (p.box_rows == 8) {
          if (lane < 8) {
            const int row = row_of(j, 0, blk0[0]);
            uint8_t* const dst = tile + lane * C::kGroup;
            tma_load_3d_pf(dst, &p.k_lat, 0, row, 0, &k_full[st]);
            tma_load_2d(dst + C::kCB * 1024, &p.k_row, L, row, &k_full[st]);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            const int k = lane + 32 * i;
            const int row = row_of(j, i, blk0[i]);
            uint8_t* const dst = tile + (k >> 3) * C::kGroup + (k & 7) * 128;
#pragma unroll 1
            for (int cb = 0; cb < C::kCH; ++cb)
              tma_load_2d(dst + cb * 1024, &p.k_row, 64 * cb, row, &k_full[st]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          blk0[i] = blk1[i];
          blk1[i] = block_of(j + 2, i);
        }
      }
    }
    // never leave copies in flight into this CTA's shared memory (even after an abort)
    for (int i = max(0, it - S); i < it; ++i)
      mbar_wait_bounded(&k_full[i % S], (i / S) & 1, p.status, DEV_TIMEOUT);
    if (sg > 0) mbar_wait_bounded(q_full, (sg - 1) & 1, p.status, DEV_TIMEOUT);
  } else if (warp == kMma) {
    // ======================================================== MMA issue
    // Per segment: S_0, S_1, then for every tile j: [P_j ready] O^T += V_j^T P_j^T, S_{j+2}.
    // S_{j+2} overwrites S_j, which the softmax has read when P_j is ready.
    constexpr uint32_t kIdQK = umma_idesc_f16(kLatRows, kLatKeys, BF16, false);
    constexpr uint32_t kIdPV = umma_idesc_f16(128, kLatRows, BF16, false) | (1u << 15);
    const int qk_steps = L / 16 + p.rope_dim / 16;
    for (; ok && w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      if (s.nt <= 0) continue;
      if (!pf_wait_warp(q_full, sg & 1, abort_flag, p.status)) { ok = false; break; }
      auto qk = [&](int n) -> bool {
        const int i = it + n, st = i % S;
        if (!pf_wait_warp(&k_full[st], (i / S) & 1, abort_flag, p.status)) return false;
        tc_fence_after();
        const uint32_t qb = smem_addr(sQ), kb = smem_addr(sK + st * C::kTileBytes);
#pragma unroll 4
        for (int kk = 0; kk < qk_steps; ++kk) {
          const uint64_t ad = smem_desc_sw128(qb + (kk >> 2) * C::kQCB + (kk & 3) * 32, 16, 1024);
          const uint64_t bd =
              smem_desc_sw128(kb + (kk >> 2) * 1024 + (kk & 3) * 32, 16, C::kGroup);
          umma_f16_ss_warp(tmem + (i & 1) * kLatKeys, ad, bd, kIdQK, kk > 0 ? 1u : 0u);
        }
        umma_commit_warp(&s_full[i & 1]);
        if (n == s.nt - 1) umma_commit_warp(q_empty);
        return true;
      };
      auto pv = [&](int n) -> bool {
        const int i = it + n, st = i % S;
        if (!pf_wait_warp(p_full, i & 1, abort_flag, p.status)) return false;
        if (n == 0 && sg > 0 && !pf_wait_warp(o_empty, (sg - 1) & 1, abort_flag, p.status))
          return false;
        tc_fence_after();
        const uint32_t vb = smem_addr(sK + st * C::kTileBytes), pb = smem_addr(sP);
#pragma unroll
        for (int ks = 0; ks < kLatKeys / 16; ++ks)
#pragma unroll
          for (int mb = 0; mb < C::kMB; ++mb) {
            const uint64_t ad =
                smem_desc_sw128(vb + ks * 2 * C::kGroup + mb * 2048, 1024, C::kGroup);
            const uint64_t bd = smem_desc_sw128(pb + ks * 32, 16, 1024);
            umma_f16_ss_warp(tmem + C::kTmemO + mb * kLatRows, ad, bd, kIdPV,
                             n > 0 || ks > 0 ? 1u : 0u);
          }
        umma_commit_warp(pv_done);
        umma_commit_warp(&k_empty[st]);
        return true;
      };
      ok = qk(0);
      if (ok && s.nt > 1) ok = qk(1);
      for (int n = 0; ok && n < s.nt; ++n) {
        ok = pv(n);
        if (ok && n + 2 < s.nt) ok = qk(n + 2);
      }
      it += s.nt;
      ++sg;
    }
    // nothing may still be in flight on the tensor cores when the memory is freed
    umma_commit_warp(fin);
    mbar_wait_bounded(fin, 0, p.status, DEV_TIMEOUT);
  } else {
    // ======================================================== softmax, rescale, epilogue
    // An M = 64 accumulator keeps rows 16 w .. 16 w + 15 in the first half of warp w's lanes.
    const bool has_row = lane < 16;
    const int r = 16 * warp + (lane & 15);
    const uint32_t lane_off = (32u * warp) << 16;
    const uint32_t tO = tmem + C::kTmemO + lane_off;
    const float c = p.scale * kLog2e;
    int4 meta = make_int4(0, 0, 0, 0);
    // (After a wait that gave up, these warps go on to the end, through every barrier that they
    // share; their later waits return at once, and nothing is stored.)
    for (; w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      const int grow0 = w.q0 * p.heads + s.row0;  // its first row in q and out
      const bool whole = w.j == 0 && w.length() == w.kt;
      const int slot = 2 * blockIdx.x + (w.j == 0 ? 1 : 0);
      const int rows = s.rows;
      if (rows <= 0) continue;
      if (w.j == 0 && !whole)
        meta = make_int4(grow0, rows,
                         static_cast<int>((w.pos + w.kt - 1) / w.share) - worker + 1, 0);
      const bool rv = has_row && r < rows;
      const int i_q = (s.row0 + min(r, rows - 1)) / p.heads;  // the row's token
      const int32_t* tree = p.tree == nullptr || !rv
                                ? nullptr
                                : p.tree + (static_cast<long long>(w.q0) + i_q) * p.tree_stride;
      // keys that every row of the tile sees without looking at its mask
      const int clear = min(w.kv_len, p.tree != nullptr ? s.ctx : s.ctx + s.row0 / p.heads + 1);
      float m = -INFINITY, l = 0.f;
      for (int n = 0; n < s.nt; ++n, ++it) {
        ok = pf_wait_warp(&s_full[it & 1], (it >> 1) & 1, abort_flag, p.status) && ok;
        tc_fence_after();
        const int k0 = (s.j0 + n) * kLatKeys;
        const uint32_t tS = tmem + (it & 1) * kLatKeys + lane_off;
        uint32_t xa[32], xb[32];
        tmem_ld32(tS, xa);
        tmem_ld32(tS + 32, xb);
        tmem_ld_wait();
        if (k0 + kLatKeys > clear) {
          // the keys that the row sees: of the prefix (tree) or up to its own, and those its
          // mask names
          const int end = min(w.kv_len, p.tree != nullptr ? s.ctx : s.ctx + i_q + 1) - k0;
          uint32_t ma = low_bits(end), mb = low_bits(end - 32);
          if (tree != nullptr) {
            const int last = w.kv_len - k0;
            ma |= mask_bits32(tree, p.tree_words, k0 - s.ctx) & low_bits(last) &
                  ~low_bits(s.ctx - k0);
            mb |= mask_bits32(tree, p.tree_words, k0 + 32 - s.ctx) & low_bits(last - 32) &
                  ~low_bits(s.ctx - k0 - 32);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (!((ma >> e) & 1u)) xa[e] = 0xff800000u;
            if (!((mb >> e) & 1u)) xb[e] = 0xff800000u;
          }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          mx0 = fmax3(mx0, __uint_as_float(xa[e]), __uint_as_float(xa[e + 1]));
          mx1 = fmax3(mx1, __uint_as_float(xb[e]), __uint_as_float(xb[e + 1]));
        }
        const float mx = fmaxf(mx0, mx1) * c;
        // The running max moves only by more than 8 in log2 units (P stays <= 256, inside f16's
        // range and fp32 sums'), or to a row's first key.
        float alpha = 1.f;
        const bool grow = rv && (mx > m + 8.f || (m == -INFINITY && mx > -INFINITY));
        if (grow) {
          alpha = m == -INFINITY ? 0.f : fast_exp2(m - mx);
          m = mx;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        // P rounded to 16 bits for the MMA (half a step of 2^-8 or 2^-11 of each weight); the
        // sum is of the unrounded weights
        uint32_t pk[32];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = fast_exp2(fmaf(__uint_as_float(xa[2 * e]), c, -mu));
          const float b = fast_exp2(fmaf(__uint_as_float(xa[2 * e + 1]), c, -mu));
          l0 += a;
          l1 += b;
          pk[e] = pack_half2<BF16>(a, b);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = fast_exp2(fmaf(__uint_as_float(xb[2 * e]), c, -mu));
          const float b = fast_exp2(fmaf(__uint_as_float(xb[2 * e + 1]), c, -mu));
          l0 += a;
          l1 += b;
          pk[16 + e] = pack_half2<BF16>(a, b);
        }
        l = l * alpha + (l0 + l1);
        // P's buffer and O are free when the P.V before is done
        if (it > 0) ok = pf_wait_warp(pv_done, (it - 1) & 1, abort_flag, p.status) && ok;
        tc_fence_after();
        if (n > 0) {
          float* const f = sF + (it & 1) * kLatRows;
          if (has_row) f[r] = alpha;
          if (named_bar_any(1, 128, grow)) {
#pragma unroll 1
            for (int cc = 0; cc < C::kMB * 2; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * cc, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 a = *reinterpret_cast<const float4*>(f + 32 * (cc & 1) + e);
                o[e] = __float_as_uint(__uint_as_float(o[e]) * a.x);
                o[e + 1] = __float_as_uint(__uint_as_float(o[e + 1]) * a.y);
                o[e + 2] = __float_as_uint(__uint_as_float(o[e + 2]) * a.z);
                o[e + 3] = __float_as_uint(__uint_as_float(o[e + 3]) * a.w);
              }
              tmem_st32(tO + 32 * cc, o);
            }
            tmem_st_wait();
          }
        }
        if (has_row) {
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(sP + r * 128 + ((ch ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
        }
        // Cache slots at or past kv_len may hold anything (NaN included): those that a copy of
        // eight rows brought in become zeros before they meet P = 0.
        if (k0 + kLatKeys > w.kv_len && (w.kv_len & 7) != 0) {
          const int lo = w.kv_len - k0, n0 = 8 - (lo & 7);
          uint8_t* const tile = sK + (it % S) * C::kTileBytes + (lo >> 3) * C::kGroup;
          for (int e = threadIdx.x; e < n0 * C::kCB * 8; e += 128) {
            const int row = (lo & 7) + e / (C::kCB * 8), x = e % (C::kCB * 8);
            *reinterpret_cast<uint4*>(tile + (x >> 3) * 1024 + row * 128 + (x & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }

      // ---- epilogue: O / l of a tile that is this worker's alone, else the partial rows
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that saw no key is 0; NaN stays)
      float* const f = sF + (it & 1) * kLatRows;
      if (s.nt > 0) {
        ok = pf_wait_warp(pv_done, (it - 1) & 1, abort_flag, p.status) && ok;
        tc_fence_after();
      }
      if (rv && ok) {
        if (whole) {
          if (p.lse != nullptr)
            p.lse[grow0 + r] = latent_lse(m, l);
        } else {
          p.ws_m[slot * kLatRows + r] = m;
          p.ws_l[slot * kLatRows + r] = l;
        }
      }
      if (has_row) f[r] = whole ? inv : 1.f;
      named_bar_sync(1, 128);
      const int d = 32 * warp + lane;  // this lane's element of a 128-element block of O
      if (ok && (whole || s.nt > 0)) {  // (an empty partial row's sum is 0: its elements are not read)
#pragma unroll 1
        for (int cc = 0; cc < C::kMB * 2; ++cc) {
          const int rb = 32 * (cc & 1), blk = (cc >> 1) * 128;
          if (rb >= rows) continue;
          uint32_t o[32];
          if (s.nt > 0) {
            tmem_ld32(tO + 32 * cc, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (rb + e >= rows) break;
            const float v = __uint_as_float(o[e]);
            if (whole)
              store_as(p.out, static_cast<size_t>(grow0 + rb + e) * L + blk + d,
                       f[rb + e] == 0.f ? 0.f : v * f[rb + e], p.out_dtype);
            else
              p.ws_acc[static_cast<size_t>(slot * kLatRows + rb + e) * L + blk + d] = v;
          }
        }
      }
      if (s.nt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);
        ++sg;
      }
      named_bar_sync(1, 128);  // the factors have been read
    }
    if (threadIdx.x == 0) p.ws_meta[blockIdx.x] = ok ? meta : make_int4(0, 0, 0, 0);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(tmem, C::kTmemCols);
}

template <int L, bool BF16>
cudaError_t launch_latent_t(const LatentParams& p, cudaStream_t stream) {
  using C = LatentCfg<L>;
  auto kern = ua_latent_kernel<L, BF16>;
  static std::atomic<unsigned long long> configured{0};  // one bit per device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (err != cudaSuccess) return err;
    configured.fetch_or(bit);
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(p.workers * p.cl)), dim3(C::kThreads),
                    C::kSmemBytes, stream, 1, p);
}

}  // namespace ua
