// ua_latent_prefill.cuh -- latent attention, expanded form (included by ua_latent_prefill*.cu).
//
// Keys [k_nope | k_rope] and values of every head, from the up-projection of the latents; the rope
// keys are shared by the heads.  For a query row at position p of its sequence:
//   s_j = scale (q_nope . k_nope_j + q_rope . k_rope_j) for j <= p,   o = sum_j softmax(s)_j v_j
// 2 H (N + R + V) flops a visible pair: bound by the tensor cores for all but short prompts.
//
// A CTA owns two tiles of 128 query tokens of one head.  Per key tile (128 keys) and q tile:
// S = Q K^T over N / 64 + 1 column blocks of 64 (the last is the rope part, its k-steps past R left
// out), softmax with one thread a row, P (16 bits) over S in tensor memory, O += P V.  While one
// q tile's rows are in the softmax the tensor cores work on the other's.  Beside Q (96 KB at N =
// 128) there is room for eight blocks of 128 keys x 64 elements, where a key tile has three and a
// value tile two: they go through one ring in the order in which they are used up, K_0 V_0 K_1 V_1
// ..., so that what one tile frees takes the next but one.  (Barriers are a tile's: a commit costs
// the issuing warp about 200 cycles.)  (With whole tiles, two of K and one of
// V, the tensor cores waited 1800 of 4700 cycles a step for V.)
//
// Where q-blocks are few, a cluster of two or four CTAs shares the keys of each (SPLIT), and their rows
// meet through distributed shared memory.
//
// Measured (one GB300, N = V = 128, R = 64): two prompts of 8192, 16 heads, bf16 479 to 486 us in turn
// with other work, 1413 to 1436 TFLOP/s (0.75 of cuBLAS; alone, at a higher clock, 448 us; tensor cores
// busy 66 % of the time); five chunks of up to 1901 behind prefixes, 8 heads, f16 58 us (0.44: 216 CTAs
// with work on 152 SMs, the longest alone takes 45 of the mean SM's 34.5 steps); 64 tokens behind 3936,
// 16 heads 20.5 us (one CTA a q-block 54.4).
#pragma once

#include <atomic>

#include "ua_latent.h"
#include "ua_latent_tc.cuh"

#include "ua.h"

namespace ua {

template <int N, int V>
struct LatentPrefillCfg {
  static constexpr int kBM = 128, kBN = 128, kNQ = 2;
  static constexpr int kCB = N / 64 + 1;           // column blocks of a key
  static constexpr int kVB = V / 64;               // and of a value
  static constexpr int kBlk = 128 * 128;           // bytes of one column block of a tile
  static constexpr int kQBytes = kCB * kBlk;       // one q tile
  static constexpr int kPer = kCB + kVB;           // blocks of a key tile and its values
  static constexpr int kBarBytes = 256;
  static constexpr int kRoom = (227 * 1024 - 1024 - kBarBytes - kNQ * kQBytes) / kBlk;
  static constexpr int kRing = kRoom > 4 * kPer ? 4 * kPer : kRoom;
  static constexpr int kTiles = 4;                 // barriers: tiles that may be in the ring
  static constexpr int kSmemBytes = 1024 + kBarBytes + kNQ * kQBytes + kRing * kBlk;
  static constexpr int kTmemStride = kBN + V;      // S (and P over it), then O, of one q tile
  static constexpr int kTmemCols = 512;
  static constexpr int kThreads = 32 * (4 * kNQ + 2);  // softmax, copies, MMA issue
  static_assert(N % 64 == 0 && (V == 64 || V == 128) && kNQ * kTmemStride <= kTmemCols);
  static_assert(kRing >= kPer + kVB && kSmemBytes + 16 <= 227 * 1024);
  static_assert(8 * (9 + 4 * kTiles) + 4 <= kBarBytes);
  // a part's rows and their statistics, where Q and the ring were
  static constexpr int kPartBytes = kNQ * kBM * 4 * (V + 2);
  static_assert(kPartBytes <= kNQ * kQBytes + kRing * kBlk);
};

// The sequence owning slot x of q-blocks of tb tokens, by one warp: the last b with
// floor(cu_q[b] / tb) + b <= x.
struct LatentSeqOf {
  int b, q0, q_len, k0, k_len;
};
__device__ __forceinline__ LatentSeqOf latent_seq_of_slot(const int32_t* __restrict__ cq,
                                                          const int32_t* __restrict__ ck,
                                                          int num_seqs, int x, int tb) {
  const int lane = threadIdx.x & 31;
  LatentSeqOf r{0, 0, 0, 0, 0};
  for (int base = 0; base < num_seqs; base += 32) {
    const int i = base + lane;
    const bool in = i < num_seqs;
    const int q0 = in ? __ldg(cq + i) : 0, q1 = in ? __ldg(cq + i + 1) : 0;
    const int k0 = in ? __ldg(ck + i) : 0, k1 = in ? __ldg(ck + i + 1) : 0;
    const unsigned m = __ballot_sync(0xffffffffu, in && q0 / tb + i <= x);
    if (m != 0u) {
      const int src = 31 - __clz(m);
      r.b = base + src;
      r.q0 = __shfl_sync(0xffffffffu, q0, src);
      r.q_len = __shfl_sync(0xffffffffu, q1, src) - r.q0;
      r.k0 = __shfl_sync(0xffffffffu, k0, src);
      r.k_len = __shfl_sync(0xffffffffu, k1, src) - r.k0;
    }
    if (m != 0xffffffffu) break;
  }
  return r;
}

// The slot with the y-th longest walk, of up to 64, by one warp: with few q-blocks an SM has one or
// two, and those that start last must not be the longest (58.1 against 67.7 us for five chunks behind
// prefixes, whose longest sequence comes first in the batch).
__device__ __forceinline__ int latent_slot_by_length(const int32_t* __restrict__ cq,
                                                     const int32_t* __restrict__ ck, int num_seqs,
                                                     int slots, int y, int tb) {
  const int lane = threadIdx.x & 31;
  int walk[2] = {-1, -1};  // of slots lane and lane + 32 (an idle one: -1)
  for (int base = 0; base < num_seqs; base += 32) {
    const int i = base + lane;
    const bool in = i < num_seqs;
    const int q0 = in ? __ldg(cq + i) : 0, q1 = in ? __ldg(cq + i + 1) : 0;
    const int k_len = in ? __ldg(ck + i + 1) - __ldg(ck + i) : 0;
    for (int e = 0; e < min(32, num_seqs - base); ++e) {
      const int s0 = __shfl_sync(0xffffffffu, q0, e), n = __shfl_sync(0xffffffffu, q1, e) - s0;
      const int k = __shfl_sync(0xffffffffu, k_len, e), first = s0 / tb + base + e;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = (lane + 32 * u - first) * tb;  // the slot's first token in this sequence
        if (t >= 0) walk[u] = t < n ? max(0, k - n + min(t + tb, n)) : -1;  // (the last one owns it)
      }
    }
  }
  int rank[2] = {0, 0};
#pragma unroll
  for (int v = 0; v < 2; ++v)
    for (int e = 0; e < 32; ++e) {
      const int o = __shfl_sync(0xffffffffu, walk[v], e), x = e + 32 * v;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        rank[u] += x < slots && (o > walk[u] || (o == walk[u] && x < lane + 32 * u));
    }
  const unsigned a = __ballot_sync(0xffffffffu, lane < slots && rank[0] == y);
  const unsigned b = __ballot_sync(0xffffffffu, lane + 32 < slots && rank[1] == y);
  return a != 0u ? __ffs(a) - 1 : b != 0u ? __ffs(b) + 31 : y;
}

// Where a part keeps the 16-byte chunk c of its row r (a thread writes a row, a warp reads one).
template <int V>
__device__ __forceinline__ int latent_part_at(int r, int c) {
  return r * V * 4 + ((c ^ r) & (V / 4 - 1)) * 16;
}

// The rows of a q-block from the parts in the cluster's shared memory, whole rows a warp.
template <int V>
__device__ __forceinline__ void latent_prefill_join(const LatentPrefillParams& p, uint32_t rows_at,
                                                    uint32_t stats_at, int rows, int parts,
                                                    size_t token0, int h, int warp, int warps) {
  constexpr int kChunks = V / 4, kRows = 32 / kChunks;  // chunks of a row, rows of a warp at a time
  constexpr int kStat = LatentPrefillCfg<64, V>::kNQ * LatentPrefillCfg<64, V>::kBM * 4;
  const int lane = threadIdx.x & 31, c = lane % kChunks;
#pragma unroll 1
  for (int r = warp * kRows + lane / kChunks; r < rows; r += warps * kRows) {
    float m[kLatentParts], l[kLatentParts];
    float4 v[kLatentParts];
#pragma unroll
    for (int k = 0; k < kLatentParts; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.f;
      if (k < parts) {
        const uint32_t at = cluster_map(stats_at + 4 * r, k);
        m[k] = ld_cluster_f32(at);
        l[k] = ld_cluster_f32(at + kStat);
        v[k] = ld_cluster_f32x4(cluster_map(rows_at + latent_part_at<V>(r, c), k));
      }
    }
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kLatentParts; ++k) M = fmaxf(M, m[k]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kLatentParts; ++k) {
      if (k >= parts || l[k] == 0.f) continue;  // (its row may not have been written)
      const float f = fast_exp2(m[k] - M);
      sum += l[k] * f;
      o.x += v[k].x * f;
      o.y += v[k].y * f;
      o.z += v[k].z * f;
      o.w += v[k].w * f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t row = (token0 + r) * p.heads + h, at = row * V + 4 * c;
    if (p.out_dtype == UA_DT_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    } else {
      const bool bf = p.out_dtype == UA_DT_BF16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
          make_uint2(bf ? pack_bf16(o.x * inv, o.y * inv) : pack_f16(o.x * inv, o.y * inv),
                     bf ? pack_bf16(o.z * inv, o.w * inv) : pack_f16(o.z * inv, o.w * inv));
    }
    if (p.lse != nullptr && c == 0)
      p.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
}

template <int N, int V, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(LatentPrefillCfg<N, V>::kThreads, 1)
    ua_latent_prefill_kernel(const __grid_constant__ LatentPrefillParams p) {
  using C = LatentPrefillCfg<N, V>;
  constexpr int BM = C::kBM, BN = C::kBN, NQ = C::kNQ, RING = C::kRing, PER = C::kPer;
  constexpr int TB = NQ * BM;
  constexpr int kCopy = 4 * NQ, kMma = 4 * NQ + 1;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sQ = smem;
  uint8_t* const ring = sQ + NQ * C::kQBytes;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + RING * C::kBlk);
  uint64_t* const q_full = bars + 0;   // [NQ]
  uint64_t* const s_full = bars + 2;   // [NQ]
  uint64_t* const p_full = bars + 4;   // [NQ]
  uint64_t* const pv_done = bars + 6;  // [NQ]
  uint64_t* const fin = bars + 8;
  // full, empty of key tile j: [2 (j mod kTiles)] its keys, and the next, its values
  uint64_t* const full = bars + 9;
  uint64_t* const empty = full + 2 * C::kTiles;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(empty + 2 * C::kTiles);
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(fin, 1);
    for (int i = 0; i < 2 * C::kTiles; ++i) {
      mbar_init(&full[i], i % 2 == 0 ? C::kCB : C::kVB);
      mbar_init(&empty[i], 1);
    }
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kCopy && lane == 0) {
    tma_prefetch_desc(&p.q);
    tma_prefetch_desc(&p.k);
    tma_prefetch_desc(&p.k_rope);
    tma_prefetch_desc(&p.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  volatile int* abort_flag = &s_abort;
  grid_dependency_wait();
  grid_launch_dependents();

  // longest walks first: by length, or (many slots, or all at once) in reverse order
  const int slots = static_cast<int>(gridDim.y), y = static_cast<int>(blockIdx.y);
  const int x = p.by_length ? latent_slot_by_length(p.cu_seqlens_q, p.cu_seqlens_k, p.num_seqs, slots,
                                                    y, TB)
                            : slots - 1 - y;
  const LatentSeqOf sq = latent_seq_of_slot(p.cu_seqlens_q, p.cu_seqlens_k, p.num_seqs, x, TB);
  const int t_first = (x - (sq.q0 / TB + sq.b)) * TB;
  // (tokens from total_q on, and keys from total_k on, do not exist)
  const int q_end = min(sq.q_len, p.total_q - sq.q0);
  const int k_len = max(0, min(sq.k_len, p.total_k - sq.k0));
  if (sq.q0 < 0 || sq.k0 < 0 || t_first < 0 || t_first >= q_end) {  // idle slot: uniform for the CTA
    if (warp == kMma) tmem_dealloc(tmem, C::kTmemCols);
    return;
  }
  const int ctx = sq.k_len - sq.q_len;
  const int nq = min(NQ, (q_end - t_first + BM - 1) / BM);
  // key tiles of q tile qt: up to its last token's own key
  auto tiles = [&](int qt) -> int {
    if (qt >= nq) return 0;
    const int last = ctx + min(t_first + (qt + 1) * BM, q_end);  // one past it
    return (max(0, min(last, k_len)) + BN - 1) / BN;
  };
  // SPLIT: the CTA's part of them, from tile j0 on
  const int all = max(tiles(0), tiles(1));
  const int per = SPLIT ? (all + static_cast<int>(gridDim.z) - 1) / static_cast<int>(gridDim.z) : all;
  const int j0 = SPLIT ? static_cast<int>(blockIdx.z) * per : 0;
  const int n0 = max(0, min(tiles(0) - j0, per)), n1 = max(0, min(tiles(1) - j0, per));
  // the barriers of tile j's keys (v 0) or values (1), and their phase
  auto bar_of = [&](int j, int v) { return 2 * (j % C::kTiles) + v; };
  auto phase_of = [&](int j) { return (j / C::kTiles) & 1; };
  const int nt = max(n0, n1);

  if (warp == kCopy) {
    // ======================================================== Q, then the blocks of K_0 V_0 K_1 ..
    int issued = 0;
    if (lane == 0 && nt > 0) {
      for (int qt = 0; qt < nq; ++qt) {
        mbar_arrive_expect_tx(&q_full[qt], C::kQBytes);
        for (int cb = 0; cb < C::kCB; ++cb)
          tma_load_3d_pf(sQ + qt * C::kQBytes + cb * C::kBlk, &p.q, 64 * cb, h,
                         sq.q0 + t_first + qt * BM, &q_full[qt]);
      }
    }
    for (int j = 0, e = 0; j < nt; ++issued) {
      const int before = issued - RING;  // the block whose place this one takes
      if (before >= 0 &&
          !pf_wait_warp(&empty[bar_of(before / PER, before % PER >= C::kCB)], phase_of(before / PER),
                        abort_flag, p.status))
        break;
      if (lane == 0) {
        uint8_t* const dst = ring + issued % RING * C::kBlk;
        uint64_t* const bar = &full[bar_of(j, e >= C::kCB)];
        const int row = sq.k0 + (j0 + j) * BN;
        mbar_arrive_expect_tx(bar, C::kBlk);
        if (e < N / 64) tma_load_3d_pf(dst, &p.k, 64 * e, h, row, bar);
        else if (e == N / 64) tma_load_2d(dst, &p.k_rope, 0, row, bar);
        else tma_load_3d_pf(dst, &p.v, 64 * (e - C::kCB), h, row, bar);
      }
      __syncwarp();
      if (++e == PER) {
        e = 0;
        ++j;
      }
    }
    // never leave copies in flight into this CTA's shared memory (even after an abort: a tile of
    // which only some blocks were sent for never completes, and its wait gives up)
    for (int j = max(0, issued / PER - C::kTiles); j * PER < issued; ++j)
      for (int v = 0; v < 2; ++v)
        if (v == 0 || j * PER + C::kCB < issued)
          mbar_wait_bounded(&full[bar_of(j, v)], phase_of(j), p.status, DEV_TIMEOUT);
    for (int qt = 0; nt > 0 && qt < nq; ++qt)
      mbar_wait_bounded(&q_full[qt], 0, p.status, DEV_TIMEOUT);
  } else if (warp == kMma) {
    // ======================================================== MMA issue
    // Step j: for each q tile, O += P_{j-1} V_{j-1} (which frees its S/P columns), then
    // S = Q K_j^T.  Tensor-core operations of one thread run in issue order, and the order keeps
    // one q tile in the softmax while the other has the tensor cores.  Their queue is a few deep
    // only, so that what lies between two products leaves them idle: the softmax hands K_j on.
    constexpr uint32_t kIdQK = umma_idesc_f16(BM, BN, BF16, false);
    constexpr uint32_t kIdPV = umma_idesc_f16(BM, V, BF16, true);
    constexpr uint32_t kIdPVBlock = umma_idesc_f16(BM, 64, BF16, true);
    const int rope_steps = p.rope_dim / 16;
    const uint32_t ring0 = smem_units(ring), q0 = smem_units(sQ);
    bool ok = true;
    int kslot = 0;  // ring slot of K_j's first block
    for (int j = 0; ok && j <= nt; ++j) {
      const int i = j - 1;  // key tile of this step's P.V
      const int vslot = kslot >= C::kVB ? kslot - C::kVB : kslot - C::kVB + RING;  // V_i's
      if (i >= 0 && !pf_wait_warp(&full[bar_of(i, 1)], phase_of(i), abort_flag, p.status)) { ok = false; break; }
#pragma unroll
      for (int qt = 0; qt < NQ; ++qt) {
        const int n = qt == 0 ? n0 : n1;
        const bool last = qt == (n1 > 0 ? 1 : 0);  // of the q tiles that read a block
        const uint32_t tS = tmem + qt * C::kTmemStride;
        if (i >= 0 && i < n) {
          if (!pf_wait_warp(&p_full[qt], i & 1, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t vb = ring0 + vslot * (C::kBlk / 16);
          if (vslot + C::kVB <= RING) {
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              umma_f16_ts_warp(tS + BN, tS + 8 * kk, smem_desc_at(vb + kk * 128, C::kBlk), kIdPV,
                               i > 0 || kk > 0 ? 1u : 0u);
          } else {  // the blocks lie at the ring's two ends
#pragma unroll
            for (int e = 0; e < C::kVB; ++e)
#pragma unroll
              for (int kk = 0; kk < BN / 16; ++kk)
                umma_f16_ts_warp(tS + BN + 64 * e, tS + 8 * kk,
                                 smem_desc_at((e == 0 ? vb : ring0) + kk * 128, C::kBlk), kIdPVBlock,
                                 i > 0 || kk > 0 ? 1u : 0u);
          }
          if (i == n - 1) umma_commit_warp(&pv_done[qt]);
        }
        if (last && i >= 0) umma_commit_warp(&empty[bar_of(i, 1)]);
        if (j < n) {
          if ((j == 0 && !pf_wait_warp(&q_full[qt], 0, abort_flag, p.status)) ||
              ((qt == 0 || j >= n0) &&
               !pf_wait_warp(&full[bar_of(j, 0)], phase_of(j), abort_flag, p.status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t qb = q0 + qt * (C::kQBytes / 16);
#pragma unroll
          for (int e = 0; e < C::kCB; ++e) {
            const int slot = kslot + e >= RING ? kslot + e - RING : kslot + e;
            const uint32_t kb = ring0 + slot * (C::kBlk / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (e < N / 64 || kk < rope_steps)
                umma_f16_ss_at(tS, qb + e * (C::kBlk / 16) + 2 * kk, 16, kb + 2 * kk, 16, kIdQK,
                               e > 0 || kk > 0 ? 1u : 0u);
          }
          umma_commit_warp(&s_full[qt]);
        }
      }
      kslot = kslot + PER >= RING ? kslot + PER - RING : kslot + PER;
    }
    // nothing may still be in flight on the tensor cores when the memory is freed
    umma_commit_warp(fin);
    mbar_wait_bounded(fin, 0, p.status, DEV_TIMEOUT);
  } else {
    // ======================================================== softmax: a thread a row
    const int qt = warp >> 2, quad = warp & 3;
    const int n_tiles = qt == 0 ? n0 : n1;
    const int i_q = t_first + qt * BM + 32 * quad + lane;  // the row's token
    const bool rv = i_q < q_end;
    const int see = min(k_len, ctx + i_q + 1);  // keys that the row sees
    const int clear = min(k_len, ctx + t_first + qt * BM + 32 * quad + 1);  // and all of the warp's
    const float c = p.scale * kLog2e;
    constexpr float kDown = latent_down(BF16), kRoom = 8.f + kDown;
    const uint32_t tS = tmem + qt * C::kTmemStride + ((32u * quad) << 16);
    const uint32_t tO = tS + BN;
    const bool hands_on = quad == 0 && qt == (n1 > 0 ? 1 : 0);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      if (!pf_wait_warp(&s_full[qt], n & 1, abort_flag, p.status)) { ok = false; break; }
      tc_fence_after();
      // (the commit behind the last q tile's S covers both tiles' products with K_n)
      if (hands_on && lane == 0) mbar_arrive(&empty[bar_of(n, 0)]);
      uint32_t s[4][32];
#pragma unroll
      for (int g = 0; g < 4; ++g) tmem_ld32(tS + 32 * g, s[g]);
      tmem_ld_wait();
      const int k0 = (j0 + n) * BN;
      if (k0 + BN > clear) {
        const int last = see - k0;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * g + e >= last) s[g][e] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        mx[g] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          mx[g] = fmax3(mx[g], __uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
      // The reference m (the running max, in f16 kDown below it) moves only when the max is more
      // than kRoom above it, or at a row's first key.
      float alpha = 1.f;
      const bool grow = top > m + kRoom || (m == -INFINITY && top > -INFINITY);
      if (grow) {
        alpha = m == -INFINITY ? 0.f : fast_exp2(m - (top - kDown));
        m = top - kDown;
      }
      // (O holds P.V up to the tile before: the commit of this tile's S covered it)
      if (n > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
        for (int c0 = 0; c0 < V; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(tO + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st16(tO + c0, o);
        }
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const float2 cc = make_float2(c, c), mm = make_float2(-mu, -mu);
      float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
      // P rounded to 16 bits for the MMA (half a step of 2^-8 or 2^-11 of each weight, in f16 at
      // least 2^-32 of the largest); the sum is of the unrounded weights
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float2 u = __ffma2_rn(make_float2(__uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1])), cc, mm);
          float2 w = __ffma2_rn(make_float2(__uint_as_float(s[g][e + 2]), __uint_as_float(s[g][e + 3])), cc, mm);
          u = make_float2(fast_exp2(u.x), fast_exp2(u.y));
          w = make_float2(fast_exp2(w.x), fast_exp2(w.y));
          acc0 = __fadd2_rn(acc0, u);
          acc1 = __fadd2_rn(acc1, w);
          pk[e / 2] = BF16 ? pack_bf16(u.x, u.y) : pack_f16(u.x, u.y);
          pk[e / 2 + 1] = BF16 ? pack_bf16(w.x, w.y) : pack_f16(w.x, w.y);
        }
        tmem_st16(tS + 16 * g, pk);
      }
      l = l * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y));
      tmem_st_wait();
      // V rows past the sequence's keys are another's, or none's, and may hold anything (NaN
      // included): they become zeros before they meet P = 0
      const int from = k_len - k0;
      if (from < BN) {
        if (!pf_wait_warp(&full[bar_of(n, 1)], phase_of(n), abort_flag, p.status)) { ok = false; break; }
        for (int e = threadIdx.x & 127; e < (BN - from) * C::kVB * 8; e += 128) {
          const int r = from + e / (C::kVB * 8), x = e % (C::kVB * 8);
          *reinterpret_cast<uint4*>(ring + (n * PER + C::kCB + x / 8) % RING * C::kBlk + r * 128 +
                                    (x % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[qt]);
    }
    if (ok && n_tiles > 0) ok = pf_wait_warp(&pv_done[qt], 0, abort_flag, p.status);
    if constexpr (SPLIT) {
      // (Q and the ring are free when the other q tile's products are done too)
      if (ok && (qt == 0 ? n1 : n0) > 0) ok = pf_wait_warp(&pv_done[qt ^ 1], 0, abort_flag, p.status);
      tc_fence_after();
      const int r = qt * BM + 32 * quad + lane;
      float* const stats = reinterpret_cast<float*>(sQ + NQ * BM * V * 4);
      stats[r] = m;
      stats[NQ * BM + r] = ok ? l : NAN;  // (after a wait that gave up the rows are NaN)
      if (ok && n_tiles > 0) {
#pragma unroll 1
        for (int c0 = 0; c0 < V; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(sQ + latent_part_at<V>(r, c0 / 4 + e)) =
                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
    }
    tc_fence_after();
    if (!SPLIT && ok && qt < nq) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that saw no key is 0; NaN stays)
      const size_t row = (static_cast<size_t>(sq.q0) + i_q) * p.heads + h;
      if (rv && p.lse != nullptr)
        p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
#pragma unroll 1
      for (int c0 = 0; c0 < V; c0 += 32) {
        uint32_t o[32];
        if (n_tiles > 0) {
          tmem_ld32(tO + c0, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = n_tiles > 0 && inv != 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
        if (!rv) continue;
        if (p.out_dtype == UA_DT_F32) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + row * V + c0);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          const bool bf = p.out_dtype == UA_DT_BF16;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * V + c0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = __uint_as_float(o[8 * e + 2 * k]);
              const float b = __uint_as_float(o[8 * e + 2 * k + 1]);
              w[k] = bf ? pack_bf16(a, b) : pack_f16(a, b);
            }
            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(tmem, C::kTmemCols);
  if constexpr (SPLIT) {
    cluster_sync();  // every part's rows, maxima and sums are in its shared memory
    const int parts = static_cast<int>(gridDim.z);
    latent_prefill_join<V>(p, smem_addr(sQ), smem_addr(sQ) + NQ * BM * V * 4, min(TB, q_end - t_first),
                           parts, static_cast<size_t>(sq.q0) + t_first, h,
                           static_cast<int>(blockIdx.z) * (C::kThreads / 32) + warp,
                           parts * (C::kThreads / 32));
    cluster_sync_relaxed();  // no CTA leaves while another reads its shared memory
  }
}

template <int N, int V, bool BF16, bool SPLIT>
cudaError_t launch_latent_prefill_t(const LatentPrefillParams& p, cudaStream_t stream) {
  using C = LatentPrefillCfg<N, V>;
  auto kern = ua_latent_prefill_kernel<N, V, BF16, SPLIT>;
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
  const dim3 grid(static_cast<unsigned>(p.heads), static_cast<unsigned>(p.slots),
                  static_cast<unsigned>(p.parts));
  return launch_pdl_cluster(kern, grid, dim3(C::kThreads), C::kSmemBytes, stream, 1, p.parts, p);
}

template <int N, int V>
cudaError_t launch_latent_prefill_any(const LatentPrefillParams& p, bool bf16, cudaStream_t s) {
  if (p.parts > 1)
    return bf16 ? launch_latent_prefill_t<N, V, true, true>(p, s)
                : launch_latent_prefill_t<N, V, false, true>(p, s);
  return bf16 ? launch_latent_prefill_t<N, V, true, false>(p, s)
              : launch_latent_prefill_t<N, V, false, false>(p, s);
}

}  // namespace ua
