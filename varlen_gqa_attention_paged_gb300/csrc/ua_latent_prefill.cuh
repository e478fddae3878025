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
// q tile's rows are in the softmax the tensor cores work on the other's.  K tiles (48 KB at
// N = 128) have two buffers beside Q (96 KB) and V (32 KB) one: V_j arrives under Q K^T of the next
// tile.
#pragma once

#include <atomic>

#include "ua_latent.h"
#include "ua_prefill.cuh"

#include "ua.h"

namespace ua {

template <int N, int V>
struct LatentPrefillCfg {
  static constexpr int kBM = 128, kBN = 128, kNQ = 2;
  static constexpr int kCB = N / 64 + 1;           // column blocks of a key
  static constexpr int kVB = V / 64;               // and of a value
  static constexpr int kBlk = 128 * 128;           // bytes of one column block of a tile
  static constexpr int kQBytes = kCB * kBlk;       // one q tile
  static constexpr int kKBytes = kCB * kBlk;
  static constexpr int kVBytes = kVB * kBlk;
  static constexpr int kBarBytes = 512;
  static constexpr int kRoom = 227 * 1024 - 1024 - kBarBytes - kNQ * kQBytes;
  static constexpr int kRingK = 2;
  static constexpr int kRingV = (kRoom - kRingK * kKBytes) / kVBytes >= 2 ? 2 : 1;
  static constexpr int kSmemBytes =
      1024 + kBarBytes + kNQ * kQBytes + kRingK * kKBytes + kRingV * kVBytes;
  static constexpr int kTmemStride = kBN + V;      // S (and P over it), then O, of one q tile
  static constexpr int kTmemCols = 512;
  static constexpr int kThreads = 32 * (4 * kNQ + 3);
  static_assert(N % 64 == 0 && V % 64 == 0 && kNQ * kTmemStride <= kTmemCols);
  static_assert(kSmemBytes + 16 <= 227 * 1024);
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

template <int N, int V, bool BF16>
__global__ void __launch_bounds__(LatentPrefillCfg<N, V>::kThreads, 1)
    ua_latent_prefill_kernel(const __grid_constant__ LatentPrefillParams p) {
  using C = LatentPrefillCfg<N, V>;
  constexpr int BM = C::kBM, BN = C::kBN, NQ = C::kNQ, RK = C::kRingK, RV = C::kRingV;
  constexpr int TB = NQ * BM;
  constexpr int kCopyK = 4 * NQ, kCopyV = 4 * NQ + 1, kMma = 4 * NQ + 2;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sQ = smem;
  uint8_t* const sK = sQ + NQ * C::kQBytes;
  uint8_t* const sV = sK + RK * C::kKBytes;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sV + RV * C::kVBytes);
  uint64_t* const q_full = bars + 0;   // [NQ]
  uint64_t* const s_full = bars + 2;   // [NQ]
  uint64_t* const p_full = bars + 4;   // [NQ]
  uint64_t* const pv_done = bars + 6;  // [NQ]
  uint64_t* const fin = bars + 8;
  uint64_t* const k_full = bars + 9;   // [RK]
  uint64_t* const k_empty = k_full + RK;
  uint64_t* const v_full = k_empty + RK;  // [RV]
  uint64_t* const v_empty = v_full + RV;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(v_empty + RV);
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
    for (int i = 0; i < RK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < RV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kCopyK && lane == 0) {
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

  // longest walks first: slots are taken in reverse order
  const int x = static_cast<int>(gridDim.y - 1 - blockIdx.y);
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
  const int n0 = tiles(0), n1 = tiles(1);
  const int nt = max(n0, n1);

  if (warp == kCopyK) {
    // ======================================================== Q, then K tiles
    bool ok = true;
    int issued = 0;
    if (lane == 0 && nt > 0) {
      for (int qt = 0; qt < nq; ++qt) {
        mbar_arrive_expect_tx(&q_full[qt], C::kQBytes);
        for (int cb = 0; cb < C::kCB; ++cb)
          tma_load_3d_pf(sQ + qt * C::kQBytes + cb * C::kBlk, &p.q, 64 * cb, h,
                         sq.q0 + t_first + qt * BM, &q_full[qt]);
      }
    }
    for (int j = 0; ok && j < nt; ++j) {
      const int st = j % RK;
      if (j >= RK && !pf_wait_warp(&k_empty[st], ((j / RK) - 1) & 1, abort_flag, p.status)) break;
      if (lane == 0) {
        uint8_t* const dst = sK + st * C::kKBytes;
        const int row = sq.k0 + j * BN;
        mbar_arrive_expect_tx(&k_full[st], C::kKBytes);
        for (int cb = 0; cb < N / 64; ++cb)
          tma_load_3d_pf(dst + cb * C::kBlk, &p.k, 64 * cb, h, row, &k_full[st]);
        tma_load_2d(dst + (N / 64) * C::kBlk, &p.k_rope, 0, row, &k_full[st]);
      }
      __syncwarp();
      issued = j + 1;
    }
    // never leave copies in flight into this CTA's shared memory (even after an abort)
    for (int j = max(0, issued - RK); j < issued; ++j)
      mbar_wait_bounded(&k_full[j % RK], (j / RK) & 1, p.status, DEV_TIMEOUT);
    for (int qt = 0; nt > 0 && qt < nq; ++qt)
      mbar_wait_bounded(&q_full[qt], 0, p.status, DEV_TIMEOUT);
  } else if (warp == kCopyV) {
    // ======================================================== V tiles
    int issued = 0;
    for (int j = 0; j < nt; ++j) {
      const int st = j % RV;
      if (j >= RV && !pf_wait_warp(&v_empty[st], ((j / RV) - 1) & 1, abort_flag, p.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&v_full[st], C::kVBytes);
        for (int cb = 0; cb < C::kVB; ++cb)
          tma_load_3d_pf(sV + st * C::kVBytes + cb * C::kBlk, &p.v, 64 * cb, h, sq.k0 + j * BN,
                         &v_full[st]);
      }
      __syncwarp();
      issued = j + 1;
    }
    for (int j = max(0, issued - RV); j < issued; ++j)
      mbar_wait_bounded(&v_full[j % RV], (j / RV) & 1, p.status, DEV_TIMEOUT);
  } else if (warp == kMma) {
    // ======================================================== MMA issue
    // Step j: for each q tile, O += P_{j-1} V_{j-1} (which frees its S/P columns), then
    // S = Q K_j^T.  Tensor-core operations of one thread run in issue order.
    constexpr uint32_t kIdQK = umma_idesc_f16(BM, BN, BF16, false);
    constexpr uint32_t kIdPV = umma_idesc_f16(BM, V, BF16, true);
    const int qk_steps = N / 16 + p.rope_dim / 16;
    bool ok = true;
    for (int j = 0; ok && j <= nt; ++j) {
      const int i = j - 1;  // key tile of this step's P.V
      uint8_t* const vs = sV + (i >= 0 ? i % RV : 0) * C::kVBytes;
      if (i >= 0) {
        if (!pf_wait_warp(&v_full[i % RV], (i / RV) & 1, abort_flag, p.status)) { ok = false; break; }
        // rows past the sequence's keys are another's, or none's, and may hold anything (NaN
        // included): they become zeros before they meet P = 0
        const int from = k_len - i * BN;
        if (from < BN) {
          for (int e = lane; e < (BN - from) * C::kVB * 8; e += 32) {
            const int r = from + e / (C::kVB * 8), c = e % (C::kVB * 8);
            *reinterpret_cast<uint4*>(vs + (c / 8) * C::kBlk + r * 128 + (c % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (j < nt && !pf_wait_warp(&k_full[j % RK], (j / RK) & 1, abort_flag, p.status)) { ok = false; break; }
#pragma unroll
      for (int qt = 0; qt < NQ; ++qt) {
        const int n = qt == 0 ? n0 : n1;
        const uint32_t tS = tmem + qt * C::kTmemStride;
        if (i >= 0 && i < n) {
          if (!pf_wait_warp(&p_full[qt], i & 1, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint64_t bd = smem_desc_sw128(smem_addr(vs) + kk * 16 * 128, C::kBlk, 1024);
            umma_f16_ts_warp(tS + BN, tS + 8 * kk, bd, kIdPV, i > 0 || kk > 0 ? 1u : 0u);
          }
          if (i == n - 1) umma_commit_warp(&pv_done[qt]);
        }
        if (j < n) {
          if (j == 0 && !pf_wait_warp(&q_full[qt], 0, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t qb = smem_addr(sQ + qt * C::kQBytes);
          const uint32_t kb = smem_addr(sK + (j % RK) * C::kKBytes);
#pragma unroll 4
          for (int kk = 0; kk < qk_steps; ++kk) {
            const uint64_t ad = smem_desc_sw128(qb + (kk >> 2) * C::kBlk + (kk & 3) * 32, 16, 1024);
            const uint64_t bd = smem_desc_sw128(kb + (kk >> 2) * C::kBlk + (kk & 3) * 32, 16, 1024);
            umma_f16_ss_warp(tS, ad, bd, kIdQK, kk > 0 ? 1u : 0u);
          }
          umma_commit_warp(&s_full[qt]);
        }
      }
      if (!ok) break;
      if (j < nt) umma_commit_warp(&k_empty[j % RK]);
      if (i >= 0) umma_commit_warp(&v_empty[i % RV]);
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
    const uint32_t tS = tmem + qt * C::kTmemStride + ((32u * quad) << 16);
    const uint32_t tO = tS + BN;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      if (!pf_wait_warp(&s_full[qt], n & 1, abort_flag, p.status)) { ok = false; break; }
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int g = 0; g < 4; ++g) tmem_ld32(tS + 32 * g, s[g]);
      tmem_ld_wait();
      const int k0 = n * BN;
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
      // The running max moves only by more than 8 in log2 units (P stays <= 256, inside f16's
      // range and fp32 sums'), or to a row's first key.
      float alpha = 1.f;
      const bool grow = top > m + 8.f || (m == -INFINITY && top > -INFINITY);
      if (grow) {
        alpha = m == -INFINITY ? 0.f : fast_exp2(m - top);
        m = top;
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
      // P rounded to 16 bits for the MMA (half a step of 2^-8 or 2^-11 of each weight); the sum is
      // of the unrounded weights
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[qt]);
    }
    if (ok && n_tiles > 0) ok = pf_wait_warp(&pv_done[qt], 0, abort_flag, p.status);
    tc_fence_after();
    if (ok && qt < nq) {
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
}

template <int N, int V, bool BF16>
cudaError_t launch_latent_prefill_t(const LatentPrefillParams& p, cudaStream_t stream) {
  using C = LatentPrefillCfg<N, V>;
  auto kern = ua_latent_prefill_kernel<N, V, BF16>;
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
  const dim3 grid(static_cast<unsigned>(p.heads), static_cast<unsigned>(p.slots));
  return launch_pdl(kern, grid, dim3(C::kThreads), C::kSmemBytes, stream, 1, p);
}

}  // namespace ua
