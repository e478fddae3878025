// ua_prefill.cuh -- helpers shared by the tensor-memory prefill kernels of libua.so
// (ua_prefill_tm.cuh for head_dim <= 128, ua_prefill_wide.cuh for head_dim 256).
#pragma once

#include <cuda.h>

#include "ua_device.cuh"
#include "ua_internal.h"

namespace ua {

__device__ __forceinline__ void tma_load_3d_pf(void* dst, const CUtensorMap* map, int x, int y,
                                               int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Bounded wait that also gives up at once when another warp of the CTA already did.
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                        unsigned int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, DEV_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// pf_wait for a whole warp: every lane waits, and the result is the same in every lane
// (a lane that gave up makes the warp give up), so the warp stays converged.
__device__ __forceinline__ bool pf_wait_warp(uint64_t* bar, uint32_t parity,
                                             volatile int* abort_flag, unsigned int* status) {
  return __all_sync(0xffffffffu, pf_wait(bar, parity, abort_flag, status));
}

// Sequence owning token-block slot x and its sizes, found by each warp on its own: lane i
// reads cu_seqlens_q[i], cu_seqlens_q[i + 1] and seq_lens_k[i] (32 sequences a round, the
// loads independent and coalesced), the owner is the last b with
// floor(cu[b] / tb) + b <= x (a ballot; the left side grows strictly with b), and its
// sizes reach every lane by shuffles.  One round of loads instead of the binary search's
// chain of dependent ones.
struct PfSeq {
  int b, q0, q_len, kv_len;
};
__device__ __forceinline__ PfSeq pf_seq_of_slot(const int32_t* __restrict__ cu,
                                                const int32_t* __restrict__ kvl, int num_seqs,
                                                int x, int tb) {
  const int lane = threadIdx.x & 31;
  PfSeq r{0, 0, 0, 0};
  for (int base = 0; base < num_seqs; base += 32) {
    const int i = base + lane;
    const bool in = i < num_seqs;
    const int c0 = in ? __ldg(cu + i) : 0;
    const int c1 = in ? __ldg(cu + i + 1) : 0;
    const int kv = in ? __ldg(kvl + i) : 0;
    const unsigned m = __ballot_sync(0xffffffffu, in && c0 / tb + i <= x);
    if (m != 0u) {
      const int src = 31 - __clz(m);
      r.b = base + src;
      r.q0 = __shfl_sync(0xffffffffu, c0, src);
      r.q_len = __shfl_sync(0xffffffffu, c1, src) - r.q0;
      r.kv_len = __shfl_sync(0xffffffffu, kv, src);
    }
    if (m != 0xffffffffu) break;  // the owner lies in this round
  }
  return r;
}

// Block-scaled caches (BLK 1: e4m3 codes, 2: int8).  Per key tile the dequant warps leave, for
// each of its eight 16-key groups (one block's), the K scale, log2 of the V scale and its
// reciprocal in a ring of shared memory; the softmax takes
//   x = c ks s + log2 vs,   w = 2^(x - M),   l += w / vs,   O += w (codes)
// with M the running max of x: one FMA per score as without scales, P.V on the codes, and
// weights that stay in f16's range whatever the scales are.  The weights are rounded to f16 for
// P.V (half a step of 2^-11) and summed unrounded.  Two chunks of 4096 tokens behind 4096,
// 32/8 heads, d128, e4m3: 674 us, 1222 TFLOP/s, with every unit at about half its rate (tensor
// 54 %, issue slots 50 %): what a tile waits for is a row's chain of load, exponentials and
// store in one thread, under which the CTA's other q tile runs its MMAs.
constexpr int kTileGroups = 8;
struct GroupScales {
  float kf[kTileGroups], vl[kTileGroups], vi[kTileGroups];
};

// A key group's block (-1 past ke), and a block's scales (both 1 without one, or for a bad id).
// The block is loaded two tiles ahead and the scales one, so that neither load, each of which
// needs the one before, is waited for (in one step a tile ahead a warp stood 800 cycles a tile).
__device__ __forceinline__ int key_block(const AttnParams& p, const int32_t* bt, int key, int ke) {
  if (key >= ke) return -1;
  const int col = key / p.block_size;
  return col < p.max_blocks_per_seq ? __ldg(bt + col) : -1;
}
__device__ __forceinline__ float2 block_scales(const AttnParams& p, int g, int blk) {
  if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks))
    return make_float2(1.f, 1.f);
  return make_float2(__ldg(p.k_scale_blk + blk * p.k_blk_stride[0] + g * p.k_blk_stride[1]),
                     __ldg(p.v_scale_blk + blk * p.v_blk_stride[0] + g * p.v_blk_stride[1]));
}

__device__ __forceinline__ void put_group_scales(GroupScales* dst, int grp, float2 s) {
  const float vs = block_scale(s.y);
  dst->kf[grp] = block_scale(s.x);
  dst->vl[grp] = fast_log2(vs);
  dst->vi[grp] = fast_rcp(vs);
}

// One row's part in the scores of a block-scaled cache.
struct BlkRow {
  float scale, softcap, slope;
  const float* qq_row;  // or null
  bool bias;            // ALiBi or a QQ-bias in this call
  bool valid;
  int ctx, pos, lo, ke;
};

// 32 raw scores (keys key0 .. key0 + 31, two groups of K scales kf) in place: with FEAT the
// transformed score (its K scale in it), and the mask on a boundary tile.  Each feature is a loop of
// its own behind a branch that the whole grid takes alike: a softcap alone costs two special
// function operations and 1.5 others a score (as one loop with every feature tested at each
// score it took over 30: 463 against 261 us for three chunks of up to 1501 tokens at head_dim 256).
template <bool FEAT>
__device__ __forceinline__ void blk_transform32(const BlkRow& w, float2 kf, int key0,
                                                bool need_mask, uint32_t (&r)[32]) {
  if constexpr (FEAT) {
    if (w.softcap > 0.f) {
      // sc tanh(s / sc) = sc - 2 sc / (1 + 2^(2 log2(e) s / sc))
      const float k = w.scale * 2.f * kLog2e / w.softcap;
      const float2 one = make_float2(1.f, 1.f), sc = make_float2(w.softcap, w.softcap);
      const float2 m2 = make_float2(-2.f * w.softcap, -2.f * w.softcap);
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float f = k * (e < 16 ? kf.x : kf.y);
        float2 u = __fmul2_rn(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                              make_float2(f, f));
        u = __fadd2_rn(make_float2(fast_exp2(u.x), fast_exp2(u.y)), one);
        u = __ffma2_rn(make_float2(fast_rcp(u.x), fast_rcp(u.y)), m2, sc);
        r[e] = __float_as_uint(u.x);
        r[e + 1] = __float_as_uint(u.y);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        r[e] = __float_as_uint(__uint_as_float(r[e]) * (w.scale * (e < 16 ? kf.x : kf.y)));
    }
    if (w.bias) {
      const float base = w.slope * static_cast<float>(key0 - w.ctx);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        r[e] = __float_as_uint(__uint_as_float(r[e]) + fmaf(w.slope, static_cast<float>(e), base));
      if (w.qq_row != nullptr) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int j = key0 + e;
          if (j >= w.ctx && j <= w.pos)
            r[e] = __float_as_uint(__uint_as_float(r[e]) + __ldg(w.qq_row + (j - w.ctx)));
        }
      }
    }
  }
  if (need_mask) {
    const int a = max(w.lo - key0, 0), b = min(min(w.pos, w.ke - 1) - key0, 31);
    const uint32_t live = w.valid && a <= b ? (0xffffffffu >> (31 - b)) & (0xffffffffu << a) : 0u;
#pragma unroll
    for (int e = 0; e < 32; ++e)
      r[e] = (live & (1u << e)) ? r[e] : __float_as_uint(-INFINITY);
  }
}

// The same with score features, and the larger of mx and their maximum in log2 units with the V
// scales.
__device__ __forceinline__ float blk_scores32(const BlkRow& w, const GroupScales* gs, int grp,
                                              int key0, bool need_mask, uint32_t (&r)[32],
                                              float mx) {
  const float2 kf = *reinterpret_cast<const float2*>(gs->kf + grp);
  const float2 vl = *reinterpret_cast<const float2*>(gs->vl + grp);
  blk_transform32<true>(w, kf, key0, need_mask, r);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float mg = -INFINITY;
#pragma unroll
    for (int e = 16 * q; e < 16 * q + 16; e += 2)
      mg = fmax3(mg, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
    mx = fmaxf(mx, fmaf(mg, kLog2e, q ? vl.y : vl.x));
  }
  return mx;
}

// One key tile's softmax in one pass, by a warp whose threads own whole rows (S at tS, O at tO):
// P = 2^(x - M) over S as f16 pairs, 64 keys at a time.  M stays what it was after the tiles
// before while no 16 keys' weights add up to more than 2^12 (so no maximum is taken, and every
// weight is a finite f16); where a row's do, or it sees its first keys, its sums, O and the P of
// this tile's earlier keys are brought down to the maximum of the 64 (the last rounded to f16
// once more, half a step of 2^-11: S is gone, and keys that a later one outweighs by 2^8 count
// for little).  That is rare past a row's first keys.  (Two passes, the first for the row maxima:
// 791 us for two chunks of 4096 tokens behind 4096, e4m3, 32/8 heads, d128; one pass with a
// maximum every 32 keys 771 us, as a thread's chain of load, maximum, vote and exponentials is
// what the tile waits for; this one 674 us.)  wait_pv: P.V of the tile before is done.
template <bool FEAT, int D, typename WaitPv>
__device__ __forceinline__ bool blk_softmax_tile(const BlkRow& w, const GroupScales* gs,
                                                 uint32_t tS, uint32_t tO, int k0, bool need_mask,
                                                 float c, bool have_o, float& m_used, float& l,
                                                 WaitPv wait_pv) {
  constexpr float kMostSum = 4096.f;
  float lacc = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < 16 * kTileGroups; c0 += 64) {
    uint32_t r[2][32];
    float f[4], o[4], sum[4];
    // the scores' factors and offsets of the four groups, with the present M in them
    auto factors = [&]() {
      const float4 kf = *reinterpret_cast<const float4*>(gs->kf + c0 / 16);
      const float4 vl = *reinterpret_cast<const float4*>(gs->vl + c0 / 16);
      const float m = m_used == -INFINITY ? 0.f : m_used;
      f[0] = FEAT ? c : c * kf.x, f[1] = FEAT ? c : c * kf.y;
      f[2] = FEAT ? c : c * kf.z, f[3] = FEAT ? c : c * kf.w;
      o[0] = vl.x - m, o[1] = vl.y - m, o[2] = vl.z - m, o[3] = vl.w - m;
    };
    auto scores = [&]() {
      const float4 kf = *reinterpret_cast<const float4*>(gs->kf + c0 / 16);
      blk_transform32<FEAT>(w, make_float2(kf.x, kf.y), k0 + c0, need_mask, r[0]);
      blk_transform32<FEAT>(w, make_float2(kf.z, kf.w), k0 + c0 + 32, need_mask, r[1]);
    };
    // weights as packed f16 (the first 16 registers of each half), and the groups' sums
    auto weights = [&]() {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t* const x = r[q / 2] + 16 * (q & 1);
        float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
        uint32_t hw[8];
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          float2 u = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                make_float2(f[q], f[q]), make_float2(o[q], o[q]));
          float2 v = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])),
                                make_float2(f[q], f[q]), make_float2(o[q], o[q]));
          u = make_float2(fast_exp2(u.x), fast_exp2(u.y));
          v = make_float2(fast_exp2(v.x), fast_exp2(v.y));
          a0 = __fadd2_rn(a0, u);
          a1 = __fadd2_rn(a1, v);
          hw[e / 2] = pack_f16(u.x, u.y);
          hw[e / 2 + 1] = pack_f16(v.x, v.y);
        }
        sum[q] = (a0.x + a0.y) + (a1.x + a1.y);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[q / 2][8 * (q & 1) + e] = hw[e];
      }
    };
    tmem_ld32(tS + c0, r[0]);
    tmem_ld32(tS + c0 + 32, r[1]);
    factors();
    tmem_ld_wait();
    scores();
    bool again = m_used == -INFINITY;  // the row has seen no key
    const bool fresh = __any_sync(0xffffffffu, again);
    if (!fresh) {
      weights();
      again = fmaxf(fmaxf(sum[0], sum[1]), fmaxf(sum[2], sum[3])) > kMostSum;
    }
    if (fresh || __any_sync(0xffffffffu, again)) {
      if (!fresh) {  // the scores once more: S is still there
        tmem_ld32(tS + c0, r[0]);
        tmem_ld32(tS + c0 + 32, r[1]);
        tmem_ld_wait();
        scores();
      }
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float mg = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          mg = fmax3(mg, __uint_as_float(r[q / 2][16 * (q & 1) + e]),
                     __uint_as_float(r[q / 2][16 * (q & 1) + e + 1]));
        mx = fmaxf(mx, fmaf(mg, f[q], o[q]));
      }
      // (mx is relative to M; a row past the bound on its sum lies at least 2^8 above it)
      const bool grow = mx > (m_used == -INFINITY ? -INFINITY : 8.f);
      const float alpha = !grow ? 1.f : m_used == -INFINITY ? 0.f : fast_exp2(-mx);
      if (grow) m_used = (m_used == -INFINITY ? 0.f : m_used) + mx;
      l *= alpha;
      lacc *= alpha;
      factors();
      if (have_o) {
        if (!wait_pv()) return false;
#pragma unroll 1
        for (int o0 = 0; o0 < D; o0 += 16) {
          uint32_t t[16];
          tmem_ld16(tO + o0, t);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * alpha);
          tmem_st16(tO + o0, t);
        }
      }
      tmem_st_wait();  // the P written above
#pragma unroll 1
      for (int p0 = 0; p0 < c0; p0 += 32) {
        uint32_t t[16];
        tmem_ld16(tS + p0, t);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&t[e]));
          t[e] = pack_f16(v.x * alpha, v.y * alpha);
        }
        tmem_st16(tS + p0, t);
      }
      weights();
    }
    const float4 vi = *reinterpret_cast<const float4*>(gs->vi + c0 / 16);
    lacc = fmaf(sum[0], vi.x, fmaf(sum[1], vi.y, fmaf(sum[2], vi.z, fmaf(sum[3], vi.w, lacc))));
    tmem_st16(tS + c0, *reinterpret_cast<uint32_t(*)[16]>(r[0]));
    tmem_st16(tS + c0 + 32, *reinterpret_cast<uint32_t(*)[16]>(r[1]));
  }
  l += lacc;
  tmem_st_wait();
  return true;
}

}  // namespace ua
