// ua_append.cuh -- the cache-writing kernels of libua.so (included by ua_append.cu): new
// keys and values of a batch go to their sequences' ends in the paged cache, the keys (and
// the queries beside them) rotated by position on the way.
//
// Token i of sequence b sits at cache position pos = seq_lens_k[b] - q_len + i, slot
// pos mod block_size of block block_table[b][pos / block_size].  The rotation turns the
// pairs (a, b) of a head's first rot_dim elements, frequency f of a pair taken at the
// token's position on axis axis_of[f], by the angle whose cosine and sine the caller's
// table holds:
//   a' = a cos - b sin,   b' = b cos + a sin
// in fp32 with every product and every sum rounded on its own (no fused multiply-add), so
// that what is rounded to a code afterwards is the same bit for bit in any fp32 form of the
// formula: this kernel's, a reference's, a prefill's and a decode step's.
//
// Both kernels give a lane two 16-byte chunks of a row (8 elements each) that hold both
// elements of their pairs, D / 16 lanes a row.  They move each byte once and compute little:
// bound by HBM for many tokens, by the chain of dependent loads (sequence search, block
// table, rotation table) for few.
#pragma once

#include "ua_device.cuh"
#include "ua_internal.h"

#include "ua.h"

namespace ua {

constexpr int kMaxAxes = 4;

// What a cache element is and which scale it goes by.
enum AppendKind { APP_16 = 0, APP_E4M3 = 1, APP_E4M3_TOK = 2, APP_E4M3_BLK = 3, APP_I8_BLK = 4 };

struct AppendParams {
  const uint16_t* q;  // or null
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  void* k_cache;  // [num_blocks, block_size, hkv, D]
  void* v_cache;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;
  const int32_t* block_table;
  const float* cos_sin;       // [max_position, rot_dim]: cosines, then sines; or null
  const int32_t* positions;   // [n_axes][total_q] (row stride pos_stride) or null
  const float* kv_scale;      // e4m3, per tensor
  float* k_scale;             // per token [block][slot][head] or per block [block][head]
  float* v_scale;
  long long q_stride[2], k_stride[2], v_stride[2], q_out_stride[2];  // token, head (elements)
  long long k_scale_stride[3], v_scale_stride[3];  // block, slot (per token), head
  long long pos_stride;
  unsigned int* status;
  int num_seqs, total_q, max_blocks_per_seq, num_blocks, block_size;
  int hq, hkv, rot_dim, max_position, interleaved, n_axes;
  int passes, pass_group;     // row kernel: passes of 512 / D heads a token, and those of a warp
  int slots, heads_per_cta;   // block kernel: page slots, and kv-heads of a CTA
  int slot_per_seq;           // block kernel: slot x is sequence x (one new token at most)
  uint8_t axis_of[128];
};

// The last b in [0, n) with f(b) <= x (f non-decreasing, f(0) <= x), by one warp: 32 probes a
// round, so one round of independent loads for up to 32 sequences, two for up to 1024.
template <typename F>
__device__ __forceinline__ int warp_last_le(int n, long long x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, lane * step < len && f(i) <= x);
    const int last = m == 0u ? 0 : 31 - __clz(m);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      x[2 * i] = bf16_lo(ww[i]);
      x[2 * i + 1] = bf16_hi(ww[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = BF ? pack_bf16(x[2 * i], x[2 * i + 1]) : pack_f16(x[2 * i], x[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight codes of x * inv: e4m3 (round to nearest even, saturating) or int8 (the same, within
// +-127).
template <bool I8>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (I8) {
      uint32_t r = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = fminf(fmaxf(__fmul_rn(x[4 * h + i], inv), -127.f), 127.f);
        r |= (static_cast<uint32_t>(__float2int_rn(y)) & 0xFFu) << (8 * i);
      }
      w[h] = r;
    } else {
      w[h] = f32x2_to_e4m3x2(__fmul_rn(x[4 * h], inv), __fmul_rn(x[4 * h + 1], inv)) |
             (f32x2_to_e4m3x2(__fmul_rn(x[4 * h + 2], inv), __fmul_rn(x[4 * h + 3], inv)) << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Eight codes' own values.
template <bool I8>
__device__ __forceinline__ void decode8(const uint2& w, float (&x)[8]) {
  const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (I8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * h + i] = static_cast<float>(static_cast<int8_t>(ww[h] >> (8 * i)));
    } else {
      uint32_t lo, hi;
      e4m3x4_to_f16x4(ww[h], lo, hi);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      x[4 * h] = a.x;
      x[4 * h + 1] = a.y;
      x[4 * h + 2] = b.x;
      x[4 * h + 3] = b.y;
    }
  }
}

// The two 16-byte chunks of lane c (of D / 16) of a row: a rotated pair of chunks rot / 16
// apart, or two chunks of the part that is not rotated.
template <int D>
struct LaneChunks {
  int lo, hi;
  bool turned;
  __device__ __forceinline__ LaneChunks(int c, int rot) {
    const int n = rot / 16;
    turned = c < n;
    lo = turned ? c : rot / 8 + (c - n);
    hi = lo + (turned ? n : (D - rot) / 16);
  }
};

// A lane's cosines and sines at its token's position.  Halves: its 8 frequencies, 8 lo ..;
// pairs: the 4 of chunk lo, then the 4 of chunk hi.  False: a position outside the table.
__device__ __forceinline__ bool load_turn(const AppendParams& p, int t, int pos, int lo, int hi,
                                          bool turned, float (&cs)[8], float (&sn)[8]) {
  const int half = p.rot_dim / 2;
  int pa[kMaxAxes];
  bool ok = true;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) {
    pa[a] = pos;
    if (p.positions != nullptr && a < p.n_axes) pa[a] = __ldg(p.positions + a * p.pos_stride + t);
    if (a < p.n_axes) ok = ok && pa[a] >= 0 && pa[a] < p.max_position;
  }
  if (!ok || !turned) return ok;
  const int f0 = p.interleaved ? 4 * lo : 8 * lo;
  const int f1 = p.interleaved ? 4 * hi : 8 * lo + 4;
  if (p.n_axes <= 1) {
    const float* row = p.cos_sin + static_cast<size_t>(pa[0]) * p.rot_dim;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = h ? f1 : f0;
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + f));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + f));
      cs[4 * h] = c4.x, cs[4 * h + 1] = c4.y, cs[4 * h + 2] = c4.z, cs[4 * h + 3] = c4.w;
      sn[4 * h] = s4.x, sn[4 * h + 1] = s4.y, sn[4 * h + 2] = s4.z, sn[4 * h + 3] = s4.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int f = (e < 4 ? f0 : f1) + (e & 3);
      const int a = p.axis_of[f];
      int at = pa[0];
#pragma unroll
      for (int k = 1; k < kMaxAxes; ++k) at = a == k ? pa[k] : at;
      const float* row = p.cos_sin + static_cast<size_t>(at) * p.rot_dim;
      cs[e] = __ldg(row + f);
      sn[e] = __ldg(row + half + f);
    }
  }
  return true;
}

// One pair: every product and sum rounded.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
  b = y;
}

__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float (&cs)[8],
                                     const float (&sn)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn_pair(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) turn_pair(y[2 * i], y[2 * i + 1], cs[4 + i], sn[4 + i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[i], y[i], cs[i], sn[i]);
  }
}

__device__ __forceinline__ float amax8(const float (&x)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// The scale of a group whose largest magnitude is amax: within [2^-40, 2^40], so that neither
// it nor its reciprocal leaves the normal range and a group of zeros has one too.
__device__ __forceinline__ float group_scale(float amax, float inv_qmax) {
  return fminf(fmaxf(__fmul_rn(amax, inv_qmax), kScaleMin), kScaleMax);
}

// The rows (heads) p0 .. p1 - 1 (in passes of 512 / D) of token t: queries, keys and values, or
// (ONLY_Q) queries alone.  U passes' loads are in flight before the token's sequence and
// position are known.
template <int D, bool BF, int KIND, bool ONLY_Q>
__device__ __forceinline__ void append_rows(const AppendParams& p, int t, int p0, int p1) {
  constexpr int LPR = D / 16;      // lanes a row
  constexpr int RPP = 32 / LPR;    // rows a pass
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, c = lane % LPR;
  const int hq = p.q != nullptr ? p.hq : 0;
  const int nh = ONLY_Q ? hq : hq + 2 * p.hkv;
  const LaneChunks<D> ch(c, p.rot_dim);
  bool found = false, live = false, in_cache = false, turned = false;
  size_t cache_row = 0;
  int blk = 0, slot = 0;
  float cs[8], sn[8];
#pragma unroll 1
  for (int pass = p0; pass < p1; pass += U) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (pass + u) * RPP + sub;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      if (pass + u < p1 && h < nh) {
        const uint16_t* src =
            h < hq ? p.q + t * p.q_stride[0] + h * p.q_stride[1]
            : h < hq + p.hkv ? p.k + t * p.k_stride[0] + (h - hq) * p.k_stride[1]
                             : p.v + t * p.v_stride[0] + (h - hq - p.hkv) * p.v_stride[1];
        a[u] = __ldg(reinterpret_cast<const uint4*>(src) + ch.lo);
        b[u] = __ldg(reinterpret_cast<const uint4*>(src) + ch.hi);
      }
    }
    if (!found) {
      found = true;
      const int sq = warp_last_le(p.num_seqs, t, [&](int i) -> long long {
        return __ldg(p.cu_seqlens_q + i);
      });
      const int end = __ldg(p.cu_seqlens_q + sq + 1);
      const int pos = __ldg(p.seq_lens_k + sq) - end + t;
      live = t < end && pos >= 0;
      if (live && !ONLY_Q) {
        const int col = pos / p.block_size;
        slot = pos % p.block_size;
        blk = col < p.max_blocks_per_seq
                  ? __ldg(p.block_table + static_cast<size_t>(sq) * p.max_blocks_per_seq + col)
                  : -1;
        in_cache = static_cast<unsigned>(blk) < static_cast<unsigned>(p.num_blocks);
        if (!in_cache && lane == 0) atomicOr(p.status, DEV_BAD_BLOCK);
        cache_row = (static_cast<size_t>(in_cache ? blk : 0) * p.block_size + slot) * p.hkv;
      }
      if (live && p.rot_dim > 0) {
        live = load_turn(p, t, pos, ch.lo, ch.hi, ch.turned, cs, sn);
        if (!live && lane == 0) atomicOr(p.status, DEV_BAD_POSITION);
        turned = ch.turned;
      }
      if (!live) return;  // uniform for the warp: one token
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (pass + u) * RPP + sub;
      const bool valid = pass + u < p1 && h < nh;
      float x[8], y[8];
      const bool is_v = !ONLY_Q && h >= hq + p.hkv;
      uint4 ra = a[u], rb = b[u];
      if (!is_v && turned) {
        unpack8<BF>(ra, x);
        unpack8<BF>(rb, y);
        turn(x, y, cs, sn, p.interleaved != 0);
        if (KIND == APP_16 || h < hq) {
          ra = pack8<BF>(x);
          rb = pack8<BF>(y);
        }
      } else if (KIND != APP_16) {
        unpack8<BF>(ra, x);
        unpack8<BF>(rb, y);
      }
      if (ONLY_Q || h < hq) {
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride[0] +
                                                h * p.q_out_stride[1]);
          dst[ch.lo] = ra;
          dst[ch.hi] = rb;
        }
      }
      if constexpr (!ONLY_Q) {
        const int hk = is_v ? h - hq - p.hkv : h - hq;
        const bool put = valid && in_cache && h >= hq;
        void* const cache = is_v ? p.v_cache : p.k_cache;
        if constexpr (KIND == APP_16) {
          if (put) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) +
                                                  (cache_row + hk) * D);
            dst[ch.lo] = ra;
            dst[ch.hi] = rb;
          }
        } else {
          float inv = 1.f;
          if constexpr (KIND == APP_E4M3) {
            if (put) inv = __frcp_rn(__ldg(p.kv_scale + (is_v ? 1 : 0)));
          } else {  // the row's own scale: the largest magnitude of its lanes
            float m = amax8(y, amax8(x, 0.f));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float sc = group_scale(m, 1.f / 448.f);
            inv = __frcp_rn(sc);
            if (put && c == 0) {
              const long long* st = is_v ? p.v_scale_stride : p.k_scale_stride;
              (is_v ? p.v_scale : p.k_scale)[blk * st[0] + slot * st[1] + hk * st[2]] = sc;
            }
          }
          if (put) {
            uint2* dst =
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + (cache_row + hk) * D);
            dst[ch.lo] = codes8<false>(x, inv);
            dst[ch.hi] = codes8<false>(y, inv);
          }
        }
      }
    }
  }
}

// Caches whose elements depend on their own row only: one warp takes pass_group passes of one
// token (all of them for many tokens, one for few: the launch fills the device either way).
template <int D, bool BF, int KIND>
__global__ void __launch_bounds__(128) ua_append_rows_kernel(const __grid_constant__ AppendParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int groups = (p.passes + p.pass_group - 1) / p.pass_group;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const long long t = w / groups;
  if (t >= p.total_q) return;
  const int p0 = static_cast<int>(w % groups) * p.pass_group;
  append_rows<D, BF, KIND, false>(p, static_cast<int>(t), p0, min(p0 + p.pass_group, p.passes));
}

// Block-scaled caches.  CTA x < slots * (hkv / heads_per_cta) owns one page that new tokens
// of a sequence reach, for heads_per_cta kv-heads; the CTAs behind them rotate the queries.
// A thread holds one chunk pair of one of the page's rows (slots): a row of a new token is
// read and rotated, a row that held a token before is read as codes.  Per head and operand
//   s = the larger of (largest new magnitude) / qmax and, with tokens held, the old scale;
// new rows are stored as rne(x / s), and rows held before as rne(code * (old / s)) where s
// grew (else they stay).  Slot layout: sequence b's pages start at floor(cu[b] / bs) + 2 b
// (n new tokens reach at most floor(n / bs) + 2 pages).
template <int D, bool BF, bool I8, bool ONE>
__global__ void __launch_bounds__(512) ua_append_blk_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 16;
  constexpr float kInvQ = 1.f / (I8 ? 127.f : 448.f);
  __shared__ float red[2][2][16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int hgroups = (p.hkv + p.heads_per_cta - 1) / p.heads_per_cta;
  const long long cta = blockIdx.x;
  if (cta >= static_cast<long long>(p.slots) * hgroups) {  // the queries
    const int groups = (p.passes + p.pass_group - 1) / p.pass_group;
    const long long w = (cta - static_cast<long long>(p.slots) * hgroups) * warps + warp;
    const long long t = w / groups;
    if (t >= p.total_q) return;
    const int p0 = static_cast<int>(w % groups) * p.pass_group;
    append_rows<D, BF, APP_16, true>(p, static_cast<int>(t), p0,
                                     min(p0 + p.pass_group, p.passes));
    return;
  }
  const int x = static_cast<int>(cta / hgroups);
  const int h0 = static_cast<int>(cta % hgroups) * p.heads_per_cta;
  const int h1 = min(h0 + p.heads_per_cta, p.hkv);
  const int bs = p.block_size;
  const int b = p.slot_per_seq ? x : warp_last_le(p.num_seqs, x, [&](int i) -> long long {
    return __ldg(p.cu_seqlens_q + i) / bs + 2LL * i;
  });
  const int q0 = __ldg(p.cu_seqlens_q + b);
  const int q_len = __ldg(p.cu_seqlens_q + b + 1) - q0;
  const int kv_len = __ldg(p.seq_lens_k + b);
  const int ctx = kv_len - q_len;
  const int seg = p.slot_per_seq ? 0 : x - (q0 / bs + 2 * b);
  if (p.slot_per_seq && q_len > 1 && h0 == 0 && threadIdx.x == 0)
    atomicOr(p.status, DEV_BAD_SHAPE);  // q_len above max_seqlen_q
  if (q_len <= 0 || seg < 0) return;
  const int pg = max(ctx, 0) / bs + seg;
  if (static_cast<long long>(pg) * bs >= kv_len) return;  // idle slot
  const int base = pg * bs;
  const int s0 = max(ctx - base, 0);           // tokens the page held before
  const int s1 = min(kv_len - base, bs);       // its slots in use now
  const int blk = pg < p.max_blocks_per_seq
                      ? __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks_per_seq + pg)
                      : -1;
  if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
    if (threadIdx.x == 0) atomicOr(p.status, DEV_BAD_BLOCK);
    return;
  }
  const int row0 = threadIdx.x / LPR, rows = blockDim.x / LPR;
  const LaneChunks<D> ch(threadIdx.x % LPR, p.rot_dim);
  float cs[8], sn[8];
  // one of the page's rows: 0 outside the page's slots in use, 1 held before, 2 new
  auto state = [&](int r) -> int {
    if (r >= s1) return 0;
    if (r < s0) return 1;
    if (p.rot_dim == 0) return 2;
    if (load_turn(p, q0 + base + r - ctx, base + r, ch.lo, ch.hi, ch.turned, cs, sn)) return 2;
    atomicOr(p.status, DEV_BAD_POSITION);
    return 0;
  };
  const int st0 = ONE ? state(row0) : 0;
  for (int h = h0; h < h1; ++h) {
    float kx[8], ky[8], vx[8], vy[8];
    uint2 ok0, ok1, ov0, ov1;
    uint8_t *kp = nullptr, *vp = nullptr;
    const float old_k = p.k_scale[blk * p.k_scale_stride[0] + h * p.k_scale_stride[2]];
    const float old_v = p.v_scale[blk * p.v_scale_stride[0] + h * p.v_scale_stride[2]];
    // a row's data: new elements rotated, or the codes held
    auto fetch = [&](int r, int st) {
      const size_t off = ((static_cast<size_t>(blk) * bs + r) * p.hkv + h) * D;
      kp = static_cast<uint8_t*>(p.k_cache) + off;
      vp = static_cast<uint8_t*>(p.v_cache) + off;
      if (st == 2) {
        const long long t = q0 + base + r - ctx;
        const uint4* ks = reinterpret_cast<const uint4*>(p.k + t * p.k_stride[0] + h * p.k_stride[1]);
        const uint4* vs = reinterpret_cast<const uint4*>(p.v + t * p.v_stride[0] + h * p.v_stride[1]);
        const uint4 k0 = __ldg(ks + ch.lo), k1 = __ldg(ks + ch.hi);
        const uint4 v0 = __ldg(vs + ch.lo), v1 = __ldg(vs + ch.hi);
        unpack8<BF>(k0, kx);
        unpack8<BF>(k1, ky);
        unpack8<BF>(v0, vx);
        unpack8<BF>(v1, vy);
        if (ch.turned) turn(kx, ky, cs, sn, p.interleaved != 0);
      } else if (st == 1) {
        ok0 = reinterpret_cast<const uint2*>(kp)[ch.lo];
        ok1 = reinterpret_cast<const uint2*>(kp)[ch.hi];
        ov0 = reinterpret_cast<const uint2*>(vp)[ch.lo];
        ov1 = reinterpret_cast<const uint2*>(vp)[ch.hi];
      }
    };
    float mk = 0.f, mv = 0.f;
    for (int r = row0; r < bs; r += rows) {
      const int st = ONE ? st0 : state(r);
      if (ONE || st == 2) fetch(r, st);
      if (st == 2) {
        mk = amax8(ky, amax8(kx, mk));
        mv = amax8(vy, amax8(vx, mv));
      }
      if (ONE) break;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    float (&rd)[2][16] = red[h & 1];
    if (lane == 0) {
      rd[0][warp] = mk;
      rd[1][warp] = mv;
    }
    __syncthreads();
    mk = lane < warps ? rd[0][lane] : 0.f;
    mv = lane < warps ? rd[1][lane] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    mk = __shfl_sync(0xffffffffu, mk, 0);
    mv = __shfl_sync(0xffffffffu, mv, 0);
    float sk = group_scale(mk, kInvQ), sv = group_scale(mv, kInvQ);
    const float hk = fminf(fmaxf(old_k, kScaleMin), kScaleMax);
    const float hv = fminf(fmaxf(old_v, kScaleMin), kScaleMax);
    if (s0 > 0) {
      sk = fmaxf(sk, hk);
      sv = fmaxf(sv, hv);
    }
    const float ik = __frcp_rn(sk), iv = __frcp_rn(sv);
    for (int r = row0; r < bs; r += rows) {
      const int st = ONE ? st0 : state(r);
      const bool again_k = st == 1 && sk > hk, again_v = st == 1 && sv > hv;
      if (!ONE && (st == 2 || again_k || again_v)) fetch(r, st);
      if (st == 2) {
        reinterpret_cast<uint2*>(kp)[ch.lo] = codes8<I8>(kx, ik);
        reinterpret_cast<uint2*>(kp)[ch.hi] = codes8<I8>(ky, ik);
        reinterpret_cast<uint2*>(vp)[ch.lo] = codes8<I8>(vx, iv);
        reinterpret_cast<uint2*>(vp)[ch.hi] = codes8<I8>(vy, iv);
      }
      if (again_k) {
        const float ratio = __fdiv_rn(hk, sk);
        decode8<I8>(ok0, kx);
        decode8<I8>(ok1, ky);
        reinterpret_cast<uint2*>(kp)[ch.lo] = codes8<I8>(kx, ratio);
        reinterpret_cast<uint2*>(kp)[ch.hi] = codes8<I8>(ky, ratio);
      }
      if (again_v) {
        const float ratio = __fdiv_rn(hv, sv);
        decode8<I8>(ov0, vx);
        decode8<I8>(ov1, vy);
        reinterpret_cast<uint2*>(vp)[ch.lo] = codes8<I8>(vx, ratio);
        reinterpret_cast<uint2*>(vp)[ch.hi] = codes8<I8>(vy, ratio);
      }
      if (ONE) break;
    }
    // every thread read the old scales before the barrier above
    if (threadIdx.x == 0) {
      p.k_scale[blk * p.k_scale_stride[0] + h * p.k_scale_stride[2]] = sk;
      p.v_scale[blk * p.v_scale_stride[0] + h * p.v_scale_stride[2]] = sv;
    }
  }
}

}  // namespace ua
