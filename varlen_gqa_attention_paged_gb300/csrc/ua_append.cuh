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
  uint8_t axis4[32];          // the axis of frequencies 4 i .. 4 i + 3, or 255: not one
};

// The sequence owning x and its sizes: the last b in [0, n) with f(cu[b], b) <= x (f
// non-decreasing, f(cu[0], 0) <= x), by one warp.  32 probes a round narrow it to 32
// sequences, whose sizes all load in the last round (the only one for up to 32 sequences), so
// that no load waits for the choice.
struct SeqOf {
  int b, q0, end, kv_len;
};
template <typename F>
__device__ __forceinline__ SeqOf seq_of(const int32_t* __restrict__ cu,
                                        const int32_t* __restrict__ kvl, int n, long long x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 32) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, lane * step < len && f(__ldg(cu + i), i) <= x);
    const int last = m == 0u ? 0 : 31 - __clz(m);
    lo += last * step;
    len = min(step, len - last * step);
  }
  const int i = lo + min(lane, len - 1);
  const int c0 = __ldg(cu + i), c1 = __ldg(cu + i + 1), kv = __ldg(kvl + i);
  const unsigned m = __ballot_sync(0xffffffffu, lane < len && f(c0, i) <= x);
  const int src = m == 0u ? 0 : 31 - __clz(m);
  return SeqOf{lo + src, __shfl_sync(0xffffffffu, c0, src), __shfl_sync(0xffffffffu, c1, src),
               __shfl_sync(0xffffffffu, kv, src)};
}

// A lane's 16 elements as fp32, first and second elements of its pairs apart: with halves
// apart (and wherever nothing turns) word j of the first chunk is (a[2j], a[2j + 1]) and of the
// second (b[2j], b[2j + 1]); interleaved, word j of the two chunks' eight is (a[j], b[j]).
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF) return make_float2(bf16_lo(w), bf16_hi(w));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return BF ? pack_bf16(x, y) : pack_f16(x, y);
}

template <bool BF>
__device__ __forceinline__ void unpack16(const uint4& lo, const uint4& hi, bool interleaved,
                                         float (&a)[8], float (&b)[8]) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = unpack2<BF>(w[j]);
      a[j] = f.x;
      b[j] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<BF>(w[j]), g = unpack2<BF>(w[4 + j]);
      a[2 * j] = f.x, a[2 * j + 1] = f.y;
      b[2 * j] = g.x, b[2 * j + 1] = g.y;
    }
  }
}

template <bool BF>
__device__ __forceinline__ void pack16(const float (&a)[8], const float (&b)[8], bool interleaved,
                                       uint4& lo, uint4& hi) {
  uint32_t w[8];
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack2<BF>(a[j], b[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = pack2<BF>(a[2 * j], a[2 * j + 1]);
      w[4 + j] = pack2<BF>(b[2 * j], b[2 * j + 1]);
    }
  }
  lo = make_uint4(w[0], w[1], w[2], w[3]);
  hi = make_uint4(w[4], w[5], w[6], w[7]);
}

// The largest magnitude of 16 packed elements, exactly, without unpacking them.
template <bool BF>
__device__ __forceinline__ float amax_packed(const uint4& lo, const uint4& hi) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if constexpr (BF) {
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
    for (int j = 1; j < 8; ++j)
      m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    __half2 m = __habs2(*reinterpret_cast<const __half2*>(&w[0]));
#pragma unroll
    for (int j = 1; j < 8; ++j)
      m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&w[j])));
    return fmaxf(__low2float(m), __high2float(m));
  }
}

__device__ __forceinline__ float amax16(const float (&a)[8], const float (&b)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmax3(m, fabsf(a[i]), fabsf(b[i]));
  return m;
}

// Two products, each rounded.  What is added to them afterwards goes through __fadd_rn and
// __fsub_rn: a packed sum would be contracted with the packed products into one rounding
// (seen with add.rn.f32x2 too), and the codes would not be reproducible.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// Four codes of x (already divided by the scale): e4m3 (round to nearest even, saturating) or
// int8 (the same).  An int8 value plus 1.5 * 2^23 is rounded to a whole number whose low byte
// is the code; `wide` says that it may lie outside +-127 (a scale at the end of its range).
template <bool I8>
__device__ __forceinline__ uint32_t codes4(float2 x, float2 y, bool wide) {
  if constexpr (I8) {
    if (wide) {
      x = make_float2(fminf(fmaxf(x.x, -127.f), 127.f), fminf(fmaxf(x.y, -127.f), 127.f));
      y = make_float2(fminf(fmaxf(y.x, -127.f), 127.f), fminf(fmaxf(y.y, -127.f), 127.f));
    }
    constexpr float magic = 12582912.f;
    const uint32_t u0 = __float_as_uint(__fadd_rn(x.x, magic));
    const uint32_t u1 = __float_as_uint(__fadd_rn(x.y, magic));
    const uint32_t u2 = __float_as_uint(__fadd_rn(y.x, magic));
    const uint32_t u3 = __float_as_uint(__fadd_rn(y.y, magic));
    return __byte_perm(__byte_perm(u0, u1, 0x0040), __byte_perm(u2, u3, 0x0040), 0x5410);
  } else {
    return f32x2_to_e4m3x2(x.x, x.y) | (f32x2_to_e4m3x2(y.x, y.y) << 16);
  }
}

// The lane's 16 codes of (a, b) * mul, each product rounded.
template <bool I8>
__device__ __forceinline__ void codes16(const float (&a)[8], const float (&b)[8], float mul,
                                        bool interleaved, bool wide, uint2& lo, uint2& hi) {
  const float2 m = make_float2(mul, mul);
  float2 x[4], y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = mul2(make_float2(a[2 * j], a[2 * j + 1]), m);
    y[j] = mul2(make_float2(b[2 * j], b[2 * j + 1]), m);
  }
  uint32_t w[4];
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = codes4<I8>(make_float2(x[j].x, y[j].x), make_float2(x[j].y, y[j].y), wide);
  } else {
    w[0] = codes4<I8>(x[0], x[1], wide);
    w[1] = codes4<I8>(x[2], x[3], wide);
    w[2] = codes4<I8>(y[0], y[1], wide);
    w[3] = codes4<I8>(y[2], y[3], wide);
  }
  lo = make_uint2(w[0], w[1]);
  hi = make_uint2(w[2], w[3]);
}

// Eight codes' own values.
template <bool I8>
__device__ __forceinline__ void decode8(const uint2& w, float (&x)[8]) {
  const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t lo, hi;
    codes4_to_f16x4<I8>(ww[h], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[4 * h] = a.x, x[4 * h + 1] = a.y;
    x[4 * h + 2] = b.x, x[4 * h + 3] = b.y;
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
    auto row_of = [&](int a) -> const float* {
      int at = pa[0];
#pragma unroll
      for (int k = 1; k < kMaxAxes; ++k) at = a == k ? pa[k] : at;
      return p.cos_sin + static_cast<size_t>(at) * p.rot_dim;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = h ? f1 : f0, a = p.axis4[f / 4];
      if (a != 255) {
        const float* row = row_of(a);
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + f));
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + half + f));
        cs[4 * h] = c4.x, cs[4 * h + 1] = c4.y, cs[4 * h + 2] = c4.z, cs[4 * h + 3] = c4.w;
        sn[4 * h] = s4.x, sn[4 * h + 1] = s4.y, sn[4 * h + 2] = s4.z, sn[4 * h + 3] = s4.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float* row = row_of(p.axis_of[f + e]);
          cs[4 * h + e] = __ldg(row + f + e);
          sn[4 * h + e] = __ldg(row + half + f + e);
        }
      }
    }
  }
  return true;
}

// Eight pairs, two at a time: every product and every sum rounded.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                     const float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x = make_float2(a[i], a[i + 1]), y = make_float2(b[i], b[i + 1]);
    const float2 c = make_float2(cs[i], cs[i + 1]), s = make_float2(sn[i], sn[i + 1]);
    const float2 xc = mul2(x, c), ys = mul2(y, s), yc = mul2(y, c), xs = mul2(x, s);
    a[i] = __fsub_rn(xc.x, ys.x), a[i + 1] = __fsub_rn(xc.y, ys.y);
    b[i] = __fadd_rn(yc.x, xs.x), b[i + 1] = __fadd_rn(yc.y, xs.y);
  }
}

// The scale of a group whose largest magnitude is amax: within [2^-40, 2^40], so that neither
// it nor its reciprocal leaves the normal range and a group of zeros has one too.
__device__ __forceinline__ float group_scale(float amax, float inv_qmax) {
  return fminf(fmaxf(__fmul_rn(amax, inv_qmax), kScaleMin), kScaleMax);
}

// Where a token's keys and values go, and its turn.
struct TokenAt {
  size_t cache_row;  // row of kv-head 0 in the cache
  int blk, slot;
  bool in_cache, turned;
  float cs[8], sn[8];
};

// U passes (rows h, h + 512 / D, ... of q, k or v: R 0, 1, 2) of one token as read in a and b;
// n of them are real.
template <int D, bool BF, int KIND, int R, int U>
__device__ __forceinline__ void put_rows(const AppendParams& p, const TokenAt& at, int t, int h0,
                                         int n, int c, const LaneChunks<D>& ch, uint4 (&a)[U],
                                         uint4 (&b)[U]) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;
  const int heads = R == 0 ? p.hq : p.hkv;
  const bool inter = p.interleaved != 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * RPP;
    const bool valid = u < n && h < heads;
    float x[8], y[8];
    bool open = false;  // the row is in x and y
    if (R != 2 && at.turned) {
      unpack16<BF>(a[u], b[u], inter, x, y);
      turn(x, y, at.cs, at.sn);
      if (R == 0 || KIND == APP_16) pack16<BF>(x, y, inter, a[u], b[u]);
      open = true;
    }
    if (R == 0) {
      if (valid) {
        uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride[0] +
                                              h * p.q_out_stride[1]);
        dst[ch.lo] = a[u];
        dst[ch.hi] = b[u];
      }
      continue;
    }
    const bool put = valid && at.in_cache;
    void* const cache = R == 2 ? p.v_cache : p.k_cache;
    if constexpr (KIND == APP_16) {
      if (put) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) +
                                              (at.cache_row + h) * D);
        dst[ch.lo] = a[u];
        dst[ch.hi] = b[u];
      }
    } else {
      float inv;
      if constexpr (KIND == APP_E4M3) {
        inv = __frcp_rn(__ldg(p.kv_scale + (R == 2 ? 1 : 0)));
      } else {  // the row's own scale: the largest magnitude of its lanes
        float m = R != 2 && open ? amax16(x, y) : amax_packed<BF>(a[u], b[u]);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = group_scale(m, 1.f / 448.f);
        inv = __frcp_rn(sc);
        if (put && c == 0) {
          const long long* st = R == 2 ? p.v_scale_stride : p.k_scale_stride;
          (R == 2 ? p.v_scale : p.k_scale)[at.blk * st[0] + at.slot * st[1] + h * st[2]] = sc;
        }
      }
      if (!open) unpack16<BF>(a[u], b[u], false, x, y);
      uint2 lo, hi;
      codes16<false>(x, y, inv, R != 2 && open && inter, false, lo, hi);
      if (put) {
        uint2* dst =
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + (at.cache_row + h) * D);
        dst[ch.lo] = lo;
        dst[ch.hi] = hi;
      }
    }
  }
}

// Passes p0 .. p1 - 1 of token t, by one warp: 512 / D rows a pass, the queries' passes first,
// then (not ONLY_Q) the keys' and the values'.  U passes load together, and the first loads are
// on their way before the token's sequence, place and angles are known.
template <int D, bool BF, int KIND, bool ONLY_Q, int U>
__device__ __forceinline__ void append_rows(const AppendParams& p, int t, int p0, int p1) {
  constexpr int LPR = D / 16;      // lanes a row
  constexpr int RPP = 32 / LPR;    // rows a pass
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, c = lane % LPR;
  const int nq = (p.hq + RPP - 1) / RPP, nk = (p.hkv + RPP - 1) / RPP;
  const LaneChunks<D> ch(c, p.rot_dim);
  TokenAt at;
  at.in_cache = at.turned = false;
  bool found = false;
#pragma unroll 1
  for (int pass = p0; pass < p1;) {
    // the pass's tensor, and how many more passes of it (at most U) come next
    const int r = ONLY_Q || pass < nq ? 0 : pass < nq + nk ? 1 : 2;
    const int first = r == 0 ? 0 : r == 1 ? nq : nq + nk;
    const int n = min(U, min(p1, r == 0 ? nq : first + nk) - pass);
    const int heads = r == 0 ? p.hq : p.hkv;
    const int h0 = (pass - first) * RPP + sub;
    const uint16_t* const src = r == 0   ? p.q + t * p.q_stride[0]
                                : r == 1 ? p.k + t * p.k_stride[0]
                                         : p.v + t * p.v_stride[0];
    const long long hs = r == 0 ? p.q_stride[1] : r == 1 ? p.k_stride[1] : p.v_stride[1];
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * RPP;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      if (u < n && h < heads) {
        const uint4* row = reinterpret_cast<const uint4*>(src + h * hs);
        a[u] = __ldg(row + ch.lo);
        b[u] = __ldg(row + ch.hi);
      }
    }
    if (!found) {
      found = true;
      const SeqOf sq = seq_of(p.cu_seqlens_q, p.seq_lens_k, p.num_seqs, t,
                              [](int c0, int) -> long long { return c0; });
      const int pos = sq.kv_len - sq.end + t;
      if (t >= sq.end || pos < 0) return;  // uniform for the warp: one token
      if (!ONLY_Q) {
        const int col = pos / p.block_size;
        at.slot = pos % p.block_size;
        at.blk = col < p.max_blocks_per_seq
                     ? __ldg(p.block_table + static_cast<size_t>(sq.b) * p.max_blocks_per_seq + col)
                     : -1;
      }
      if (p.rot_dim > 0) {
        if (!load_turn(p, t, pos, ch.lo, ch.hi, ch.turned, at.cs, at.sn)) {
          if (lane == 0) atomicOr(p.status, DEV_BAD_POSITION);
          return;
        }
        at.turned = ch.turned;
      }
      if (!ONLY_Q) {
        at.in_cache = static_cast<unsigned>(at.blk) < static_cast<unsigned>(p.num_blocks);
        if (!at.in_cache && lane == 0) atomicOr(p.status, DEV_BAD_BLOCK);
        at.cache_row =
            (static_cast<size_t>(at.in_cache ? at.blk : 0) * p.block_size + at.slot) * p.hkv;
      }
    }
    if (r == 0) {
      put_rows<D, BF, KIND, 0, U>(p, at, t, h0, n, c, ch, a, b);
    } else if constexpr (!ONLY_Q) {
      if (r == 1) put_rows<D, BF, KIND, 1, U>(p, at, t, h0, n, c, ch, a, b);
      else put_rows<D, BF, KIND, 2, U>(p, at, t, h0, n, c, ch, a, b);
    }
    pass += n;
  }
}

// Caches whose elements depend on their own row only: one warp takes pass_group passes of one
// token.  Bound by HBM: two passes' loads a warp (64 bytes a lane) and six CTAs, 24 warps, an
// SM keep 48 KB in flight (four passes and 16 warps: 67.0 against 64.5 us for 4 prompts of
// 4096 tokens, 76.7 against 67.4 us for 16384 video tokens into e4m3 with token scales).
constexpr int kRowsMinBlocks = 6, kRowsPasses = 2;
template <int D, bool BF, int KIND>
__global__ void __launch_bounds__(128, kRowsMinBlocks)
    ua_append_rows_kernel(const __grid_constant__ AppendParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int groups = (p.passes + p.pass_group - 1) / p.pass_group;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const long long t = w / groups;
  if (t >= p.total_q) return;
  const int p0 = static_cast<int>(w % groups) * p.pass_group;
  append_rows<D, BF, KIND, false, kRowsPasses>(p, static_cast<int>(t), p0,
                                               min(p0 + p.pass_group, p.passes));
}

// Block-scaled caches.  CTA x < slots * (hkv / heads_per_cta) owns one page that new tokens
// of a sequence reach, for heads_per_cta kv-heads; the CTAs behind them rotate the queries.
// A thread holds one chunk pair of one of the page's rows (slots): a row of a new token is
// read and rotated, a row that held a token before is read as codes.  Per head and operand
//   s = the larger of (largest new magnitude) / qmax and, with tokens held, the old scale;
// new rows are stored as rne(x / s), and rows held before as rne(code * (old / s)) where s
// grew (else they stay).  Slot layout: sequence b's pages start at floor(cu[b] / bs) + 2 b
// (n new tokens reach at most floor(n / bs) + 2 pages).  ONE: the page's rows fit the CTA's
// threads once, and a row stays in registers between its two uses; else (more than 32 slots at
// head_dim 128, 16 at 256) it is read twice, and its angles are looked up for every head and use:
// 41.7 us at pages of 64 against 36.1 at 32 for chunks of up to 1999 tokens (int8, d128), 74.8 at
// 32 against 66.1 at 16 at d256, and 6.4 at 64 against 3.7 at 16 for the newest tokens of 64
// sequences (e4m3, d128).
// MINB CTAs an SM: four (64 registers a thread, a few spilled) where the grid fills them, as
// the latency of a page's chain of loads is what many pages are bound by (36.3 against 40.8
// us for chunks of up to 1999 tokens, int8); three where it does not (3.7 against 4.3 us for
// a decode step of 64 sequences).
constexpr int kBlkThreads = 256;
template <int D, bool BF, bool I8, bool ONE, int MINB>
__global__ void __launch_bounds__(kBlkThreads, MINB)
    ua_append_blk_kernel(const __grid_constant__ AppendParams p) {
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
    append_rows<D, BF, APP_16, true, kRowsPasses>(p, static_cast<int>(t), p0,
                                             min(p0 + p.pass_group, p.passes));
    return;
  }
  const int x = static_cast<int>(cta / hgroups);
  const int h0 = static_cast<int>(cta % hgroups) * p.heads_per_cta;
  const int h1 = min(h0 + p.heads_per_cta, p.hkv);
  const int bs = p.block_size;
  SeqOf sq;
  if (p.slot_per_seq)
    sq = SeqOf{x, __ldg(p.cu_seqlens_q + x), __ldg(p.cu_seqlens_q + x + 1),
               __ldg(p.seq_lens_k + x)};
  else
    sq = seq_of(p.cu_seqlens_q, p.seq_lens_k, p.num_seqs, x,
                [bs](int c0, int i) -> long long { return c0 / bs + 2LL * i; });
  const int q_len = sq.end - sq.q0;
  const int ctx = sq.kv_len - q_len;
  const int seg = p.slot_per_seq ? 0 : x - (sq.q0 / bs + 2 * sq.b);
  if (p.slot_per_seq && q_len > 1 && h0 == 0 && threadIdx.x == 0)
    atomicOr(p.status, DEV_BAD_SHAPE);  // q_len above max_seqlen_q
  if (q_len <= 0 || seg < 0) return;
  const int pg = max(ctx, 0) / bs + seg;
  if (static_cast<long long>(pg) * bs >= sq.kv_len) return;  // idle slot
  const int base = pg * bs;
  const int t0 = sq.q0 + base - ctx;         // token of the page's slot 0
  const int s0 = max(ctx - base, 0);        // tokens the page held before
  // its slots in use now (never a token past the inputs, should cu_seqlens_q end behind them)
  const int s1 = min(min(sq.kv_len - base, bs), p.total_q - t0);
  if (s1 <= s0) return;
  const int row0 = threadIdx.x / LPR, rows = blockDim.x / LPR;
  const LaneChunks<D> ch(threadIdx.x % LPR, p.rot_dim);
  uint4 k0, k1, v0, v1;  // a new row's chunks as read; codes held before in .x, .y
  auto fetch_new = [&](int r, int h) {
    const long long t = t0 + r;
    const uint4* ks = reinterpret_cast<const uint4*>(p.k + t * p.k_stride[0] + h * p.k_stride[1]);
    const uint4* vs = reinterpret_cast<const uint4*>(p.v + t * p.v_stride[0] + h * p.v_stride[1]);
    k0 = __ldg(ks + ch.lo), k1 = __ldg(ks + ch.hi);
    v0 = __ldg(vs + ch.lo), v1 = __ldg(vs + ch.hi);
  };
  // the first head's new rows start on their way before the page and the angles are known
  if (ONE && row0 >= s0 && row0 < s1) fetch_new(row0, h0);
  const int blk = pg < p.max_blocks_per_seq
                      ? __ldg(p.block_table + static_cast<size_t>(sq.b) * p.max_blocks_per_seq + pg)
                      : -1;
  float cs[8], sn[8];
  // one of the page's rows: 0 outside the page's slots in use, 1 held before, 2 new
  auto state = [&](int r) -> int {
    if (r >= s1) return 0;
    if (r < s0) return 1;
    if (p.rot_dim == 0) return 2;
    if (load_turn(p, t0 + r, base + r, ch.lo, ch.hi, ch.turned, cs, sn)) return 2;
    atomicOr(p.status, DEV_BAD_POSITION);
    return 0;
  };
  const int st0 = ONE ? state(row0) : 0;
  if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
    if (threadIdx.x == 0) atomicOr(p.status, DEV_BAD_BLOCK);
    return;
  }
  auto cache_row = [&](void* cache, int r, int h) -> uint2* {
    return reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) +
                                    ((static_cast<size_t>(blk) * bs + r) * p.hkv + h) * D);
  };
  auto fetch_held = [&](int r, int h) {
    const uint2* kp = cache_row(p.k_cache, r, h);
    const uint2* vp = cache_row(p.v_cache, r, h);
    const uint2 a = kp[ch.lo], b = kp[ch.hi], c = vp[ch.lo], d = vp[ch.hi];
    k0.x = a.x, k0.y = a.y, k1.x = b.x, k1.y = b.y;
    v0.x = c.x, v0.y = c.y, v1.x = d.x, v1.y = d.y;
  };
  const bool inter = p.interleaved != 0;
  float xs[8], ys[8];
  auto new_k = [&]() {
    unpack16<BF>(k0, k1, inter && ch.turned, xs, ys);
    if (ch.turned) turn(xs, ys, cs, sn);
  };
  auto put = [&](uint2* dst, float mul, bool pairs, bool wide) {
    uint2 lo, hi;
    codes16<I8>(xs, ys, mul, pairs, wide, lo, hi);
    dst[ch.lo] = lo;
    dst[ch.hi] = hi;
  };
  for (int h = h0; h < h1; ++h) {
    const float old_k = p.k_scale[blk * p.k_scale_stride[0] + h * p.k_scale_stride[2]];
    const float old_v = p.v_scale[blk * p.v_scale_stride[0] + h * p.v_scale_stride[2]];
    float mk = 0.f, mv = 0.f;
    for (int r = row0; r < bs; r += rows) {
      const int st = ONE ? st0 : state(r);
      if (st == 2) {
        if (!ONE || h > h0) fetch_new(r, h);
        if (ch.turned) {
          new_k();
          mk = fmaxf(mk, amax16(xs, ys));
        } else {
          mk = fmaxf(mk, amax_packed<BF>(k0, k1));
        }
        mv = fmaxf(mv, amax_packed<BF>(v0, v1));
      } else if (ONE && st == 1) {
        fetch_held(r, h);
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
      if (st == 2) {  // (the rotation again rather than 16 more registers)
        if (!ONE) fetch_new(r, h);
        new_k();
        put(cache_row(p.k_cache, r, h), ik, inter && ch.turned, sk == kScaleMax);
        unpack16<BF>(v0, v1, false, xs, ys);
        put(cache_row(p.v_cache, r, h), iv, false, sv == kScaleMax);
      } else if (st == 1 && (sk > hk || sv > hv)) {
        if (!ONE) fetch_held(r, h);
        if (sk > hk) {
          decode8<I8>(make_uint2(k0.x, k0.y), xs);
          decode8<I8>(make_uint2(k1.x, k1.y), ys);
          put(cache_row(p.k_cache, r, h), __fdiv_rn(hk, sk), false, false);
        }
        if (sv > hv) {
          decode8<I8>(make_uint2(v0.x, v0.y), xs);
          decode8<I8>(make_uint2(v1.x, v1.y), ys);
          put(cache_row(p.v_cache, r, h), __fdiv_rn(hv, sv), false, false);
        }
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
