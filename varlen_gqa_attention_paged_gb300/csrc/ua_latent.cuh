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
// hands it over when P.V of tile j is done, and a tile changes hands in three parts.
//
// Work split: all (row tile, key tile) pairs of the batch, row tile after row tile, are cut into
// equal shares for the workers (one CTA, or two that take neighbouring row tiles of a sequence over
// the same keys, so that the second read of a key hits L2).  A row tile that ends up with
// several workers leaves fp32 partial rows for the merge kernel.  A few row tiles over few keys take
// another split (SPREAD): a cluster of CTAs a row tile, an even part of its keys each, whose rows meet
// through distributed shared memory, without scratch and without a second kernel.
//
// Measured (one GB300, bf16, L 512, R 64): 64 sequences of up to 8191 keys, 16 heads, 75 us with the
// merge, 4.9 TB/s (0.72 of a copy; start, last share and merge are 12 us of it); 32 x 6000 keys, 128
// heads, 85.7 us, 624 TFLOP/s (0.33 of cuBLAS: the tensor cores are busy 45 % of the time, a tile takes
// 3060 cycles of which its products need 1940; two tiles in shared memory leave the chain of copy
// (1400), Q K^T, softmax (1400) and P.V bare); 16 heads, one token, 700 keys 10.1 us (launch and one
// chain).
#pragma once

#include <atomic>

#include "ua_latent.h"
#include "ua_latent_tc.cuh"

#include "ua.h"

namespace ua {

template <int L>
struct LatentCfg {
  static constexpr int kCB = L / 64;             // column blocks of the latent part
  static constexpr int kCH = kCB + 1;            // and the rope part's
  static constexpr int kMB = L / 128;            // accumulators of O^T
  static constexpr int kQCB = kLatRows * 128;    // one column block of Q
  static constexpr int kQBytes = kCH * kQCB;
  static constexpr int kKCB = kLatKeys * 128;    // one column block of a key tile
  static constexpr int kTileBytes = kCH * kKCB;
  // Parts of a key tile, which change hands one by one: the rope part (only Q K^T reads it), then
  // the latent part's halves.
  static constexpr int kHalves = kMB > 1 ? 2 : 1;
  static constexpr int kParts = 1 + kHalves;
  static constexpr int kHalfMB = kMB / kHalves;
  static constexpr int kPBytes = kLatRows * 128;
  static constexpr int kBarBytes = 320;           // barriers
  static constexpr int kSmallBytes = kBarBytes + 6 * kLatRows * 4;  // and row factors and maxima
  static constexpr int kFit =
      (227 * 1024 - 1024 - kSmallBytes - kQBytes - kPBytes) / kTileBytes;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kSmemBytes =
      1024 + kQBytes + kStages * kTileBytes + kPBytes + kSmallBytes;
  static constexpr int kTmemO = 2 * kLatKeys;    // two S buffers, then O^T
  static constexpr int kTmemCols = kTmemO + kMB * kLatRows > 256 ? 512 : 256;
  static constexpr int kThreads = 32 * (10 + kParts);  // softmax (8), MMA issue (2), a part's copies each
  static_assert(L % 128 == 0 && L <= 512 && kMB % kHalves == 0);
  static_assert(kStages * kTileBytes >= kLatRows * L * 4);  // a part's rows, where tiles were
  static_assert(kStages >= 2 && kSmemBytes + 96 <= 227 * 1024);
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

  // Part z of `parts` of the keys of row tile x (tiles of a sequence counted from floor(first row /
  // 64) + b): none left where there is no such tile, or no part.
  __device__ __forceinline__ LatentWalk(const LatentParams& p, int x, int z, int parts) {
    const int lane = threadIdx.x & 31;
    pos = left = 0;
    share = 1;
    b = t = j = 0;
    q0 = q_len = kv_len = rows = rt = kt = 0;
    for (int base = 0; base < p.num_seqs; base += 32) {
      const int i = base + lane;
      const bool in = i < p.num_seqs;
      const int c0 = in ? __ldg(p.cu_seqlens_q + i) : 0, c1 = in ? __ldg(p.cu_seqlens_q + i + 1) : 0;
      const int len = in ? __ldg(p.seq_lens_k + i) : 0;  // (all in one round of loads)
      const unsigned m = __ballot_sync(0xffffffffu, in && c0 * p.heads / kLatRows + i <= x);
      if (m != 0u) {
        const int src = 31 - __clz(m);
        b = base + src;
        q0 = __shfl_sync(0xffffffffu, c0, src);
        q_len = __shfl_sync(0xffffffffu, c1, src) - q0;
        kv_len = max(0, __shfl_sync(0xffffffffu, len, src));
      }
      if (m != 0xffffffffu) break;
    }
    rows = rows_of(p, q0, q0 + q_len);
    rt = row_tiles(p, rows);
    kt = key_tiles(kv_len);
    t = x - (q0 * p.heads / kLatRows + b);
    if (t < 0 || t >= rt) {
      rows = 0;
      return;
    }
    const int n = (kt + parts - 1) / parts;
    j = min(z * n, kt);
    left = min(n, kt - j);
  }

  // a / b, mostly of small numbers.
  __device__ __forceinline__ static int quotient(long long a, int b) {
    return static_cast<unsigned long long>(a) < 0x80000000ull ? static_cast<int>(a) / b
                                                              : static_cast<int>(a / b);
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
#pragma unroll 4
    for (int base = 32; base < p.num_seqs; base += 32) total += units(base + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    share = max(p.min_share, quotient(total + p.workers - 1, p.workers));
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
        t = quotient(off, kt);
        j = static_cast<int>(off - static_cast<long long>(t) * kt);
        // (the block table's entries are on their way to L2 while the roles set out)
        if (lane == 0)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(
              p.block_table + static_cast<size_t>(b) * p.max_blocks_per_seq +
              min(j * kLatKeys / p.block_size, p.max_blocks_per_seq - 1)));
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

// A box of a tensor map on its way to L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
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

// Two neighbouring elements of the output (`at` even).
__device__ __forceinline__ void store_two(void* out, size_t at, float a, float b, int dtype) {
  if (dtype == UA_DT_F32)
    *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = make_float2(a, b);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at) =
        dtype == UA_DT_BF16 ? pack_bf16(a, b) : pack_f16(a, b);
}

// 16 lanes x 32 columns of an accumulator over a warp: register 4 g + 2 k + e of lane t holds row
// t / 4 + 8 k, column 8 g + 2 (t mod 4) + e.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ln of a row's sum: m its reference in log2 units, l the sum of 2^(x - m).
__device__ __forceinline__ float latent_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The rows of a tile from the parts in the cluster's shared memory: a warp of the cluster takes 256
// elements (or a whole shorter row) at a time.
template <int L>
__device__ __forceinline__ void latent_join_parts(const LatentParams& p, uint32_t rows_at,
                                                  uint32_t stats_at, int rows, int row0, int warp,
                                                  int warps) {
  constexpr int kPieces = L > 256 ? L / 256 : 1, kPer = L / kPieces / 128;  // float4s of a lane
  const int lane = threadIdx.x & 31, parts = static_cast<int>(gridDim.y);
  for (int e = warp; e < rows * kPieces; e += warps) {
    const int r = e / kPieces, piece = e % kPieces;
    float m = -INFINITY, l = 0.f;
    if (lane < parts) {
      const uint32_t at = cluster_map(stats_at + 4 * r, lane);
      m = ld_cluster_f32(at);
      l = ld_cluster_f32(at + 4 * kLatRows);
    }
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float f = l == 0.f ? 0.f : fast_exp2(m - M);
    float sum = l == 0.f ? 0.f : l * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float4 acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < parts; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      if (__shfl_sync(0xffffffffu, l, k) == 0.f) continue;
      const uint32_t at = cluster_map(rows_at + 4 * (r * L + piece * 256 + 4 * lane), k);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float4 v = ld_cluster_f32x4(at + 512 * i);
        acc[i].x += v.x * fk;
        acc[i].y += v.y * fk;
        acc[i].z += v.z * fk;
        acc[i].w += v.w * fk;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const size_t to = static_cast<size_t>(row0 + r) * L + piece * 256 + 128 * i + 4 * lane;
      store_two(p.out, to, acc[i].x * inv, acc[i].y * inv, p.out_dtype);
      store_two(p.out, to + 2, acc[i].z * inv, acc[i].w * inv, p.out_dtype);
    }
    if (p.lse != nullptr && lane == 0 && piece == 0) p.lse[row0 + r] = latent_lse(M, sum);
  }
}

template <int L, bool BF16, bool SPREAD>
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
  uint64_t* const grown = bars + 8;    // the tile's rescale factors are written
  uint64_t* const s_empty = bars + 9;  // [2]
  uint64_t* const scaled = bars + 11;  // the factors of a tile that moves a max are written
  uint64_t* const k_full = bars + 12;  // [S][parts]
  uint64_t* const k_empty = k_full + S * C::kParts;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(k_empty + S * C::kParts);
  float* const sF = reinterpret_cast<float*>(bars + C::kBarBytes / 8);  // [2][64] factors of O's rows
  float* const sT = sF + 2 * kLatRows;                    // [2][2][64] row maxima (sums) of column halves
  static_assert(8 * (12 + 2 * S * C::kParts) + 4 <= C::kBarBytes);
  __shared__ int s_abort;
  // [tile mod 2][warp]: the tile + 1, if a row of the warp's is to move its max in it
  __shared__ int4 s_grow[2][2];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int worker = SPREAD ? blockIdx.x : blockIdx.x / p.cl, rank = SPREAD ? 0 : blockIdx.x % p.cl;
  constexpr int kQk = 8, kPv = 9, kCopy = 10;  // (kCopy + g copies part g)

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_full, 8);
    mbar_init(pv_done, 1);
    mbar_init(o_empty, 8);
    mbar_init(fin, 2);
    mbar_init(grown, 8);
    mbar_init(scaled, 8);
    mbar_init(&s_empty[0], 8);
    mbar_init(&s_empty[1], 8);
    for (int i = 0; i < S * C::kParts; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    s_abort = 0;
    for (int i = 0; i < 4; ++i) s_grow[i >> 1][i & 1] = make_int4(0, 0, 0, 0);
    mbar_fence_init();
  }
  if (warp == kQk) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kCopy && lane == 0) {
    tma_prefetch_desc(&p.q_map);
    tma_prefetch_desc(&p.q_lat);
    tma_prefetch_desc(&p.k_map);
    tma_prefetch_desc(&p.k_half);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  volatile int* abort_flag = &s_abort;
  grid_dependency_wait();
  grid_launch_dependents();

  LatentWalk w = SPREAD ? LatentWalk(p, worker, blockIdx.y, gridDim.y) : LatentWalk(p, worker);
  // SPREAD: the row tile, in every CTA of the cluster
  const int tile_rows = SPREAD ? min(kLatRows, w.rows - w.t * kLatRows) : 0;
  const int tile_row0 = SPREAD ? w.q0 * p.heads + w.t * kLatRows : 0;
  int it = 0;  // key tiles of all segments so far
  int sg = 0;  // segments with key tiles so far
  bool ok = true;

  if (warp >= kCopy) {
    // ======================================================== copies
    // A warp a part of the tiles, each copied as soon as its place is free: Q K^T frees the rope
    // part's, the P.V of a half the half's.  (One warp for all parts took 1000 cycles a part.)
    const int g = warp - kCopy;
    const int cb0 = g == 0 ? C::kCB : 2 * C::kHalfMB * (g - 1);
    const int blocks = g == 0 ? 1 : 2 * C::kHalfMB;
    const int bs = p.block_size;
    const int oob = p.num_blocks * bs;
    // keys of a box, boxes of a column block (a power of two)
    const int bw = p.box_rows, nb = kLatKeys / bw, sh = __ffs(nb) - 1;
    for (; ok && w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      if (s.nt <= 0) continue;
      if (g == 0 && sg > 0 && !pf_wait_warp(q_empty, (sg - 1) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      if (g == 0 && lane == 0) {
        const int row = w.q0 * p.heads + s.row0;
        mbar_arrive_expect_tx(q_full, C::kQBytes);
        tma_load_3d_pf(sQ, &p.q_lat, 0, row, 0, q_full);
        tma_load_2d(sQ + C::kCB * C::kQCB, &p.q_map, L, row, q_full);
      }
      ++sg;
      const int32_t* bt = p.block_table + static_cast<size_t>(w.b) * p.max_blocks_per_seq;
      // Boxes of the segment, tile after tile, go by batches of 32, a lane each: rows_a and rows_b
      // are the cache rows of batch c and the next, blk the blocks of the one after, on their way.
      // (Found tile by tile, with divisions and a wait for a load in each, a tile took a copy warp 1400
      // to 2100 cycles: 64 sequences of up to 8191 keys, latents of 128, 50.1 us, now 42.7; latents
      // of 512 in pages of 16, 86.8, now 78.2.)
      const unsigned boxes = static_cast<unsigned>(s.nt) << sh;
      auto block_of = [&](int batch) -> int {
        const unsigned box = 32u * batch + lane, key = s.j0 * kLatKeys + box * bw, col = key / bs;
        return box < boxes && key < static_cast<unsigned>(w.kv_len) &&
                       col < static_cast<unsigned>(p.max_blocks_per_seq)
                   ? __ldg(bt + col)
                   : -1;
      };
      // (past the cache, so that the copy fills zeros, where there is no key)
      auto row_of = [&](int batch, int block) -> int {
        const unsigned box = 32u * batch + lane, key = s.j0 * kLatKeys + box * bw;
        if (box >= boxes || key >= static_cast<unsigned>(w.kv_len)) return oob;
        if (static_cast<unsigned>(block) >= static_cast<unsigned>(p.num_blocks)) {
          if (g == 0) atomicOr(p.status, DEV_BAD_BLOCK);
          return oob;
        }
        return block * bs + static_cast<int>(key % bs);
      };
      int c = 0;
      const int first = block_of(0), second = block_of(1);
      int blk = block_of(2);
      int rows_a = row_of(0, first), rows_b = nb > 32 ? row_of(1, second) : oob;
      for (int n = 0; ok && n < s.nt; ++n, ++it) {
        const unsigned box0 = static_cast<unsigned>(n) << sh;  // the tile's first box
        while (static_cast<int>(box0 >> 5) > c) {
          rows_a = rows_b;
          rows_b = row_of(c + 2, blk);
          ++c;
          blk = block_of(c + 2);
        }
        const int st = it % S;
        uint8_t* const tile = sK + st * C::kTileBytes;
        uint64_t* const full = &k_full[st * C::kParts + g];
        if (it >= S && !pf_wait_warp(&k_empty[st * C::kParts + g], ((it / S) - 1) & 1, abort_flag,
                                     p.status)) {
          ok = false;
          break;
        }
        // (only now: the tile before has arrived, so that its phase of the barrier is over)
        if (lane == 0) mbar_arrive_expect_tx(full, blocks * C::kKCB);
        if (bw == kLatKeys) {  // one box a block of columns; a half in one copy
          const int row = __shfl_sync(0xffffffffu, rows_a, box0 & 31);
          if (lane == 0) {
            if (g > 0) tma_load_3d_pf(tile + cb0 * C::kKCB, &p.k_half, 0, row, cb0, full);
            else tma_load_2d(tile + cb0 * C::kKCB, &p.k_map, 64 * cb0, row, full);
          }
        } else {
          __syncwarp();
          for (int e = lane; e - lane < blocks << sh; e += 32) {
            const int cb = cb0 + (e >> sh), box = e & (nb - 1);
            const int lo = __shfl_sync(0xffffffffu, rows_a, (box0 + box) & 31);
            const int hi = __shfl_sync(0xffffffffu, rows_b, box & 31);
            if (e < blocks << sh)
              tma_load_2d(tile + cb * C::kKCB + box * bw * 128, &p.k_map, 64 * cb,
                          box < 32 ? lo : hi, full);
          }
        }
        if (n == 0 && nb <= 32) rows_b = row_of(1, second);
        // With two tiles in shared memory the copy of one waits for the products of the one before:
        // the next but one comes as far as L2 meanwhile.
        // (Four tiles are far enough ahead by themselves.)
        if (S < 4 && n + 2 < s.nt) {
          const unsigned box2 = static_cast<unsigned>(n + 2) << sh;
          const int batch = static_cast<int>(box2 >> 5);
          const int ahead = __shfl_sync(0xffffffffu, batch == c ? rows_a : rows_b, (box2 + lane) & 31);
          if (batch > c + 1) {  // (pages of one or two tokens)
          } else if (g > 0 && bw == kLatKeys) {
            if (lane == 0) tma_prefetch_3d(&p.k_half, 0, ahead, cb0);
          } else if (lane < nb) {
            for (int cb = cb0; cb < cb0 + blocks; ++cb) tma_prefetch_2d(&p.k_map, 64 * cb, ahead);
          }
        }
        __syncwarp();
      }
    }
    // never leave copies in flight into this CTA's shared memory (even after an abort)
    for (int i = max(0, it - S); i < it; ++i)
      mbar_wait_bounded(&k_full[i % S * C::kParts + g], (i / S) & 1, p.status, DEV_TIMEOUT);
    if (g == 0 && sg > 0) mbar_wait_bounded(q_full, (sg - 1) & 1, p.status, DEV_TIMEOUT);
  } else if (warp == kQk) {
    // ======================================================== MMA issue: S = Q K^T
    // A warp issues these products and another P.V's, so that neither waits behind the other's
    // inputs (one that took whichever was ready spent 350 cycles a look).  The MMAs are unrolled:
    // in a rolled loop an issue took 52 cycles a 64 x 64 x 16 product instead of the 33 that it
    // takes to run.
    constexpr uint32_t kId = umma_idesc_f16(kLatRows, kLatKeys, BF16, false);
    const int rope_steps = p.rope_dim / 16;
    for (; ok && w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      if (s.nt <= 0) continue;
      ok = pf_wait_warp(q_full, sg & 1, abort_flag, p.status);
      for (int n = 0; ok && n < s.nt; ++n, ++it) {
        const int st = it % S;
        const uint32_t qd = smem_units(sQ), kd = smem_units(sK + st * C::kTileBytes);
        const uint32_t tS = tmem + (it & 1) * kLatKeys;
        uint64_t* const full = &k_full[st * C::kParts];
        // the scores of two tiles before have been read
        if (it >= 2 && !pf_wait_warp(&s_empty[it & 1], ((it >> 1) - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (!pf_wait_warp(&full[0], (it / S) & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < rope_steps)
            umma_f16_ss_at(tS, qd + (C::kCB * C::kQCB) / 16 + 2 * kk, 16,
                           kd + (C::kCB * C::kKCB) / 16 + 2 * kk, 16, kId, kk > 0 ? 1u : 0u);
        umma_commit_warp(&k_empty[st * C::kParts]);
#pragma unroll
        for (int g = 0; g < C::kHalves; ++g) {
          if (!pf_wait_warp(&full[1 + g], (it / S) & 1, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8 * C::kHalfMB; ++k) {
            const int kk = g * 8 * C::kHalfMB + k;
            umma_f16_ss_at(tS, qd + (kk >> 2) * (C::kQCB / 16) + (kk & 3) * 2, 16,
                           kd + (kk >> 2) * (C::kKCB / 16) + (kk & 3) * 2, 16, kId, 1u);
          }
        }
        if (!ok) break;
        umma_commit_warp(&s_full[it & 1]);
        if (n == s.nt - 1) umma_commit_warp(q_empty);
      }
      ++sg;
    }
    // nothing may still be in flight on the tensor cores when the memory is freed
    umma_commit_warp(fin);
    mbar_wait_bounded(fin, 0, p.status, DEV_TIMEOUT);
  } else if (warp == kPv) {
    // ======================================================== MMA issue: O^T += V^T P^T
    constexpr uint32_t kId = umma_idesc_f16(128, kLatRows, BF16, false) | (1u << 15);
    for (; ok && w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      if (s.nt <= 0) continue;
      for (int n = 0; n < s.nt; ++n, ++it) {
        const int st = it % S;
        if (!pf_wait_warp(p_full, it & 1, abort_flag, p.status) ||
            (n == 0 && sg > 0 && !pf_wait_warp(o_empty, (sg - 1) & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t vd = smem_units(sK + st * C::kTileBytes), pd = smem_units(sP);
#pragma unroll
        for (int mb = 0; mb < C::kMB; ++mb) {
#pragma unroll
          for (int ks = 0; ks < kLatKeys / 16; ++ks)
            umma_f16_ss_at(tmem + C::kTmemO + mb * kLatRows, vd + (mb * 2 * C::kKCB + ks * 2048) / 16,
                           C::kKCB, pd + ks * 2, 16, kId, ks > 0 ? 1u : n > 0 ? 1u : 0u);
          if ((mb + 1) % C::kHalfMB == 0)
            umma_commit_warp(&k_empty[st * C::kParts + 1 + mb / C::kHalfMB]);
        }
        umma_commit_warp(pv_done);
      }
      ++sg;
    }
    umma_commit_warp(fin);
    mbar_wait_bounded(fin, 0, p.status, DEV_TIMEOUT);
  } else {
    // ======================================================== softmax, rescale, epilogue
    // An M = 64 accumulator keeps rows 16 w .. 16 w + 15 in the first half of lane quarter w.  Two
    // warps share them, half of the columns each: a lane has rows ra and ra + 8, columns 32 half +
    // 8 g + 2 cq and the next.
    const int quad = warp & 3, half = warp >> 2;
    const int ra = 16 * quad + (lane >> 2), cq = lane & 3;
    const uint32_t lane_off = (32u * quad) << 16;
    const uint32_t tO = tmem + C::kTmemO + lane_off;
    const float c = p.scale * kLog2e;
    constexpr float kDown = latent_down(BF16), kRoom = 8.f + kDown;
    // (of O's 32-column pieces, the warps of a lane quarter take every other 128-element block, or,
    // with one block, a piece each)
    auto mine = [&](int piece) { return (C::kMB > 1 ? piece >> 1 & 1 : piece & 1) == half; };
    int moved = 0;  // tiles that moved a max
    int4 meta = make_int4(0, 0, 0, 0);
    // (After a wait that gave up, these warps go on to the end, through every barrier that they
    // share; their later waits return at once, and nothing is stored.)
    for (; w.left > 0; w.next(p)) {
      const LatentSeg s(p, w, rank);
      const int grow0 = w.q0 * p.heads + s.row0;  // its first row in q and out
      const bool whole = !SPREAD && w.j == 0 && w.length() == w.kt;
      const int slot = 2 * blockIdx.x + (w.j == 0 ? 1 : 0);
      const int rows = s.rows;
      if (rows <= 0) continue;
      if (!SPREAD && w.j == 0 && !whole)
        meta = make_int4(grow0, rows,
                         static_cast<int>((w.pos + w.kt - 1) / w.share) - worker + 1, 0);
      const bool rv[2] = {ra < rows, ra + 8 < rows};
      int i_q[2];  // the rows' tokens
#pragma unroll
      for (int k = 0; k < 2; ++k) i_q[k] = (s.row0 + min(ra + 8 * k, rows - 1)) / p.heads;
      // keys that every row of the tile sees without looking at its mask
      const int clear = min(w.kv_len, p.tree != nullptr ? s.ctx : s.ctx + s.row0 / p.heads + 1);
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // (l: this lane's columns)
      for (int n = 0; n < s.nt; ++n, ++it) {
        ok = pf_wait_warp(&s_full[it & 1], (it >> 1) & 1, abort_flag, p.status) && ok;
        tc_fence_after();
        const int k0 = (s.j0 + n) * kLatKeys;
        uint32_t x[16];  // [g][row][2]
        tmem_ld_16x256b_x4(tmem + (it & 1) * kLatKeys + 32 * half + lane_off, x);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[it & 1]);
        const int kh = k0 + 32 * half;
        if (kh + 32 > clear) {
          // the keys that a row sees: of the prefix (tree) or up to its own, and those its mask
          // names
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t see =
                low_bits(min(w.kv_len, p.tree != nullptr ? s.ctx : s.ctx + i_q[k] + 1) - kh);
            if (p.tree != nullptr && rv[k]) {
              const int32_t* row = p.tree + (static_cast<long long>(w.q0) + i_q[k]) * p.tree_stride;
              see |= mask_bits32(row, p.tree_words, kh - s.ctx) & low_bits(w.kv_len - kh) &
                     ~low_bits(s.ctx - kh);
            }
            see >>= 2 * cq;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (!(see >> (8 * g) & 1u)) x[4 * g + 2 * k] = 0xff800000u;
              if (!(see >> (8 * g) & 2u)) x[4 * g + 2 * k + 1] = 0xff800000u;
            }
          }
        }
        // The reference m (the running max, in f16 kDown below it) moves only when the max is more
        // than kRoom above it, or at a row's first key.  That is rare, so the exponentials are
        // taken with the old one while the column halves hear from each other whether it moves.
        float top[2];
        bool grow = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float t = -INFINITY;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            t = fmax3(t, __uint_as_float(x[4 * g + 2 * k]), __uint_as_float(x[4 * g + 2 * k + 1]));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          top[k] = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2)) * c;
          grow = grow || (rv[k] && (top[k] > m[k] + kRoom || (m[k] == -INFINITY && top[k] > -INFINITY)));
        }
        float* const tops = sT + (it & 1) * 2 * kLatRows;
        if (cq == 0) {
          tops[half * kLatRows + ra] = top[0];
          tops[half * kLatRows + ra + 8] = top[1];
        }
        if (__any_sync(0xffffffffu, grow) && lane == 0)
          reinterpret_cast<int*>(s_grow[it & 1])[warp] = it + 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(grown);
        // P rounded to 16 bits for the MMA (half a step of 2^-8 or 2^-11 of each weight, in f16 at
        // least 2^-32 of the largest); the sum is of the unrounded weights
        uint32_t pk[8];  // [row][g]
        float add[2];
        auto weights = [&]() {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float mu = m[k] == -INFINITY ? 0.f : m[k];
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float a = fast_exp2(fmaf(__uint_as_float(x[4 * g + 2 * k]), c, -mu));
              const float b = fast_exp2(fmaf(__uint_as_float(x[4 * g + 2 * k + 1]), c, -mu));
              l0 += a;
              l1 += b;
              pk[4 * k + g] = pack_half2<BF16>(a, b);
            }
            add[k] = l0 + l1;
          }
        };
        weights();
        // P's buffer and O are free when the P.V before is done
        if (it > 0) ok = pf_wait_warp(pv_done, (it - 1) & 1, abort_flag, p.status) && ok;
        tc_fence_after();
        ok = pf_wait_warp(grown, it & 1, abort_flag, p.status) && ok;
        const int4 ga = s_grow[it & 1][0], gb = s_grow[it & 1][1];
        const int now = it + 1;
        if (ga.x == now || ga.y == now || ga.z == now || ga.w == now || gb.x == now || gb.y == now ||
            gb.z == now || gb.w == now) {
          float* const f = sF + (it & 1) * kLatRows;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float t = fmaxf(top[k], tops[(half ^ 1) * kLatRows + ra + 8 * k]);
            float alpha = 1.f;
            if (rv[k] && (t > m[k] + kRoom || (m[k] == -INFINITY && t > -INFINITY))) {
              alpha = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - (t - kDown));
              m[k] = t - kDown;
            }
            l[k] *= alpha;
            if (half == 0 && cq == 0) f[ra + 8 * k] = alpha;
          }
          weights();
          // O has every row in every warp's lanes
          __syncwarp();
          if (lane == 0) mbar_arrive(scaled);
          ok = pf_wait_warp(scaled, moved & 1, abort_flag, p.status) && ok;
          ++moved;
          if (n > 0) {
#pragma unroll 1
            for (int cc = 0; cc < C::kMB * 2; ++cc) {
              if (!mine(cc)) continue;
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
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          l[k] += add[k];
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint32_t*>(sP + (ra + 8 * k) * 128 + (((4 * half + g) ^ (ra & 7)) << 4) +
                                         4 * cq) = pk[4 * k + g];
        }
        // Cache slots at or past kv_len may hold anything (NaN included): they become zeros
        // before they meet P = 0 (a box of a copy that lies past kv_len altogether is zeros).
        if (k0 + kLatKeys > w.kv_len) {
          const int lo = w.kv_len - k0, end = min(kLatKeys, (lo + p.box_rows - 1) & -p.box_rows);
          uint8_t* const tile = sK + (it % S) * C::kTileBytes;
          for (int e = threadIdx.x; e < (end - lo) * C::kCB * 8; e += 256) {
            const int row = lo + e / (C::kCB * 8), x = e % (C::kCB * 8);
            *reinterpret_cast<uint4*>(tile + (x >> 3) * C::kKCB + row * 128 + (x & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }

      // ---- epilogue: O / l of a tile that is this worker's alone, else the partial rows
      float* const f = sF + (it & 1) * kLatRows;
      if (s.nt > 0) {
        ok = pf_wait_warp(pv_done, (it - 1) & 1, abort_flag, p.status) && ok;
        tc_fence_after();
      }
      // a row's sum: its lanes', then the column halves'
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        if (half == 1 && cq == 0) sT[(it & 1) * 2 * kLatRows + ra + 8 * k] = l[k];
      }
      named_bar_sync(1, 256);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = ra + 8 * k;
        if (half != 0 || cq != 0) continue;
        const float sum = l[k] + sT[(it & 1) * 2 * kLatRows + r];
        if constexpr (SPREAD) {
          sF[r] = m[k];
          sF[kLatRows + r] = ok ? sum : NAN;  // (after a wait that gave up the tile's rows are NaN)
          continue;
        }
        // (a row that saw no key is 0; NaN stays)
        f[r] = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        if (!rv[k] || !ok) continue;
        if (!whole) {
          p.ws_m[slot * kLatRows + r] = m[k];
          p.ws_l[slot * kLatRows + r] = sum;
        } else if (p.lse != nullptr) {
          p.lse[grow0 + r] = latent_lse(m[k], sum);
        }
      }
      named_bar_sync(1, 256);
      const int d = 32 * quad + lane;  // this lane's element of a 128-element block of O
      if (ok && (whole || s.nt > 0)) {  // (an empty partial row's sum is 0: its elements are not read)
#pragma unroll 1
        for (int cc = 0; cc < C::kMB * 2; ++cc) {
          const int rb = 32 * (cc & 1), blk = (cc >> 1) * 128;
          if (rb >= rows || !mine(cc)) continue;
          uint32_t o[32];
          if (s.nt > 0) {
            tmem_ld32(tO + 32 * cc, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if constexpr (SPREAD) {
            float* const dst = reinterpret_cast<float*>(sK) + rb * L + blk + d;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (rb + e < rows) dst[e * L] = __uint_as_float(o[e]);
            continue;
          }
          if (!whole) {
            float* const dst = p.ws_acc + static_cast<size_t>(slot * kLatRows + rb) * L + blk + d;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (rb + e < rows) dst[static_cast<size_t>(e) * L] = __uint_as_float(o[e]);
            continue;
          }
          // Two rows at a time: an even lane takes both its own and its neighbour's element of the
          // first, an odd one of the second, so that a store has two elements.
          const size_t at = static_cast<size_t>(grow0 + rb) * L + blk + (d & ~1);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            if (rb + e >= rows) break;
            const float f0 = f[rb + e], f1 = f[rb + e + 1];
            const float v0 = f0 == 0.f ? 0.f : __uint_as_float(o[e]) * f0;
            const float v1 = f1 == 0.f ? 0.f : __uint_as_float(o[e + 1]) * f1;
            const bool odd = lane & 1;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            const float a = odd ? got : v0, b = odd ? v1 : got;
            if (rb + e + (odd ? 1 : 0) < rows)
              store_two(p.out, at + static_cast<size_t>(e + (odd ? 1 : 0)) * L, a, b, p.out_dtype);
          }
        }
      }
      if (s.nt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);
        ++sg;
      }
      named_bar_sync(1, 256);  // the factors have been read
    }
    if constexpr (SPREAD) {
      if (sg == 0 && threadIdx.x < kLatRows) {  // (a part that saw no key counts for nothing)
        sF[threadIdx.x] = -INFINITY;
        sF[kLatRows + threadIdx.x] = 0.f;
      }
    } else if (threadIdx.x == 0) {
      p.ws_meta[blockIdx.x] = ok ? meta : make_int4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kQk) tmem_dealloc(tmem, C::kTmemCols);
  if constexpr (SPREAD) {
    cluster_sync();  // every part's rows, maxima and sums are in its shared memory
    latent_join_parts<L>(p, smem_addr(sK), smem_addr(sF), tile_rows, tile_row0,
                         blockIdx.y * (C::kThreads / 32) + warp, gridDim.y * (C::kThreads / 32));
    cluster_sync_relaxed();  // no CTA leaves while another reads its shared memory
  }
}

template <int L, bool BF16, bool SPREAD>
cudaError_t launch_latent_t(const LatentParams& p, cudaStream_t stream) {
  using C = LatentCfg<L>;
  auto kern = ua_latent_kernel<L, BF16, SPREAD>;
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
  const dim3 grid = SPREAD ? dim3(static_cast<unsigned>(p.workers), static_cast<unsigned>(p.spread))
                           : dim3(static_cast<unsigned>(p.workers * p.cl));
  return launch_pdl(kern, grid, dim3(C::kThreads), C::kSmemBytes, stream, SPREAD ? p.spread : 1, p);
}

template <int L>
cudaError_t launch_latent_any(const LatentParams& p, bool bf16, cudaStream_t s) {
  if (p.spread > 0)
    return bf16 ? launch_latent_t<L, true, true>(p, s) : launch_latent_t<L, false, true>(p, s);
  return bf16 ? launch_latent_t<L, true, false>(p, s) : launch_latent_t<L, false, false>(p, s);
}

}  // namespace ua
