// ua_latent_tc.cuh -- copies and tensor-core operands that both latent-attention kernels use.
#pragma once

#include "ua_prefill.cuh"

namespace ua {

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], 128-byte swizzle, stride byte offset 1024 (eight rows), issued by
// one lane of a converged warp; operands by their address / 16 and leading byte offset.
__device__ __forceinline__ void umma_f16_ss_at(uint32_t d_tmem, uint32_t a16, uint32_t a_lbo,
                                               uint32_t b16, uint32_t b_lbo, uint32_t idesc,
                                               uint32_t accumulate) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a16 + ((a_lbo >> 4) << 16)), "r"(b16 + ((b_lbo >> 4) << 16)), "r"(hi), "r"(idesc),
      "r"(accumulate)
      : "memory");
}

// How far below a row's running max its weights' reference m is, in log2 units.  Weights are
// 2^(x - m), and m moves when the max is more than 8 above where it was, so they reach 2^8 in bf16 and
// 2^15 in f16 (inside its range, and fp32 sums').  In f16 the largest weight is 2^7 at least then, and
// the smallest steps, 2^-24, are 2^-31 of that.  (With m at the max itself they were 2^-24 of it: tens
// of thousands of keys below 2^-25 counted in the sum and not in the output.)
__host__ __device__ constexpr float latent_down(bool bf16) { return bf16 ? 0.f : 7.f; }

// A shared-memory address as descriptors have it, in 16-byte units.  (In a CTA of a cluster the bits
// above the window's 18 hold its rank, which would land in the leading byte offset.)
__device__ __forceinline__ uint32_t smem_units(const void* at) {
  return (smem_addr(at) & 0x3ffffu) >> 4;
}

// The descriptor of an operand at address 16 a16: 128-byte swizzle, stride byte offset 1024.
__device__ __forceinline__ uint64_t smem_desc_at(uint32_t a16, uint32_t lbo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return static_cast<uint64_t>(hi) << 32 | (a16 + ((lbo >> 4) << 16));
}

}  // namespace ua
