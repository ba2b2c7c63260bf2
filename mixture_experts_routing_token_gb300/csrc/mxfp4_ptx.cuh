// Inline-PTX helpers of the block-scaled 4-bit products: the instruction descriptor and
// MMA of kind::mxf4 (both operands e2m1, one power-of-two scale per 32 values) and the
// copy of scales from shared memory to tensor memory. Written from the PTX ISA
// descriptions of these instructions.
//
// Scales in tensor memory: 128 rows x 4 scales (K = 128) take 4 columns; lane l, column c
// holds the four bytes of row 32 c + l, in every lane quarter alike. In shared memory that
// is 512 bytes, 16 per lane: row r's four bytes at (r % 32) * 16 + (r / 32) * 4; one
// tcgen05.cp (32 lanes x 128 bits, to all four quarters) moves them. An MMA covers K = 64,
// two scales per row: the instruction descriptor says which two of the four bytes.
#pragma once
#include "common.cuh"
#include "pair_ptx.cuh"

namespace moe {
namespace mx {

constexpr uint32_t SF_ATOM = 512;    // bytes of 128 rows x 4 scales

__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (1u << 7)                         // A: e2m1
         | (1u << 10)                      // B: e2m1
         | ((uint32_t)(N >> 3) << 17)      // N / 8
         | (1u << 23)                      // scales: powers of two (ue8m0)
         | ((uint32_t)(M >> 4) << 24);     // M / 16
}
// Which of a row's four scale bytes: the pair starting at byte `sf` (0 or 2), for A and B.
__host__ __device__ constexpr uint32_t idesc_scales(int sf) { return ((uint32_t)sf << 4) | ((uint32_t)sf << 29); }

// Descriptor of a 512-byte scale atom: no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= (A * scales) (B * scales)^T over K = 64.
template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                    uint32_t accumulate) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 16 scale bytes of a row from byte b on; those past its end are 0 (their codes are, too). `end` is
// the end of the whole array. Rows that are no multiple of 4 bytes (vec 1) are read in the aligned
// words around them and shifted into place; words that would pass the array's end byte by byte.
__device__ __forceinline__ uint4 scale16(const uint8_t* row, int b, int count, int vec, const uint8_t* end) {
  if (vec == 16) return b < count ? __ldg(reinterpret_cast<const uint4*>(row + b)) : make_uint4(0, 0, 0, 0);
  uint32_t w[4];
  if (vec == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = b + 4 * j < count ? __ldg(reinterpret_cast<const uint32_t*>(row + b + 4 * j)) : 0u;
  } else {
    const uint8_t* p = row + b;
    const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint8_t* a = p - shift;
    uint32_t q[5];
    if (a + 20 <= end) {
#pragma unroll
      for (int j = 0; j < 5; ++j) q[j] = b + 4 * j - (int)shift < count ? __ldg(reinterpret_cast<const uint32_t*>(a) + j) : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(q[j], q[j + 1], 8 * shift);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (b + 4 * j + i < count) w[j] |= (uint32_t)__ldg(p + 4 * j + i) << (8 * i);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {      // what belongs to the next row
      const int left = count - b - 4 * j;
      if (left < 4) w[j] = left <= 0 ? 0u : w[j] & ((1u << (8 * left)) - 1u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes at a time in which scale16 may read rows of `count` bytes (the base is 16-byte aligned).
inline int scale_vec(int count) { return count % 16 == 0 ? 16 : count % 4 == 0 ? 4 : 1; }

// silu(z) = z / (1 + e^-z) with the approximate division (2 ulp; results below 2^-119 in
// magnitude, z < -87, become 0): with the IEEE division the epilogue took 12.9k cycles a tile,
// three and a half times the products.
__device__ __forceinline__ float silu_fast(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

}  // namespace mx
}  // namespace moe
