// 8-bit values (e4m3: four bits of exponent, three of mantissa, no infinities, 448 the largest) with a
// float32 scale per block, and the tensor-core product of two of them.
#pragma once
#include "common.cuh"

namespace moe {
namespace fp8 {

constexpr int BLOCK = 128;       // values along a row (and rows of a weight matrix) that share a scale

// Whether a product takes the weight-streaming kernel: up to 48 rows per expert on average. Measured, us, that kernel /
// the SM-pair kernel, 64 experts [2816, 2048]: with the gate 65 / 95 at 16 rows, 72 / 96 at 32, 85 / 97 at 48, 118 / 97
// at 64; without 61 / 89, 71 / 92, 85 / 93, 122 / 95; 8 experts [14336, 4096] 78 / 102 at 32, 91 / 106 at 48, 136 / 107 at 64.
constexpr int kFewRows = 48;
inline bool few_rows(int S, int E) { return S <= (long)kFewRows * E; }

__host__ __device__ constexpr int blocks(int n) { return (n + BLOCK - 1) / BLOCK; }

// Four float32 values to four codes, the first one low (nearest, ties to even, above 448 to 448).
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four codes to the values they stand for before scaling (every one is exact in float16).
__device__ __forceinline__ float4 decode4(uint32_t codes) {
  uint32_t l, h;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(l), "=r"(h)
      : "r"(codes));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&l)), y = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return make_float4(x.x, x.y, y.x, y.y);
}

// Instruction descriptor, kind::f8f6f4: D float32, A and B e4m3 (format 0), both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem]^T over K = 32.
template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace fp8
}  // namespace moe
