// 8-bit values (e4m3: four bits of exponent, three of mantissa, no infinities, 448 the largest) with a
// float32 scale per block, and the tensor-core product of two of them.
#pragma once
#include "common.cuh"

namespace moe {
namespace fp8 {

constexpr int BLOCK = 128;       // values along a row (and rows of a weight matrix) that share a scale

// Whether a product takes the weight-streaming kernel: up to 8 rows per expert on average. Measured, us, that kernel / the
// tiled one: one row of 8 experts, 64 experts [2816, 2048] with the gate 15 / 19; of 2 experts, [14336, 4096] 25 / 33;
// 8 rows of 4 experts, [2816, 1408] 7.4 / 9.3; 4 rows an expert, 8 experts [2816, 2048] 15 / 17, 64 experts 62 / 62; 8
// rows, 64 experts [2048, 1408] 34 / 37; 16 rows, 64 experts [2816, 2048] 65 / 64, 8 experts 16 / 14; 32 rows 72 / 65 and
// 19 / 14.
constexpr int kFewRows = 8;
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
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace fp8
}  // namespace moe
