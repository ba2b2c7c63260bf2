// 4-bit microscaled values: quantisation and its inverse.
//
// A row is cut into blocks of 32 values. A block's scale is a power of two,
//   s = max(floor(log2 m) - 2, -127),  m = the block's largest magnitude,
// kept as the byte s + 127, and a value v becomes the nearest of 0, 0.5, 1, 1.5, 2, 3,
// 4, 6 (and their negatives) to v 2^-s: ties to the even code, more than 6 to 6 (m 2^-s
// lies in [4, 8)). v 2^-s is exact in float32 (it only gets small where it rounds to 0
// anyway), so the 4-bit rounding is the only one. A block that holds an infinity or a NaN
// has the byte 255 (which stands for NaN) and codes 0. Element 2i of a row is the low
// half of byte i, element 2i + 1 the high half.
//
// Both directions move each byte once and are bound by memory: four neighbouring lanes
// hold a block, eight values each, so a warp reads 512 contiguous bytes of a 16-bit row
// and writes 128 of codes; the block's largest magnitude is two shuffles of the values'
// bits as integers (magnitudes of floats order like integers, and infinity and NaN come
// out on top without a test). Every thread has kUnroll reads under way.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kUnroll = 4;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Eight float32 values to eight 4-bit codes (nearest, ties to even, saturating at 6).
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight 4-bit codes to the values they stand for before scaling, as four half pairs.
__device__ __forceinline__ void decode8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// 2^(byte - 127); 255 stands for NaN, 0 for the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

template <class T>
__global__ void __launch_bounds__(256)
    mxfp4_quantize_kernel(const T* __restrict__ x, int T_rows, int K, int sh, const int32_t* __restrict__ rows, long n,
                          uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, int32_t* status) {
  const int C = K / 8;                                     // pieces of 8 values in a row
  const long stride = (long)gridDim.x * blockDim.x;
  const int lane = threadIdx.x & 31;
  // whole warps take each turn (the shuffles need all lanes); lanes past the end carry zeros
  for (long i0 = (long)blockIdx.x * blockDim.x + threadIdx.x; i0 - lane < n; i0 += kUnroll * stride) {
    float v[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      const long r = div_idx(i < n ? i : 0, C, sh);
      long src = r;
      if (rows != nullptr && i < n) src = __ldg(rows + r);
      if (i < n && src >= 0 && src < T_rows) {
        load8(x + src * K + (i - r * C) * 8, v[u]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = 0.0f;
        if (i < n && status != nullptr) atomicOr(status, MOE_STATUS_BAD_INDEX);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[u][j]) & 0x7fffffffu);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const bool bad = m >= 0x7f800000u;
      const uint32_t byte = bad ? 255u : (uint32_t)max((int)(m >> 23) - 2, 0);
      const float up = bad ? 0.0f : __uint_as_float((254u - byte) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] *= up;
      if (i < n) {
        codes[i] = bad ? 0u : encode8(v[u]);
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
      }
    }
  }
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  T q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = from_float<T>(v[j]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(q);
}

template <class T>
__global__ void __launch_bounds__(256)
    mxfp4_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, long n,
                            T* __restrict__ out) {
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i0 = (long)blockIdx.x * blockDim.x + threadIdx.x; i0 < n; i0 += kUnroll * stride) {
    uint32_t c[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      c[u] = i < n ? __ldg(codes + i) : 0;
      b[u] = i < n ? __ldg(scales + (i >> 2)) : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      if (i >= n) break;
      uint32_t h[4];
      decode8(c[u], h);
      const float s = scale_value(b[u]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      store8(out + i * 8, v);
    }
  }
}

int blocks_for(long n) {
  const long want = (n + 256 * kUnroll - 1) / (256 * kUnroll), most = (long)num_sms() * 8;
  return (int)(want < most ? want : most);
}

template <class T>
int quantize(const void* x, int Tr, int K, const int32_t* rows, int R, uint8_t* codes, uint8_t* scales, int32_t* status,
             cudaStream_t s) {
  const long n = (long)R * (K / 8);
  ProfScope ps("mxfp4_quantize", s);
  mxfp4_quantize_kernel<T><<<blocks_for(n), 256, 0, s>>>(static_cast<const T*>(x), Tr, K, pow2_shift(K / 8), rows, n,
                                                        reinterpret_cast<uint32_t*>(codes), scales, status);
  return check_launch("mxfp4_quantize");
}

template <class T>
int dequantize(const uint8_t* codes, const uint8_t* scales, int R, int K, void* out, cudaStream_t s) {
  const long n = (long)R * (K / 8);
  ProfScope ps("mxfp4_dequantize", s);
  mxfp4_dequantize_kernel<T><<<blocks_for(n), 256, 0, s>>>(reinterpret_cast<const uint32_t*>(codes), scales, n,
                                                          static_cast<T*>(out));
  return check_launch("mxfp4_dequantize");
}

}  // namespace

int launch_mxfp4_quantize(const void* x, int dtype, int T, int K, const int32_t* rows, int R, uint8_t* codes,
                          uint8_t* scales, int32_t* status, cudaStream_t s) {
  if (dtype == MOE_F32) return quantize<float>(x, T, K, rows, R, codes, scales, status, s);
  if (dtype == MOE_BF16) return quantize<__nv_bfloat16>(x, T, K, rows, R, codes, scales, status, s);
  return quantize<__half>(x, T, K, rows, R, codes, scales, status, s);
}

int launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int R, int K, int dtype, void* out,
                            cudaStream_t s) {
  if (dtype == MOE_F32) return dequantize<float>(codes, scales, R, K, out, s);
  if (dtype == MOE_BF16) return dequantize<__nv_bfloat16>(codes, scales, R, K, out, s);
  return dequantize<__half>(codes, scales, R, K, out, s);
}

}  // namespace moe
