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
// out on top without a test). Two reads under way per thread and as many blocks as there is work
// measured best (f32 rows, 738 + 98 MB: 117 us = 7.2 TB/s; four reads 123, a grid of eight blocks an
// SM that loops 129; values of bf16 back, 679 MB: 100 us = 6.8 TB/s).
#include <algorithm>

#include "grouped.cuh"

namespace moe {
namespace {

constexpr int kUnroll = 2;

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
  pdl_wait();
  pdl_trigger();
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

// 16 values of one row as whole 32-byte sectors (or 16-byte halves where the output is not so aligned).
template <class T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16], bool sectors) {
  constexpr int Q = 4 * (int)sizeof(T);     // words
  uint32_t q[Q];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < Q; ++j) q[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < Q; ++j) q[j] = grouped::pack_pair<T>(v[2 * j], v[2 * j + 1]);
  }
  uint32_t* d = reinterpret_cast<uint32_t*>(p);
#pragma unroll
  for (int j = 0; j < Q / 8; ++j) {
    if (sectors) {
      uint32_t w[8];
#pragma unroll
      for (int l = 0; l < 8; ++l) w[l] = q[8 * j + l];
      st_v8(d + 8 * j, w);
    } else {
      reinterpret_cast<uint4*>(d)[2 * j] = make_uint4(q[8 * j], q[8 * j + 1], q[8 * j + 2], q[8 * j + 3]);
      reinterpret_cast<uint4*>(d)[2 * j + 1] = make_uint4(q[8 * j + 4], q[8 * j + 5], q[8 * j + 6], q[8 * j + 7]);
    }
  }
}

// 16 codes per thread: half a block.
template <class T>
__global__ void __launch_bounds__(256)
    mxfp4_dequantize_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, long n,
                            T* __restrict__ out, bool sectors) {
  pdl_wait();
  pdl_trigger();
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i0 = (long)blockIdx.x * blockDim.x + threadIdx.x; i0 < n; i0 += kUnroll * stride) {
    uint2 c[kUnroll];
    uint32_t b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      c[u] = i < n ? __ldg(codes + i) : make_uint2(0, 0);
      b[u] = i < n ? __ldg(scales + (i >> 1)) : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      if (i >= n) break;
      const float s = scale_value(b[u]);
      float v[16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[4];
        decode8(h ? c[u].y : c[u].x, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          v[8 * h + 2 * j] = f.x * s;
          v[8 * h + 2 * j + 1] = f.y * s;
        }
      }
      store16(out + i * 16, v, sectors);
    }
  }
}

// Quantised rows to the rows that want them: 16 bytes of codes and one scale byte per thread.
__global__ void __launch_bounds__(256)
    mxfp4_gather_kernel(const uint4* __restrict__ src, const uint8_t* __restrict__ src_scales, int T_rows, int P, int sh,
                        const int32_t* __restrict__ rows, long n, uint4* __restrict__ codes,
                        uint8_t* __restrict__ scales, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i0 = (long)blockIdx.x * blockDim.x + threadIdx.x; i0 < n; i0 += kUnroll * stride) {
    uint4 c[kUnroll];
    uint8_t b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      c[u] = make_uint4(0, 0, 0, 0);
      b[u] = 0;
      if (i < n) {
        const long r = div_idx(i, P, sh);
        const int t = __ldg(rows + r);
        if (t >= 0 && t < T_rows) {
          const long at = (long)t * P + (i - r * P);
          c[u] = __ldg(src + at);
          b[u] = __ldg(src_scales + at);
        } else if (status != nullptr) {
          atomicOr(status, MOE_STATUS_BAD_INDEX);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      if (i < n) {
        __stcs(codes + i, c[u]);
        __stcs(scales + i, b[u]);
      }
    }
  }
}

unsigned blocks_for(long n) { return (unsigned)((n + 256 * kUnroll - 1) / (256 * kUnroll)); }

// With rows that repeat, quantising each source row once into the workspace and copying the packed
// rows moves T (b + 17/32) + R 17/16 bytes a value instead of R (b + 17/32), most of the copies'
// reads from L2. Measured, 16384 bf16 rows of 2048 to 131072: 191 us in one kernel (the rows do not
// stay in L2 beside the output), 51 in two. Small calls take the single launch, and so do rows of a
// matrix without any, which are all zero and reported.
bool in_two(int T, int K, bool with_rows, long R) { return with_rows && T > 0 && R >= 2L * T && R * K >= (1L << 22); }

template <class T>
int quantize(const void* x, int Tr, int K, const int32_t* rows, int R, uint8_t* codes, uint8_t* scales, void* ws,
             int32_t* status, cudaStream_t s) {
  Carver c(ws);
  const bool two = in_two(Tr, K, rows != nullptr, R);
  uint8_t* q = two ? c.take<uint8_t>((size_t)Tr * (K / 2)) : codes;
  uint8_t* qs = two ? c.take<uint8_t>((size_t)Tr * (K / 32)) : scales;
  {
    const long n = (long)(two ? Tr : R) * (K / 8);
    ProfScope ps("mxfp4_quantize", s);
    const cudaError_t e = launch_pdl(mxfp4_quantize_kernel<T>, blocks_for(n), 256, 0, s, static_cast<const T*>(x), Tr, K,
                                     pow2_shift(K / 8), two ? nullptr : rows, n, reinterpret_cast<uint32_t*>(q), qs, status);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "mxfp4_quantize: %s", cudaGetErrorString(e));
    if (int rc = check_launch("mxfp4_quantize")) return rc;
  }
  if (!two) return MOE_OK;
  const long n = (long)R * (K / 32);
  // here a grid that loops was the faster one (29 us against 32)
  const unsigned grid = std::min(blocks_for(n), (unsigned)num_sms() * 8);
  ProfScope ps("mxfp4_gather", s);
  const cudaError_t e = launch_pdl(mxfp4_gather_kernel, grid, 256, 0, s, reinterpret_cast<const uint4*>(q),
                                   static_cast<const uint8_t*>(qs), Tr, K / 32, pow2_shift(K / 32), rows, n,
                                   reinterpret_cast<uint4*>(codes), scales, status);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "mxfp4_gather: %s", cudaGetErrorString(e));
  return check_launch("mxfp4_gather");
}

template <class T>
int dequantize(const uint8_t* codes, const uint8_t* scales, int R, int K, void* out, cudaStream_t s) {
  const long n = (long)R * (K / 16);
  ProfScope ps("mxfp4_dequantize", s);
  const cudaError_t e = launch_pdl(mxfp4_dequantize_kernel<T>, blocks_for(n), 256, 0, s,
                                   reinterpret_cast<const uint2*>(codes), scales, n, static_cast<T*>(out), aligned(out, 32));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "mxfp4_dequantize: %s", cudaGetErrorString(e));
  return check_launch("mxfp4_dequantize");
}

}  // namespace

size_t mxfp4_quantize_workspace(int T, int K, bool with_rows, int R) {
  if (!in_two(T, K, with_rows, R)) return 0;
  Carver c(nullptr);
  c.take<uint8_t>((size_t)T * (K / 2));
  c.take<uint8_t>((size_t)T * (K / 32));
  return align_up(c.used, 256);
}

int launch_mxfp4_quantize(const void* x, int dtype, int T, int K, const int32_t* rows, int R, uint8_t* codes,
                          uint8_t* scales, void* ws, int32_t* status, cudaStream_t s) {
  if (dtype == MOE_F32) return quantize<float>(x, T, K, rows, R, codes, scales, ws, status, s);
  if (dtype == MOE_BF16) return quantize<__nv_bfloat16>(x, T, K, rows, R, codes, scales, ws, status, s);
  return quantize<__half>(x, T, K, rows, R, codes, scales, ws, status, s);
}

int launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int R, int K, int dtype, void* out,
                            cudaStream_t s) {
  if (dtype == MOE_F32) return dequantize<float>(codes, scales, R, K, out, s);
  if (dtype == MOE_BF16) return dequantize<__nv_bfloat16>(codes, scales, R, K, out, s);
  return dequantize<__half>(codes, scales, R, K, out, s);
}

}  // namespace moe
