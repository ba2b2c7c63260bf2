// 8-bit rows and weights with a float32 scale per block: quantisation and its inverse, the root-mean-square
// norm that ends in such rows, and the copy of such rows into expert order.
//
// A block is 128 neighbouring values of a row, or 128 x 128 values of a matrix (blocks at the edges are
// smaller). With m the block's largest magnitude,
//   s = max(m / 448, 2^-126),   code = e4m3 of v * (1 / s)   (nearest, ties to even, above 448 to 448)
// in float32: m / 448 and 1 / s are rounded once each, and so is the product in front of the 8-bit rounding.
// 448 is the largest e4m3 value; 2^-126 keeps 1 / s finite (a block of zeros has it). A block that holds an
// infinity or a NaN has the scale NaN and codes 0.
//
// Everything here moves each byte once and is bound by memory. A lane holds eight neighbouring values, 16
// lanes a block of a row, so its largest magnitude is four shuffles of the values' bits as integers
// (magnitudes of floats order like integers, and infinity and NaN come out on top without a test).
#include <algorithm>

#include "fp8.cuh"
#include "values.cuh"

namespace moe {
namespace {

using fp8::BLOCK;
constexpr int UNITS = BLOCK / 8;        // lanes of a block
constexpr int kUnroll = 2;

struct Scale {
  float scale, inv;                     // s, and 1 / s (0 for a block that is not finite)
};
__device__ __forceinline__ Scale scale_of(uint32_t most) {
  if (most >= 0x7f800000u) return Scale{__uint_as_float(0x7fc00000u), 0.0f};
  Scale s;
  s.scale = fmaxf(__uint_as_float(most) / 448.0f, __uint_as_float(0x00800000u));
  s.inv = 1.0f / s.scale;
  return s;
}

// Largest magnitude's bits over eight values and the 16 lanes of a block.
__device__ __forceinline__ uint32_t most8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t most_of_block(const float (&v)[8]) {
  uint32_t m = most8(v);
#pragma unroll
  for (int d = 1; d < UNITS; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], const Scale& s) {
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = v[j] * s.inv;
  const uint2 q = make_uint2(fp8::encode4(a[0], a[1], a[2], a[3]), fp8::encode4(a[4], a[5], a[6], a[7]));
  return s.inv == 0.0f ? make_uint2(0, 0) : q;      // an infinity times 0 is not 0
}

// ---- rows: blocks of 1 x 128 ------------------------------------------------------------

// Unit i: eight values of row i / (16 blocks); units past the row's end hold zeros, so that whole groups
// of 16 lanes share a block.
template <class T>
__global__ void __launch_bounds__(256)
    fp8_quantize_rows_kernel(const T* __restrict__ x, int K, int units, int sh, long n, uint8_t* __restrict__ codes,
                             float* __restrict__ scales) {
  const long stride = (long)gridDim.x * blockDim.x;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  for (long i0 = (long)blockIdx.x * blockDim.x + threadIdx.x; i0 - lane < n; i0 += kUnroll * stride) {
    float v[kUnroll][8];
    long at[kUnroll];                   // first value; -1: none
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride, r = div_idx(i < n ? i : 0, units, sh);
      const int c = (int)((i < n ? i : 0) - r * units) * 8;
      at[u] = i < n && c < K ? r * K + c : -1;
      if (at[u] >= 0) {
        load8(x + at[u], v[u]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      const Scale s = scale_of(most_of_block(v[u]));
      if (at[u] >= 0) *reinterpret_cast<uint2*>(codes + at[u]) = encode8(v[u], s);
      if (i < n && i % UNITS == 0) scales[i / UNITS] = s.scale;
    }
  }
}

// ---- weights: blocks of 128 x 128 ---------------------------------------------------------

// A CTA holds a block in registers: 16 lanes a row, 16 rows at a time, eight times.
template <class T>
__global__ void __launch_bounds__(256)
    fp8_quantize_blocks_kernel(const T* __restrict__ x, int N, int K, int nb, int kb, uint8_t* __restrict__ codes,
                               float* __restrict__ scales) {
  __shared__ uint32_t warp_most[8];
  pdl_wait();
  pdl_trigger();
  const long b = blockIdx.x, mat = b / ((long)nb * kb);
  const int local = (int)(b - mat * nb * kb), rb = local / kb, cb = local - rb * kb;
  const int c = cb * BLOCK + (threadIdx.x & 15) * 8, r0 = rb * BLOCK + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = r0 + 16 * p;
    if (r < N && c < K) {
      load8(x + (mat * N + r) * K + c, v[p]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p][j] = 0.0f;
    }
  }
#pragma unroll
  for (int p = 0; p < 8; ++p) m = max(m, most8(v[p]));
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) warp_most[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, warp_most[w]);
  const Scale s = scale_of(m);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = r0 + 16 * p;
    if (r < N && c < K) *reinterpret_cast<uint2*>(codes + (mat * N + r) * K + c) = encode8(v[p], s);
  }
  if (threadIdx.x == 0) scales[b] = s.scale;
}

// ---- values back ----------------------------------------------------------------------------

// 16 codes per thread. N = 0: a scale for each row and 128 values; else rows come in matrices of N, with
// a scale for 128 x 128.
template <class T>
__global__ void __launch_bounds__(256)
    fp8_dequantize_kernel(const uint4* __restrict__ codes, const float* __restrict__ scales, int units, int sh, int kb, int N,
                          long n, T* __restrict__ out, bool sectors) {
  pdl_wait();
  pdl_trigger();
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i0 = (long)blockIdx.x * blockDim.x + threadIdx.x; i0 < n; i0 += kUnroll * stride) {
    uint4 c[kUnroll];
    float s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      if (i >= n) break;
      const long r = div_idx(i, units, sh);
      const int b = (int)(i - r * units) >> 3;          // 16 values of 128: eight units a block
      long row = r;
      if (N > 0) {
        const long mat = r / N;
        row = mat * ((N + BLOCK - 1) / BLOCK) + (r - mat * N) / BLOCK;
      }
      c[u] = __ldg(codes + i);
      s[u] = __ldg(scales + row * kb + b);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long i = i0 + u * stride;
      if (i >= n) break;
      const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
      float v[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 f = fp8::decode4(w[j]);
        v[4 * j] = f.x * s[u];
        v[4 * j + 1] = f.y * s[u];
        v[4 * j + 2] = f.z * s[u];
        v[4 * j + 3] = f.w * s[u];
      }
      store16(out + i * 16, v, sectors);
    }
  }
}

// ---- norm -------------------------------------------------------------------------------------

struct NormArgs {
  const void* x;
  const void* residual;         // null: none
  const void* weight;
  float eps;
  int T, H;
  uint8_t* codes;
  float* scales;
  void* sum;                    // x + residual, with a residual
  void* normed;                 // null: not wanted
};

// h = x + residual, rounded to T as the stream keeps it; n = h / sqrt(mean of h^2 + eps) * weight in float32.
// The sum may be written over either of them and the normed rows over x, so both come by ordinary loads.
template <class T>
__device__ __forceinline__ void take8(const NormArgs& a, long at, float (&h)[8]) {
  load8<true>(static_cast<const T*>(a.x) + at, h);
  if (a.residual != nullptr) {
    float r[8];
    load8<true>(static_cast<const T*>(a.residual) + at, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = to_float(from_float<T>(h[j] + r[j]));
  }
}

template <class T>
__device__ __forceinline__ void finish8(const NormArgs& a, long row, int c, bool in, const float (&h)[8], float inv_rms) {
  float n[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) n[j] = 0.0f;
  if (in) {
    float w[8];
    load8(static_cast<const T*>(a.weight) + c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = h[j] * inv_rms * w[j];
  }
  const Scale s = scale_of(most_of_block(n));
  if (!in) return;
  const long at = row * a.H + c;
  *reinterpret_cast<uint2*>(a.codes + at) = encode8(n, s);
  if (a.normed != nullptr) store8(static_cast<T*>(a.normed) + at, n);
  if (c % BLOCK == 0) a.scales[row * ((a.H + BLOCK - 1) / BLOCK) + c / BLOCK] = s.scale;
}

// G threads (a warp or the CTA) take a row and hold V times eight values of it each.
template <class T, int G, int V>
__global__ void __launch_bounds__(256) rms_norm_fp8_kernel(const NormArgs a) {
  __shared__ float part[8];
  const int tid = threadIdx.x % G;
  pdl_wait();
  pdl_trigger();
  const long row = (long)blockIdx.x * (256 / G) + threadIdx.x / G;
  if (G == 32 && row >= a.T) return;
  float h[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (tid + v * G) * 8;
    if (c < a.H) {
      take8<T>(a, row * a.H + c, h[v]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = 0.0f;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (tid + v * G) * 8;
    if (a.residual != nullptr && c < a.H) store8(static_cast<T*>(a.sum) + row * a.H + c, h[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += h[v][j] * h[v][j];
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (G > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) ss += part[w];
  }
  const float inv_rms = 1.0f / sqrtf(ss / (float)a.H + a.eps);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (tid + v * G) * 8;
    finish8<T>(a, row, c, c < a.H, h[v], inv_rms);
  }
}

// Rows of any width: read twice.
template <class T>
__global__ void __launch_bounds__(256) rms_norm_fp8_wide_kernel(const NormArgs a) {
  __shared__ float part[8];
  pdl_wait();
  pdl_trigger();
  const long row = blockIdx.x;
  float ss = 0.0f;
  for (int c = threadIdx.x * 8; c < a.H; c += 256 * 8) {
    float h[8];
    take8<T>(a, row * a.H + c, h);
    if (a.residual != nullptr) store8(static_cast<T*>(a.sum) + row * a.H + c, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += h[j] * h[j];
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ss += part[w];
  const float inv_rms = 1.0f / sqrtf(ss / (float)a.H + a.eps);
  const T* src = static_cast<const T*>(a.residual != nullptr ? a.sum : a.x);     // the sum may lie where the residual was
  const int whole = (a.H + BLOCK - 1) / BLOCK * BLOCK;
  for (int c0 = 0; c0 < whole; c0 += 256 * 8) {
    const int c = c0 + threadIdx.x * 8;
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = 0.0f;
    if (c < a.H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = to_float(src[row * a.H + c + j]);
    }
    finish8<T>(a, row, c, c < a.H, h, inv_rms);
  }
}

// ---- 8-bit rows into expert order ---------------------------------------------------------------

// 16 bytes of codes per thread, and the scale of the block that starts there. A CTA takes 1024 neighbouring pieces a turn,
// whose loads are under way together, and what it writes is one stretch of memory: 131072 rows of 2048, 277 MB, 60 us (4.6
// TB/s written; filling the same memory takes 75); with pieces a grid apart 90, with a CTA for each turn 74.
__global__ void __launch_bounds__(256)
    fp8_gather_kernel(const uint4* __restrict__ src, const float* __restrict__ src_scales, int T, int units, int sh, int kb,
                      const int32_t* __restrict__ ids, const int32_t* __restrict__ offsets, int E, int S,
                      uint4* __restrict__ out, float* __restrict__ scales, int32_t* status) {
  constexpr int U = 4;
  pdl_wait();
  pdl_trigger();
  const int rows = __ldg(offsets + E);
  if (blockIdx.x == 0 && threadIdx.x == 0 && (rows < 0 || rows > S) && status != nullptr) atomicOr(status, MOE_STATUS_BAD_INDEX);
  const long n = (long)min(max(rows, 0), S) * units;
  const long stride = blockDim.x;
  for (long i0 = (long)blockIdx.x * blockDim.x * U + threadIdx.x; i0 < n; i0 += (long)U * gridDim.x * blockDim.x) {
    uint4 c[U];
    float s[U];
    long r[U];
    int b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + u * stride;
      c[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.0f;
      if (i >= n) continue;
      r[u] = div_idx(i, units, sh);
      b[u] = (int)(i - r[u] * units);
      const int t = __ldg(ids + r[u]);
      if (t >= 0 && t < T) {
        c[u] = __ldg(src + (long)t * units + b[u]);
        if ((b[u] & 7) == 0) s[u] = __ldg(src_scales + (long)t * kb + (b[u] >> 3));
      } else if (status != nullptr) {
        atomicOr(status, MOE_STATUS_BAD_INDEX);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + u * stride;
      if (i >= n) break;
      __stcs(out + i, c[u]);
      if ((b[u] & 7) == 0) __stcs(scales + r[u] * kb + (b[u] >> 3), s[u]);
    }
  }
}

// ---- host -----------------------------------------------------------------------------------------

unsigned blocks_for(long n, int unroll) { return (unsigned)std::min((n + 256L * unroll - 1) / (256L * unroll), 0x7fffffffL); }

int done(cudaError_t e, const char* name) {
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

template <class T>
int quantize(const void* x, int M, int N, int K, bool blocks, uint8_t* codes, float* scales, cudaStream_t s) {
  const char* name = "fp8_quantize";
  const int kb = fp8::blocks(K), nb = fp8::blocks(N);
  ProfScope ps(name, s);
  if (blocks)
    return done(launch_pdl(fp8_quantize_blocks_kernel<T>, (unsigned)((long)M * nb * kb), 256, 0, s, static_cast<const T*>(x), N, K,
                           nb, kb, codes, scales),
                name);
  const int units = kb * UNITS;
  const long n = (long)M * N * units;
  return done(launch_pdl(fp8_quantize_rows_kernel<T>, blocks_for(n, kUnroll), 256, 0, s, static_cast<const T*>(x), K, units,
                         pow2_shift(units), n, codes, scales),
              name);
}

template <class T>
int dequantize(const uint8_t* codes, const float* scales, int M, int N, int K, bool blocks, void* out, cudaStream_t s) {
  const char* name = "fp8_dequantize";
  const int units = K / 16;
  const long n = (long)M * N * units;
  ProfScope ps(name, s);
  return done(launch_pdl(fp8_dequantize_kernel<T>, blocks_for(n, kUnroll), 256, 0, s, reinterpret_cast<const uint4*>(codes), scales,
                         units, pow2_shift(units), fp8::blocks(K), blocks ? N : 0, n, static_cast<T*>(out), aligned(out, 32)),
              name);
}

template <class T, int G, int V>
int norm_as(const NormArgs& a, cudaStream_t s) {
  const char* name = "rms_norm_fp8";
  ProfScope ps(name, s);
  return done(launch_pdl(rms_norm_fp8_kernel<T, G, V>, (unsigned)(((long)a.T + 256 / G - 1) / (256 / G)), 256, 0, s, a), name);
}

template <class T>
int norm(const NormArgs& a, cudaStream_t s) {
  const int units = fp8::blocks(a.H) * UNITS;
  if (units <= 32) return norm_as<T, 32, 1>(a, s);
  if (units <= 64) return norm_as<T, 32, 2>(a, s);
  if (units <= 128) return norm_as<T, 32, 4>(a, s);
  if (units <= 256) return norm_as<T, 256, 1>(a, s);
  if (units <= 512) return norm_as<T, 256, 2>(a, s);
  if (units <= 1024) return norm_as<T, 256, 4>(a, s);
  const char* name = "rms_norm_fp8";
  ProfScope ps(name, s);
  return done(launch_pdl(rms_norm_fp8_wide_kernel<T>, (unsigned)a.T, 256, 0, s, a), name);
}

}  // namespace

int launch_fp8_quantize(const void* x, int dtype, int M, int N, int K, bool blocks, uint8_t* codes, float* scales, cudaStream_t s) {
  if (dtype == MOE_F32) return quantize<float>(x, M, N, K, blocks, codes, scales, s);
  if (dtype == MOE_BF16) return quantize<__nv_bfloat16>(x, M, N, K, blocks, codes, scales, s);
  return quantize<__half>(x, M, N, K, blocks, codes, scales, s);
}

int launch_fp8_dequantize(const uint8_t* codes, const float* scales, int M, int N, int K, bool blocks, int dtype, void* out,
                          cudaStream_t s) {
  if (dtype == MOE_F32) return dequantize<float>(codes, scales, M, N, K, blocks, out, s);
  if (dtype == MOE_BF16) return dequantize<__nv_bfloat16>(codes, scales, M, N, K, blocks, out, s);
  return dequantize<__half>(codes, scales, M, N, K, blocks, out, s);
}

int launch_rms_norm_fp8(const void* x, const void* residual, const void* weight, int dtype, int T, int H, float eps, uint8_t* codes,
                        float* scales, void* sum, void* normed, cudaStream_t s) {
  const NormArgs a{x, residual, weight, eps, T, H, codes, scales, sum, normed};
  if (dtype == MOE_F32) return norm<float>(a, s);
  if (dtype == MOE_BF16) return norm<__nv_bfloat16>(a, s);
  return norm<__half>(a, s);
}

int launch_fp8_gather_rows(const uint8_t* codes, const float* scales, const int32_t* ids, const int32_t* offsets, int T, int H, int E,
                           int S, uint8_t* out, float* out_scales, int32_t* status, cudaStream_t s) {
  const char* name = "fp8_gather_rows";
  const int units = H / 16;
  const unsigned grid = std::min(blocks_for((long)S * units, 4), (unsigned)num_sms() * 4);
  ProfScope ps(name, s);
  return done(launch_pdl(fp8_gather_kernel, grid, 256, 0, s, reinterpret_cast<const uint4*>(codes), scales, T, units,
                         pow2_shift(units), fp8::blocks(H), ids, offsets, E, S, reinterpret_cast<uint4*>(out), out_scales, status),
              name);
}

}  // namespace moe
