// Grouped product of 4-bit microscaled operands on the CUDA cores (float32 sums).
//
//   y[p, n] = sum over blocks b of 32 of 2^(sx + sw) sum in b of cx cw
// then, with the gate, silu(y[p, n]) y[p, N/2 + n]. One CTA computes 64 rows x 64
// columns of one expert (with the gate: 32 gate columns beside their 32 up columns);
// each step takes one block of 32 of the reduction through shared memory.
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64, TK = 32, TT = 256;

__device__ __forceinline__ float value4(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m < 4 ? 0.5f * (float)m : m == 4 ? 2.0f : m == 5 ? 3.0f : m == 6 ? 4.0f : 6.0f;
  return code & 8u ? -v : v;
}
__device__ __forceinline__ float scale8(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

template <bool SILU, class T>
__global__ void __launch_bounds__(TT) mxfp4_simt_kernel(const Mxfp4Args P) {
  __shared__ float sa[TK][TM + 4], sb[TK][TN + 4];
  __shared__ int start[MOE_MAX_EXPERTS + 1], bad;
  const int tid = threadIdx.x;
  const int cols = SILU ? P.N / 2 : P.N;
  constexpr int TC = SILU ? TN / 2 : TN;
  const int NT = (cols + TC - 1) / TC;
  if (tid < 32)
    grouped::tile_list(P.offsets, P.E, P.S, [&](int rows) { return (rows + TM - 1) / TM * NT; }, start, &bad);
  __syncthreads();
  if (bad && blockIdx.x == 0 && tid == 0 && P.status) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  T* out = static_cast<T*>(P.y);
  const int tx = tid & 15, ty = tid >> 4, KB = P.K / 32;
  for (int t = blockIdx.x; t < start[P.E]; t += gridDim.x) {
    const int e = grouped::find(start, P.E, t);
    const grouped::Span g = grouped::span(P.offsets, e, P.S);
    const int local = t - start[e];
    const int m0 = local / NT * TM, n0 = (local - local / NT * NT) * TC;
    float acc[4][4] = {};
    for (int kb = 0; kb < KB; ++kb) {
      for (int i = tid; i < TM * 16; i += TT) {
        const int m = i / 16, j = i % 16;
        float lo = 0.0f, hi = 0.0f;
        if (m0 + m < g.rows()) {
          const long row = g.lo + m0 + m;
          const float s = scale8(P.x_scales[row * KB + kb]);
          const uint32_t c = P.x[row * KB * 16 + kb * 16 + j];
          lo = value4(c & 15u) * s;
          hi = value4(c >> 4) * s;
        }
        sa[2 * j][m] = lo;
        sa[2 * j + 1][m] = hi;
      }
      for (int i = tid; i < TN * 16; i += TT) {
        const int c4 = i / 16, j = i % 16;
        // column c4 of the tile: with the gate, thread tx holds gate columns 2tx, 2tx + 1 and their up columns
        const int n = SILU ? n0 + (c4 >> 2) * 2 + (c4 & 1) : n0 + c4;
        float lo = 0.0f, hi = 0.0f;
        if (n < cols) {
          const long row = (long)e * P.N + n + (SILU && (c4 & 2) ? cols : 0);
          const float s = scale8(P.w_scales[row * KB + kb]);
          const uint32_t c = P.w[row * KB * 16 + kb * 16 + j];
          lo = value4(c & 15u) * s;
          hi = value4(c >> 4) * s;
        }
        sb[2 * j][c4] = lo;
        sb[2 * j + 1][c4] = hi;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < TK; ++r) {
        const float4 a4 = *reinterpret_cast<const float4*>(&sa[r][ty * 4]);
        const float4 b4 = *reinterpret_cast<const float4*>(&sb[r][tx * 4]);
        const float av[4] = {a4.x, a4.y, a4.z, a4.w}, bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + ty * 4 + i;
      if (m >= g.rows()) continue;
      T* dst = out + (long)(g.lo + m) * cols;
      if (SILU) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (n0 + tx * 2 + j < cols) dst[n0 + tx * 2 + j] = from_float<T>(silu(acc[i][j]) * acc[i][j + 2]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + tx * 4 + j < cols) dst[n0 + tx * 4 + j] = from_float<T>(acc[i][j]);
      }
    }
  }
  grouped::zero_unowned(out, P.offsets, P.E, P.S, cols, (long)blockIdx.x * TT + tid, (long)gridDim.x * TT);
}

template <bool SILU, class T>
int launch(const Mxfp4Args& a, cudaStream_t s) {
  const long cols = SILU ? a.N / 2 : a.N, nt = (cols + TN - 1) / TN * (SILU ? 2 : 1);
  const long tiles = ((long)(a.S + TM - 1) / TM + a.E) * nt, most = (long)num_sms() * 8;
  ProfScope ps("mxfp4_grouped_gemm", s);
  mxfp4_simt_kernel<SILU, T><<<(unsigned)(tiles < most ? tiles : most), TT, 0, s>>>(a);
  return check_launch("mxfp4_grouped_gemm");
}

}  // namespace

int launch_mxfp4_grouped(const Mxfp4Args& a, cudaStream_t s) {
  if (a.out_dtype == MOE_F32) return a.silu ? launch<true, float>(a, s) : launch<false, float>(a, s);
  if (a.out_dtype == MOE_BF16) return a.silu ? launch<true, __nv_bfloat16>(a, s) : launch<false, __nv_bfloat16>(a, s);
  return a.silu ? launch<true, __half>(a, s) : launch<false, __half>(a, s);
}

}  // namespace moe
