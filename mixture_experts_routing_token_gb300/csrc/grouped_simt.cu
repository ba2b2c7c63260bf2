// Products grouped by expert in float32, on the CUDA cores: every size and alignment.
//
//   ROWS   y[p, n]    = sum_k x[p, k] w[e, n, k]     (rows p of expert e)
//   GRADX  d_x[p, k]  = sum_n d_y[p, n] w[e, n, k]
//   GRADW  d_w[e, n, k] = sum over p of e of d_y[p, n] x[p, k]
//
// One CTA computes 64 x 64 outputs of one expert; 16 steps of the reduction at a time
// go through shared memory, each thread keeps 4 x 4 sums in registers.
// Products and sums are float32 fused multiply-adds in ascending order of the
// reduction index, so results do not depend on the launch.
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64, TK = 16, TT = 256;

enum { ROWS = 0, GRADX = 1, GRADW = 2 };

struct SimtParams {
  const float* a;       // x (ROWS), d_y (GRADX, GRADW)
  const float* b;       // w (ROWS, GRADX), x (GRADW)
  float* out;
  const int32_t* offsets;
  int S, K, N, E;
  int32_t* status;
};

template <int MODE>
__global__ void __launch_bounds__(TT) grouped_simt_kernel(const SimtParams P) {
  __shared__ float sa[TK][TM + 4], sb[TK][TN + 4];
  __shared__ grouped::Groups G;
  const int tid = threadIdx.x;
  const int cols = MODE == ROWS ? P.N : P.K;           // columns of the output
  const int NT = (cols + TN - 1) / TN;
  const int MT = (P.N + TM - 1) / TM;                  // GRADW: row tiles of an expert's output
  if (tid < 32)
    grouped::group_list(P.offsets, P.E, P.S,
                       [&](int rows) { return MODE == GRADW ? MT * NT : (rows + TM - 1) / TM * NT; }, G);
  __syncthreads();
  if (G.bad && blockIdx.x == 0 && tid == 0 && P.status) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  const float *A = P.a, *B = P.b;
  float* out = P.out;
  const int tx = tid & 15, ty = tid >> 4;
  for (int t = blockIdx.x; t < G.start[P.E]; t += gridDim.x) {
    const int e = grouped::find(G.start, P.E, t);
    const grouped::Span g = G.span(e);
    const int local = t - G.start[e];
    const int m0 = local / NT * TM, n0 = (local - local / NT * NT) * TN;
    const int red = MODE == ROWS ? P.K : MODE == GRADX ? P.N : g.rows();
    const int mcount = MODE == GRADW ? P.N : g.rows();
    float acc[4][4] = {};
    for (int r0 = 0; r0 < red; r0 += TK) {
      for (int i = tid; i < TM * TK; i += TT) {
        const int m = MODE == GRADW ? i % TM : i / TK, r = MODE == GRADW ? i / TM : i % TK;
        float v = 0.0f;
        if (m0 + m < mcount && r0 + r < red) {
          const long row = MODE == GRADW ? g.lo + r0 + r : g.lo + m0 + m;
          v = A[MODE == ROWS ? row * P.K + r0 + r : row * P.N + (MODE == GRADW ? m0 + m : r0 + r)];
        }
        sa[r][m] = v;
      }
      for (int i = tid; i < TN * TK; i += TT) {
        const int n = MODE == ROWS ? i / TK : i % TN, r = MODE == ROWS ? i % TK : i / TN;
        float v = 0.0f;
        if (n0 + n < cols && r0 + r < red) {
          const long row = MODE == ROWS ? (long)e * P.N + n0 + n : MODE == GRADX ? (long)e * P.N + r0 + r : g.lo + r0 + r;
          v = B[row * P.K + (MODE == ROWS ? r0 + r : n0 + n)];
        }
        sb[r][n] = v;
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
      if (m >= mcount) continue;
      const long row = MODE == GRADW ? (long)e * P.N + m : g.lo + m;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n < cols) out[row * cols + n] = acc[i][j];
      }
    }
  }
  if (MODE != GRADW)
    grouped::zero_unowned(out, G, P.E, P.S, cols, (long)blockIdx.x * TT + tid, (long)gridDim.x * TT);
}

template <int MODE>
int launch(const SimtParams& p, cudaStream_t s, const char* name) {
  const long cols = MODE == ROWS ? p.N : p.K, nt = (cols + TN - 1) / TN;
  const long tiles = MODE == GRADW ? (long)p.E * ((p.N + TM - 1) / TM) * nt : ((long)(p.S + TM - 1) / TM + p.E) * nt;
  const long most = (long)num_sms() * 8;
  ProfScope ps(name, s);
  grouped_simt_kernel<MODE><<<(unsigned)(tiles < most ? tiles : most), TT, 0, s>>>(p);
  return check_launch(name);
}

SimtParams params(const GroupedArgs& a, const void* left, const void* right, void* out) {
  return SimtParams{static_cast<const float*>(left), static_cast<const float*>(right), static_cast<float*>(out),
                    a.offsets, a.S, a.K, a.N, a.E, a.status};
}

}  // namespace

int launch_grouped_simt(const GroupedArgs& a, cudaStream_t s) {
  return launch<ROWS>(params(a, a.x, a.w, a.y), s, "grouped_gemm");
}

int launch_grouped_simt_dx(const GroupedArgs& a, cudaStream_t s) {
  return launch<GRADX>(params(a, a.d_y, a.w, a.d_x), s, "grouped_gemm_dx");
}

int launch_grouped_simt_dw(const GroupedArgs& a, cudaStream_t s) {
  return launch<GRADW>(params(a, a.d_y, a.x, a.d_w), s, "grouped_gemm_dw");
}

}  // namespace moe
