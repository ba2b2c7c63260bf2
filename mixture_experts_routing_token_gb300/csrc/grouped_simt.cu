// Products grouped by expert in float32, on the CUDA cores: small sizes, few rows per expert, narrow
// outputs, and operands that hold infinities, NaN or very large values (then launched behind the
// tensor-core kernel, with the flags that it gives way to).
//
//   ROWS   y[p, n]    = sum_k x[p, k] w[e, n, k]     (rows p of expert e)
//   GRADX  d_x[p, k]  = sum_n d_y[p, n] w[e, n, k]
//   GRADW  d_w[e, n, k] = sum over p of e of d_y[p, n] x[p, k]
//
// One CTA of 64 threads computes 64 x 64 outputs of one expert, 8 x 8 per thread (where experts
// have few rows 16 x 64, 2 x 8): a step of the reduction reads 16 values from shared memory for 64
// fused multiply-adds. 16 steps at a time go through one of two buffers; the next 16 are in
// registers on their way meanwhile, so a turn has one barrier and no exposed load. The multiply-adds
// are issued in pairs (fma.f32x2, two columns), which leaves issue slots for everything else. Products
// and sums are float32 in ascending order of the reduction index, so results do not depend on the
// launch. Bound by shared memory and the FMA pipes (45 TFLOP/s at 8000 rows of [2048, 1024]). With few
// rows by the issue and latency of the weights' loads, a word at a time and one turn ahead: 128 rows, 32
// experts of [2048, 1024], 116 us for 268 MB, 2.3 TB/s.
#include <algorithm>

#include "grouped.cuh"

namespace moe {
namespace {

constexpr int TN = 64, TK = 16, TT = 64;

enum { ROWS = 0, GRADX = 1, GRADW = 2 };

struct SimtParams {
  const float* a;       // x (ROWS), d_y (GRADX, GRADW)
  const float* b;       // w (ROWS, GRADX), x (GRADW)
  float* out;
  const int32_t* offsets;
  int S, K, N, E;
  int parts, chunk;     // the reduction in `parts` pieces of `chunk` (row outputs): piece k goes to partial + k S cols
  float* partial;
  const int* flags;     // null, or grouped::any_flag must hold for the kernel to do anything
  int32_t* status;
};

template <int MODE, int TM>
__global__ void __launch_bounds__(TT) grouped_simt_kernel(const SimtParams P) {
  constexpr int LA = TM * TK / TT, LB = TN * TK / TT;      // values of the operands a thread moves per turn
  constexpr int MR = TM / 8;                               // rows of a thread's sums
  __shared__ __align__(16) float sa[2][TK][TM + 4], sb[2][TK][TN + 4];
  __shared__ grouped::Groups G;
  const int tid = threadIdx.x;
  const int cols = MODE == ROWS ? P.N : P.K;           // columns of the output
  const int NT = (cols + TN - 1) / TN;
  const int MT = (P.N + TM - 1) / TM;                  // GRADW: row tiles of an expert's output
  if (P.flags != nullptr && !__syncthreads_or(grouped::any_flag<TT>(P.flags, tid))) return;
  if (tid < 32)
    grouped::group_list(P.offsets, P.E, P.S,
                       [&](int rows) { return MODE == GRADW ? MT * NT : (rows + TM - 1) / TM * NT; }, G);
  __syncthreads();
  if (G.bad && blockIdx.x == 0 && tid == 0 && P.status) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  const float *A = P.a, *B = P.b;
  const int parts = MODE == GRADW ? 1 : P.parts;
  const int tx = tid & 7, ty = tid >> 3;
  const int total = G.start[P.E] * parts;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int t = parts == 1 ? u : u / parts, part = u - t * parts;
    const int e = grouped::find(G.start, P.E, t);
    const grouped::Span g = G.span(e);
    const int local = t - G.start[e];
    const int m0 = local / NT * TM, n0 = (local - local / NT * NT) * TN;
    const int whole = MODE == ROWS ? P.K : MODE == GRADX ? P.N : g.rows();
    const int begin = parts == 1 ? 0 : part * P.chunk, red = parts == 1 ? whole : min(whole, begin + P.chunk);
    float* out = parts == 1 ? P.out : P.partial + (long)part * P.S * cols;
    const int mcount = MODE == GRADW ? P.N : g.rows();
    // Thread t moves values i = t, t + 64, ...: along the operand's contiguous index within a warp.
    // Reduction-contiguous (x, w, d_y rows): r = t % 16, row t / 16 + 4 q; else column t % width,
    // r = t / width + q 64 / width.
    constexpr bool A_RED = MODE != GRADW, B_RED = MODE == ROWS;
    constexpr int A_TURN = A_RED ? TT / TK : TT / TM, B_TURN = B_RED ? TT / TK : TT / TN;
    const int ra = A_RED ? tid % TK : tid / TM, ma = A_RED ? tid / TK : tid % TM;
    const int rb = B_RED ? tid % TK : tid / TN, nb = B_RED ? tid / TK : tid % TN;
    const long lda = MODE == ROWS ? P.K : P.N, ldb = P.K;
    const float* at = A + (A_RED ? (long)(g.lo + m0 + ma) * lda + ra : (long)(g.lo + ra) * lda + m0 + ma);
    const float* bt = B + (MODE == ROWS    ? ((long)e * P.N + n0 + nb) * ldb + rb
                           : MODE == GRADX ? ((long)e * P.N + rb) * ldb + n0 + nb
                                           : (long)(g.lo + rb) * ldb + n0 + nb);
    float pa[LA], pb[LB];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int q = 0; q < LA; ++q) {
        const bool in = A_RED ? m0 + ma + A_TURN * q < mcount && r0 + ra < red
                              : m0 + ma < mcount && r0 + ra + A_TURN * q < red;
        pa[q] = in ? __ldg(at + (A_RED ? A_TURN * q * lda + r0 : (long)(r0 + A_TURN * q) * lda)) : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < LB; ++q) {
        const bool in = B_RED ? n0 + nb + B_TURN * q < cols && r0 + rb < red
                              : n0 + nb < cols && r0 + rb + B_TURN * q < red;
        pb[q] = in ? __ldg(bt + (B_RED ? B_TURN * q * ldb + r0 : (long)(r0 + B_TURN * q) * ldb)) : 0.0f;
      }
    };
    auto put = [&](int buf) {
#pragma unroll
      for (int q = 0; q < LA; ++q) sa[buf][A_RED ? ra : ra + A_TURN * q][A_RED ? ma + A_TURN * q : ma] = pa[q];
#pragma unroll
      for (int q = 0; q < LB; ++q) sb[buf][B_RED ? rb : rb + B_TURN * q][B_RED ? nb + B_TURN * q : nb] = pb[q];
    };
    uint64_t acc[MR][4] = {};       // pairs of columns
    fetch(begin);
    __syncthreads();       // the previous tile's last reads
    put(0);
    __syncthreads();
    int buf = 0;
    for (int r0 = begin; r0 < red; r0 += TK, buf ^= 1) {
      const bool more = r0 + TK < red;
      if (more) fetch(r0 + TK);
#pragma unroll
      for (int r = 0; r < TK; ++r) {
        float av[MR];
        if constexpr (MR == 8) {
          const float4 a0 = *reinterpret_cast<const float4*>(&sa[buf][r][ty * 8]);
          const float4 a1 = *reinterpret_cast<const float4*>(&sa[buf][r][ty * 8 + 4]);
          av[0] = a0.x; av[1] = a0.y; av[2] = a0.z; av[3] = a0.w;
          av[4] = a1.x; av[5] = a1.y; av[6] = a1.z; av[7] = a1.w;
        } else {
          const float2 a0 = *reinterpret_cast<const float2*>(&sa[buf][r][ty * 2]);
          av[0] = a0.x; av[1] = a0.y;
        }
        const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&sb[buf][r][tx * 4]);
        const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&sb[buf][r][tx * 4 + 32]);
        const uint64_t bv[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          uint64_t aa;
          asm("mov.b64 %0, {%1, %1};" : "=l"(aa) : "f"(av[i]));
#pragma unroll
          for (int j = 0; j < 4; ++j) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i][j]) : "l"(aa), "l"(bv[j]));
        }
      }
      if (more) {
        put(buf ^ 1);
        __syncthreads();
      }
    }
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      const int m = m0 + ty * MR + i;
      if (m >= mcount) continue;
      const long row = MODE == GRADW ? (long)e * P.N + m : g.lo + m;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int n = n0 + tx * 4 + (j & 3) + (j >> 2) * 32;
        const uint64_t pair = acc[i][j >> 1];
        if (n < cols) out[row * cols + n] = __uint_as_float((uint32_t)(j & 1 ? pair >> 32 : pair));
      }
    }
  }
  if (MODE != GRADW && parts == 1)
    grouped::zero_unowned(P.out, G, P.E, P.S, cols, (long)blockIdx.x * TT + tid, (long)gridDim.x * TT);
}

// out = the pieces' sum, in order; 0 for rows that no group owns.
__global__ void __launch_bounds__(256) grouped_join_kernel(const float* __restrict__ partial, int parts, const int32_t* offsets,
                                                           int E, int S, int cols, float* __restrict__ out) {
  __shared__ grouped::Groups G;
  if (threadIdx.x < 32) grouped::group_list(offsets, E, S, [](int) { return 0; }, G);
  __syncthreads();
  const long first = (long)G.off[0] * cols, last = (long)G.off[E] * cols, n = (long)S * cols;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
    float v = 0.0f;
    if (i >= first && i < last)
      for (int k = 0; k < parts; ++k) v += __ldg(partial + k * n + i);
    out[i] = v;
  }
}

// Rows per tile: 16 where experts have few, so that CTAs mostly stream weights (128 rows, 32 experts of
// [2048, 1024]: 128 us instead of 234; 19 rows per expert 176 / 187, 32 rows 244 / 200).
int tile_rows(int S, int E) { return S <= 16L * E ? 16 : 64; }
long resident(int TM, int sms) { return (long)sms * (TM == 64 ? 6 : 11); }

// Pieces of the reduction, of 128 steps at least: as many as make four times the CTAs that fit the GPU
// (a tile alone takes a microsecond for 16 steps, however idle the rest, and tiles that are all resident
// leave some schedulers two warps and others none). 1685 rows, 58 experts of [344, 2944]: 206 us, with
// one time the CTAs 373, with two 239; 2000 rows, 32 experts of [512, 512]: 52 us, with one 70, with pieces
// of 256 steps 56.
constexpr int kSms = 152;       // a GB300's, so that workspace sizes and sums do not depend on the device asked
int reduction_parts(int S, int E, long cols, int R) {
  const int TM = tile_rows(S, E);
  const long tiles = (((long)S + TM - 1) / TM + std::min(S, E)) * ((cols + TN - 1) / TN);
  const long parts = std::min(std::min(4 * resident(TM, kSms) / tiles, (long)R / 128), 16L);
  return parts < 2 || S * cols * parts > (1L << 24) ? 1 : (int)parts;
}

template <int MODE, int TM>
int launch_tiles(const SimtParams& p, cudaStream_t s, const char* name) {
  const long cols = MODE == ROWS ? p.N : p.K, nt = (cols + TN - 1) / TN;
  const long tiles = MODE == GRADW ? (long)p.E * ((p.N + TM - 1) / TM) * nt
                                   : ((long)(p.S + TM - 1) / TM + p.E) * nt * p.parts;
  const long full = resident(TM, num_sms());
  ProfScope ps(name, s);
  grouped_simt_kernel<MODE, TM><<<(unsigned)std::min(tiles, p.flags ? full : full * 16), TT, 0, s>>>(p);
  return check_launch(name);
}

template <int MODE>
int launch(SimtParams& p, cudaStream_t s, const char* name) {
  const int cols = MODE == ROWS ? p.N : p.K, R = MODE == ROWS ? p.K : p.N;
  p.parts = MODE == GRADW || p.flags ? 1 : reduction_parts(p.S, p.E, cols, R);
  p.chunk = ((R + p.parts - 1) / p.parts + TK - 1) / TK * TK;
  int rc;
  if (MODE != GRADW && p.flags == nullptr && tile_rows(p.S, p.E) == 16) rc = launch_tiles<MODE, 16>(p, s, name);
  else rc = launch_tiles<MODE, 64>(p, s, name);
  if (rc || p.parts == 1) return rc;
  const long n = (long)p.S * cols;
  ProfScope ps("grouped_join", s);
  grouped_join_kernel<<<(unsigned)std::min((n + 255) / 256, (long)num_sms() * 8), 256, 0, s>>>(p.partial, p.parts, p.offsets, p.E,
                                                                                         p.S, cols, p.out);
  return check_launch("grouped_join");
}

SimtParams params(const GroupedArgs& a, const void* left, const void* right, void* out, const int* flags) {
  return SimtParams{static_cast<const float*>(left), static_cast<const float*>(right), static_cast<float*>(out),
                    a.offsets, a.S, a.K, a.N, a.E, 1, 0, static_cast<float*>(a.ws), flags, a.status};
}

}  // namespace

size_t grouped_simt_workspace(int S, int K, int N, int E, bool fwd) {
  if (S < 1 || K < 1 || N < 1) return 0;     // nothing is launched
  const long cols = fwd ? N : K;
  const int parts = reduction_parts(S, E, cols, fwd ? K : N);
  return parts == 1 ? 0 : align_up((size_t)S * cols * parts * sizeof(float), 256);
}

int launch_grouped_simt(const GroupedArgs& a, const int* flags, cudaStream_t s) {
  SimtParams p = params(a, a.x, a.w, a.y, flags);
  return launch<ROWS>(p, s, "grouped_gemm");
}

int launch_grouped_simt_dx(const GroupedArgs& a, const int* flags, cudaStream_t s) {
  SimtParams p = params(a, a.d_y, a.w, a.d_x, flags);
  return launch<GRADX>(p, s, "grouped_gemm_dx");
}

int launch_grouped_simt_dw(const GroupedArgs& a, const int* flags, cudaStream_t s) {
  SimtParams p = params(a, a.d_y, a.x, a.d_w, flags);
  return launch<GRADW>(p, s, "grouped_gemm_dw");
}

}  // namespace moe
