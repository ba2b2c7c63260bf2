// Products of 8-bit rows grouped by expert (tcgen05.mma.kind::f8f6f4, M = 128 x N = 256 or 128 x K = 32, float32 accumulators in
// TMEM), with a scale for every 128 values of a row and 128 x 128 of a matrix:
//
//   y[p, n] = sum over blocks b of sx[p, b] sw[e, n / 128, b] sum over k in b of cx[p, k] cw[e, n, k]
//   (with the gate, silu(y[p, n]) y[p, N/2 + n])
//
// The scales are any float32, so the tensor cores cannot apply them. An accumulator holds one block (K = 128, four
// MMAs); the epilogue warps read it, multiply by sx sw (one float32 product) and add in registers, while the next block
// goes into the other accumulator. Sums are rounded to nearest every 128 terms, and only the 128 inside a block see the
// tensor cores' truncating additions.
//
// One CTA per SM takes tiles of 128 rows of x and 256 of w (128 where there are few, see launch) by turns; with the gate
// half of these are gate rows and half the matching up rows, so a TMEM lane has both. Eight epilogue warps (four) keep 128
// sums a thread, for which the other warps of the wide form give up registers. Tiles of 256 rows on SM pairs load a third
// less and were no faster, for a pair's accumulator takes longer to come and go and an expert's last rows fill more of a
// tile: us, SM pairs / this, 131072 rows of 64 experts, [2816, 2048] with the gate 731 / 712, [2048, 1408] without
// 394 / 380; 64 rows an expert 96 / 66.
//
// 131072 rows, 64 experts of [2816, 2048] with the gate: 670 us on a cold GPU (2.26 PFLOP/s), 700 to 715 in a long run, which
// is 1,110 cycles a block of an SM. None of what was measured by itself takes as long: the four MMAs 512, the reads and sums
// 356, the operands' intake 730, half of an accumulator's way round (of which tensor memory holds two: MMAs until the
// epilogue knows, read and sums, hand-back, next issue) 700 to 770. Where the other 340 go is not known; without most of the
// sums and the scales' loads the time is a seventh less. At 64 rows an expert it is HBM: 66 us, 5.8 TB/s.
#include <algorithm>

#include "fp8.cuh"
#include "grouped.cuh"
#include "mxfp4_ptx.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                 // rows of x per tile
constexpr int KB = fp8::BLOCK;          // bytes of a row per step
constexpr int A_BYTES = BM * KB;
constexpr int W = 128;                  // rows of w (columns) of an epilogue warp
constexpr int EPI0 = 4;                 // the first of them
// Wide form: 168 registers a thread at launch (12 warps); the epilogue's eight take what the other four give back.
constexpr int LOW_REGS = 72, HIGH_REGS = 216;

// Tiles are 128 PARTS rows of w wide, with PARTS epilogue warps per TMEM lane quarter.
// 16-bit results leave through shared memory (store_rows), for which the wide form's ring has a stage less. Measured, us,
// single rows from registers and four stages / this: 131072 rows of 64 experts, [2816, 2048] with the gate 724 / 713,
// [2048, 1408] without 402 / 385; 64 rows an expert of the first 65.6 / 66.5. float32 results, twice as many bytes, stay
// with four stages.
template <int PARTS, class T>
struct Form {
  static constexpr int BN = W * PARTS;
  static constexpr int HALF = BN / 2;   // with the gate: gate rows, and as many up rows
  static constexpr int STAGE = A_BYTES + BN * KB;
  static constexpr int NSTAGE = PARTS == 1 ? 6 : sizeof(T) == 2 ? 3 : 4;
  static constexpr int EPI_WARPS = 4 * PARTS;
  static constexpr int THREADS = (EPI0 + EPI_WARPS) * 32;
  static constexpr int OUT_BYTES = sizeof(T) == 2 ? 4096 : 0;      // of a warp
  static constexpr int DSMEM = NSTAGE * STAGE + EPI_WARPS * OUT_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
};
static_assert(EPI0 * LOW_REGS + 8 * HIGH_REGS <= (EPI0 + 8) * 168, "registers");
constexpr uint64_t DRAIN_NS = 2000000000ull;

struct Params {
  const int32_t* offsets;
  const float* x_scales;
  const float* w_scales;
  int S, E;
  int kb, nb;       // blocks along K and N
  int cols;         // of y
  int NT;
  void* y;
  int vec;
  int32_t* status;
  uint64_t wait_ns;
};

struct Tile {
  int e, m, n;
  grouped::Span g;
};

__device__ __forceinline__ int mtiles(int rows) { return (rows + BM - 1) / BM; }

// Tiles of an expert that run together share the operand with fewer tiles, which stays in L2, while the other one is
// walked once.
__device__ __forceinline__ Tile tile_at(int t, int& e, const grouped::Groups& G, const Params& P) {
  Tile d;
  e = grouped::find_from(G.start, e, t);
  d.e = e;
  d.g = G.span(e);
  const int local = t - G.start[e], mt = mtiles(d.g.rows());
  if (mt > P.NT) {
    d.m = grouped::quick_div(local, P.NT);
    d.n = local - d.m * P.NT;
  } else {
    d.n = grouped::quick_div(local, mt);
    d.m = local - d.n * mt;
  }
  return d;
}

// A thread's scales of one block.
struct Scales {
  float x, g, u0, u1;       // the row's; the columns': all of them, or the gate's, and of the up columns before and after `edge`
};

template <bool SILU, class T, int PARTS>
__global__ void __launch_bounds__(Form<PARTS, T>::THREADS, 1)
    fp8_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmY, const Params P) {
  using F = Form<PARTS, T>;
  constexpr int BN = F::BN, HALF = F::HALF, STAGE = F::STAGE, NSTAGE = F::NSTAGE, EPI_WARPS = F::EPI_WARPS;
  __shared__ __align__(8) uint64_t full_bar[NSTAGE], empty_bar[NSTAGE];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ grouped::Groups G;
  extern __shared__ uint8_t dsmem_raw[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t dsmem = (ptx::smem_u32(dsmem_raw) + 1023u) & ~1023u;
  auto st = [&](int s) { return dsmem + (uint32_t)(s * STAGE); };
  volatile int* abort_p = &abort_flag;

  if (tid == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&tfull_bar[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&tempty_bar[b]), EPI_WARPS);
    }
    ptx::mbar_init(ptx::smem_u32(&drain_bar), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmX);
    ptx::prefetch_tmap(&tmW);
  }
  if (warp == 1) ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), F::TMEM_COLS);
  pdl_wait();          // the offsets and operands may be the previous kernel's output
  pdl_trigger();
  if (warp == 2)
    grouped::group_list(P.offsets, P.E, P.S, [&](int rows) { return mtiles(rows) * P.NT; }, G);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int total = G.start[P.E];

  if (PARTS == 2 && warp < EPI0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LOW_REGS));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = (int)blockIdx.x, e = 0; t < total && ok; t += (int)gridDim.x) {
        const Tile ti = tile_at(t, e, G, P);
        const int a_row = ti.g.lo + ti.m * BM;
        const int b_row = SILU ? ti.n * HALF : ti.n * BN;
        for (int k = 0; k < P.kb; ++k) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb = ptx::smem_u32(&full_bar[stage]);
          ptx::mbar_arrive_expect_tx(fb, STAGE);
          ptx::tma_load_3d(st(stage), &tmX, k * KB, a_row, 0, fb);
          ptx::tma_load_3d(st(stage) + A_BYTES, &tmW, k * KB, b_row, ti.e, fb);
          if (SILU) ptx::tma_load_3d(st(stage) + A_BYTES + HALF * KB, &tmW, k * KB, P.cols + b_row, ti.e, fb);
          if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (ptx::elect_one()) {
      constexpr uint32_t IDESC = fp8::idesc(BM, BN);
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int t = (int)blockIdx.x; t < total && ok; t += (int)gridDim.x) {
        for (int k = 0; k < P.kb; ++k) {
          ok = ptx::mbar_wait(ptx::smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_p, P.wait_ns) &&
               ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), ph, abort_p, P.wait_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
          const uint64_t ad = ptx::sdesc_k128(st(stage)), bd = ptx::sdesc_k128(st(stage) + A_BYTES);
#pragma unroll
          for (int kk = 0; kk < KB / 32; ++kk) fp8::mma(d_tmem, ad + kk * 2, bd + kk * 2, IDESC, kk != 0);
          ptx::mma_commit(ptx::smem_u32(&tfull_bar[acc]));
          ptx::mma_commit(ptx::smem_u32(&empty_bar[stage]));
          if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
          if (++acc == 2) { acc = 0; aph ^= 1u; }
        }
      }
      ptx::mma_commit(ptx::smem_u32(&drain_bar));
      int dummy = 0;
      ptx::mbar_wait(ptx::smem_u32(&drain_bar), 0, &dummy, DRAIN_NS);
    }
  } else if (warp >= EPI0) {
    // ------------------------------------------------------------ epilogue
    if (PARTS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(HIGH_REGS));
    const int q = warp & 3;              // TMEM lane quarter this warp may read
    const int part = (warp - EPI0) >> 2;    // its columns
    const int row = q * 32 + lane;
    T* y = static_cast<T*>(P.y);
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    // where a tile's scales are; `next` is loaded a block ahead, a tile's first one before the last tile's results are
    // stored
    const float *xs, *wg, *wu0, *wu1;
    int c0, edge;
    auto locate = [&](const Tile& ti) {
      const int r = ti.g.lo + ti.m * BM + row;
      // first columns (rows of w) of this thread's sums: W of them, or W / 2 of the gate and as many up ones
      c0 = SILU ? ti.n * HALF + part * (W / 2) : ti.n * BN + part * W;
      const float* ws = P.w_scales + (long)ti.e * P.nb * P.kb;
      xs = P.x_scales + (long)min(r, P.S - 1) * P.kb;
      wg = ws + (long)min(c0 / KB, P.nb - 1) * P.kb;
      // up columns: the half need not start where a block does
      const int up = SILU ? P.cols + c0 : 0;
      edge = KB - up % KB;                             // up columns before the next block
      wu0 = ws + (long)min(up / KB, P.nb - 1) * P.kb;
      wu1 = ws + (long)min(up / KB + 1, P.nb - 1) * P.kb;
    };
    auto load = [&](int k) {
      Scales s;
      s.x = __ldg(xs + k);
      s.g = __ldg(wg + k);
      s.u0 = SILU ? __ldg(wu0 + k) : 0.0f;
      s.u1 = SILU ? __ldg(wu1 + k) : 0.0f;
      return s;
    };
    Scales next{};
    int e = 0;
    Tile ti{};
    if ((int)blockIdx.x < total) {
      ti = tile_at((int)blockIdx.x, e, G, P);
      locate(ti);
      next = load(0);
    }
    for (int t = (int)blockIdx.x; t < total; t += (int)gridDim.x) {
      float sum[W];
#pragma unroll
      for (int j = 0; j < W; ++j) sum[j] = 0.0f;
      for (int k = 0; k < P.kb; ++k) {
        const Scales s = next;
        if (k + 1 < P.kb) next = load(k + 1);
        const float g = s.x * s.g, u0 = s.x * s.u0, u1 = s.x * s.u1;
        // whole warps go on or stop
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
#pragma unroll
        for (int c = 0; c < W; c += 16) {
          uint32_t v[16];
          ptx::tmem_ld16(taddr + (!SILU ? part * W + c : c < W / 2 ? part * (W / 2) + c : HALF + part * (W / 2) + c - W / 2), v);
          ptx::tmem_ld_wait16(v);
          if (c + 16 == W) {                // all read: the accumulator goes back
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&tempty_bar[acc]));
          }
          // a block's edge lies at a multiple of 16 columns
          const float f = !SILU || c < W / 2 ? g : c - W / 2 < edge ? u0 : u1;
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c + j] = fmaf(__uint_as_float(v[j]), f, sum[c + j]);
        }
        if (++acc == 2) { acc = 0; aph ^= 1u; }
      }
      if (!ok) break;
      const int col = c0;
      const int row_y = ti.g.lo + ti.m * BM + q * 32;      // this warp's first row, and how many it has
      const int nrows = ti.g.hi - row_y;
      if (t + (int)gridDim.x < total) {
        ti = tile_at(t + (int)gridDim.x, e, G, P);
        locate(ti);
        next = load(0);
      }
      T* row0 = y + (long)row_y * P.cols;
      auto result = [&](int i) { return SILU ? mx::silu_fast(sum[i]) * sum[(W / 2 + i) % W] : sum[i]; };
      if constexpr (sizeof(T) == 2) {
        const uint32_t buf = dsmem + NSTAGE * STAGE + (warp - EPI0) * F::OUT_BYTES;
#pragma unroll
        for (int c = 0; c < (SILU ? W / 2 : W); c += 64) {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = grouped::pack_pair<T>(result(c + 2 * j), result(c + 2 * j + 1));
          if (nrows <= 0 || col + c >= P.cols) continue;
          if (P.vec > 0)
            grouped::store_rows(buf, v, &tmY, col + c, row_y, 0, nrows >= 32, row0, nrows, P.cols);
          else
            grouped::store_ragged(buf, v, row0, nrows, col + c, P.cols);
        }
      } else {
#pragma unroll
        for (int c = 0; c < (SILU ? W / 2 : W); c += 32) {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(result(c + j));
          if (nrows <= 0 || col + c >= P.cols) continue;
          if (P.vec == 0)
            grouped::store_turned(v, row0, nrows, col + c, P.cols);
          else if (lane < nrows)
            grouped::store_cols(row0 + (long)lane * P.cols, col + c, P.cols, P.vec, v);
        }
      }
    }
    if (sizeof(T) == 2 && lane == 0) ptx::tma_store_wait();      // the last rows have left
    if (!*abort_p)
      grouped::zero_unowned(y, G, P.E, P.S, P.cols, ((long)blockIdx.x * EPI_WARPS + warp - EPI0) * 32 + lane,
                            (long)gridDim.x * EPI_WARPS * 32);
  }

  if (*abort_p) {   // after a timeout, let copies in flight land before the shared memory is released
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 1000000ull) {
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, F::TMEM_COLS);
  }
  if (tid == 0 && P.status) {
    if (abort_flag) atomicOr(P.status, MOE_STATUS_TIMEOUT);
    if (G.bad && blockIdx.x == 0) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  }
}

template <bool SILU, class T, int PARTS>
int launch_form(const Fp8Args& a, cudaStream_t s) {
  using F = Form<PARTS, T>;
  const char* name = "fp8_grouped_gemm";
  if (int rc = ensure_smem_limit(fp8_tc_kernel<SILU, T, PARTS>, F::DSMEM, name)) return rc;
  // The epilogue's warps wait for the registers that they ask for, so a block has to start with as many as the split needs
  // in all: with the register limit of its launch bounds, which a kernel that moves registers is compiled for.
  if (PARTS == 2) {
    static BuiltRegisters built;
    if (int rc = built.check(fp8_tc_kernel<SILU, T, PARTS>, EPI0 + 8, EPI0 * LOW_REGS + 8 * HIGH_REGS, name)) return rc;
  }
  CUtensorMap tx, tw, ty{};
  int rc;
  if ((rc = make_tmap_3d(&tx, a.x, 1, (uint64_t)a.K, (uint64_t)a.S, 1, KB, BM))) return rc;
  if ((rc = make_tmap_3d(&tw, a.w, 1, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E, KB, SILU ? F::HALF : F::BN))) return rc;
  Params p{};
  p.offsets = a.offsets;
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.S = a.S;
  p.E = a.E;
  p.kb = fp8::blocks(a.K);
  p.nb = fp8::blocks(a.N);
  p.cols = SILU ? a.N / 2 : a.N;
  p.NT = SILU ? (p.cols + F::HALF - 1) / F::HALF : (p.cols + F::BN - 1) / F::BN;
  p.y = a.y;
  p.vec = grouped::store_width(a.y, p.cols, sizeof(T));
  if (sizeof(T) == 2 && p.vec > 0 && (rc = make_tmap_3d(&ty, a.y, 2, (uint64_t)p.cols, (uint64_t)a.S, 1, 64, 32))) return rc;
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  const long tiles = ((long)(a.S + BM - 1) / BM + a.E) * p.NT;
  const int grid = (int)std::max(1L, std::min(tiles, (long)num_sms()));
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(fp8_tc_kernel<SILU, T, PARTS>, grid, F::THREADS, F::DSMEM, s, tx, tw, ty, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

// Tiles of 128 rows of w where all of them find an SM (about: an expert has one tile of rows, or half a tile more than its
// share): their accumulators come and go faster, and half as much passes through an SM. Measured, us, wide / narrow, K = 2048:
// 256 rows of 4 experts, [1024, 2048] 10.6 / 8.7, with the gate 11.7 / 9.6, [2816, 2048] 11.4 / 9.8; 1024 rows of 16 experts,
// [1024, 2048] 13.7 / 11.1; more tiles than SMs: 4096 rows of 16 experts 22.7 / 23.2, 128 rows of 8 experts, [2816, 2048]
// 14.2 / 16.8, 1024 rows of 64 experts 62 / 69.
template <bool SILU, class T>
int launch(const Fp8Args& a, cudaStream_t s) {
  const int cols = SILU ? a.N / 2 : a.N, width = Form<1, T>::BN / (SILU ? 2 : 1);
  const long rows = std::max<long>(std::min(a.S, a.E), a.S / BM + a.E / 2);
  return rows * ((cols + width - 1) / width) <= num_sms() ? launch_form<SILU, T, 1>(a, s) : launch_form<SILU, T, 2>(a, s);
}

}  // namespace

int launch_fp8_grouped(const Fp8Args& a, cudaStream_t s) {
  if (fp8::few_rows(a.S, a.E)) return launch_fp8_few(a, s);
  if (a.out_dtype == MOE_F32) return a.silu ? launch<true, float>(a, s) : launch<false, float>(a, s);
  if (a.out_dtype == MOE_BF16) return a.silu ? launch<true, __nv_bfloat16>(a, s) : launch<false, __nv_bfloat16>(a, s);
  return a.silu ? launch<true, __half>(a, s) : launch<false, __half>(a, s);
}

}  // namespace moe
