// Products of 8-bit rows grouped by expert where experts have few rows (decode): the weights are streamed once and
// everything else is small, so the bound is HBM.
//
//   y[p, n] = sum over blocks b of sx[p, b] sw[e, n / 128, b] sum over k in b of cx[p, k] cw[e, n, k]
//   (with the gate, silu(y[p, n]) y[p, N/2 + n])
//
// The operands change places: up to 128 rows of w are the MMA's M (A operand), the group's rows of x, 16 to 64 of
// them, its N; a TMEM lane then holds one output column of every row. One CTA per SM takes units of (expert, rows of
// x, f columns of y) by turns:
//   warp 0     TMA producer: per block of 128 of the reduction one box of f rows of w (two with the gate), boxes of 16
//              rows of x, through a ring whose stages are as large as the launch's units need;
//   warp 1     MMA issuer (M = 128, N = 16 .. 64, four K = 32 a block), a block to an accumulator;
//   warps 2-5  epilogue: multiply an accumulator by sx sw and add it in registers; at the end of a unit a warp stores 32
//              neighbouring columns of a row at a time.
// Blocks go to the epilogue four at a time (2 x 4 x 64 columns of tensor memory): a hand-over takes the epilogue some
// 500 cycles beside the sums, and one per block, 16 KB of weights, held the whole kernel at 4.8 TB/s.
// f is chosen on the host as for the 16-bit products (grouped_few.cu).
#include <algorithm>

#include "fp8.cuh"
#include "grouped.cuh"
#include "mxfp4_ptx.cuh"

namespace moe {
namespace {

constexpr int KB = fp8::BLOCK;           // bytes of a row per step
constexpr int BOX = 16;                  // rows of x per TMA box
constexpr int BOX_BYTES = BOX * KB;
constexpr int MAXF = 128;                // MMA M
constexpr int MAXR = 64;                 // rows of x per unit (MMA N at most)
constexpr int MAXHEADS = MOE_MAX_EXPERTS + fp8::kFewRows * MOE_MAX_EXPERTS / MAXR;   // (expert, 64 rows) of a launch
constexpr int A_READ = MAXF * KB;        // what an MMA reads of its A operand, whatever was loaded
constexpr int UP = A_READ / 2;           // with the gate: the up rows, after 64 rows of room for the gate's
constexpr int MAXSTAGE = 20;
constexpr int THREADS = 192;
constexpr int RING = 204 * 1024;
constexpr int DSMEM = RING + 1024;
constexpr int CHUNK = 4;                 // blocks that are handed to the epilogue together, each in columns of its own
constexpr uint32_t ACC_COLS = CHUNK * MAXR, TMEM_COLS = 2 * ACC_COLS;
constexpr uint64_t DRAIN_NS = 2000000000ull;

struct Params {
  const int32_t* offsets;
  const float* x_scales;
  const float* w_scales;
  int S, E, cols;       // columns of y
  int f;                // columns per unit
  int kb, nb;           // blocks along K and N
  void* y;
  int32_t* status;
  uint64_t wait_ns;
};

struct Unit {
  int e, row, rows, n0, cols;    // group row of its first row of x; columns [n0, n0 + cols)
};

// Unit t: head t / tiles (an expert's next 64 rows), column tile t % tiles.
__device__ __forceinline__ Unit unit_at(int t, const grouped::Groups& G, const uint16_t* expert_of, const Params& P, int tiles) {
  const int head = grouped::quick_div(t, tiles), tile = t - head * tiles, e = expert_of[head];
  const grouped::Span g = G.span(e);
  Unit u;
  u.e = e;
  u.row = g.lo + (head - G.start[e]) * MAXR;
  u.rows = min(MAXR, g.hi - u.row);
  u.n0 = tile * P.f;
  u.cols = min(P.f, P.cols - u.n0);
  return u;
}

// Barrier among `nthreads` threads that also tells all of them whether any passed true.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <bool SILU, class T>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params P) {
  __shared__ __align__(8) uint64_t full_bar[MAXSTAGE], empty_bar[MAXSTAGE];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int s_most;
  __shared__ grouped::Groups G;
  __shared__ uint16_t expert_of[MAXHEADS];
  __shared__ float up_part[SILU ? 64 : 1][17];      // up columns of 16 rows, on their way to the gate's warps
  __shared__ __align__(16) float x_part[4][CHUNK][MAXR];      // a chunk's scales of the rows, of each warp's own
  extern __shared__ uint8_t dsmem_raw[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t dsmem = (ptx::smem_u32(dsmem_raw) + 1023u) & ~1023u;
  volatile int* abort_p = &abort_flag;

  if (tid == 0) {
    for (int s = 0; s < MAXSTAGE; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&tfull_bar[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&tempty_bar[b]), 4);
    }
    ptx::mbar_init(ptx::smem_u32(&drain_bar), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  if (warp == 1) ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), TMEM_COLS);
  pdl_wait();          // the offsets and operands may be the previous kernel's output
  pdl_trigger();
  if (warp == 2) {
    const int most =
        grouped::group_list(P.offsets, P.E, P.S, [](int rows) { return (rows + MAXR - 1) / MAXR; }, G);
    if (lane == 0) s_most = min(most, MAXR);
    __syncwarp();
    for (int e = lane; e < P.E; e += 32)
      for (int h = G.start[e]; h < G.start[e + 1]; ++h) expert_of[h] = (uint16_t)e;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int f = P.f, tiles = (P.cols + f - 1) / f;
  const int total = G.start[P.E] * tiles;
  // the ring: A, then B; an MMA reads A_READ bytes from a stage on, so the last stage has to end that far inside
  const int a_bytes = (SILU ? UP : 0) + f * KB;
  const int stage_bytes = a_bytes + (s_most + BOX - 1) / BOX * BOX_BYTES;
  const int nstage = min(MAXSTAGE, (RING - max(0, A_READ - stage_bytes)) / stage_bytes);
  auto st = [&](int s) { return dsmem + (uint32_t)(s * stage_bytes); };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Unit u = unit_at(t, G, expert_of, P, tiles);
        const int boxes = (u.rows + BOX - 1) / BOX;
        for (int k = 0; k < P.kb; ++k) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb = ptx::smem_u32(&full_bar[stage]);
          ptx::mbar_arrive_expect_tx(fb, (uint32_t)((SILU ? 2 : 1) * f * KB + boxes * BOX_BYTES));
          ptx::tma_load_3d(st(stage), &tmW, k * KB, u.n0, u.e, fb);
          if (SILU) ptx::tma_load_3d(st(stage) + UP, &tmW, k * KB, P.cols + u.n0, u.e, fb);
          for (int i = 0; i < boxes; ++i)
            ptx::tma_load_3d(st(stage) + a_bytes + i * BOX_BYTES, &tmX, k * KB, u.row + i * BOX, 0, fb);
          if (++stage == nstage) { stage = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (ptx::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Unit u = unit_at(t, G, expert_of, P, tiles);
        const uint32_t idesc = fp8::idesc(MAXF, (u.rows + BOX - 1) / BOX * BOX);
        for (int k = 0; k < P.kb; ++k) {
          if (k % CHUNK == 0) {
            ok = ptx::mbar_wait(ptx::smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_p, P.wait_ns);
            if (!ok) break;
          }
          ok = ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), ph, abort_p, P.wait_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * ACC_COLS + k % CHUNK * MAXR);
          const uint64_t ad = ptx::sdesc_k128(st(stage)), bd = ptx::sdesc_k128(st(stage) + a_bytes);
#pragma unroll
          for (int kk = 0; kk < KB / 32; ++kk) fp8::mma(d_tmem, ad + kk * 2, bd + kk * 2, idesc, kk != 0);
          ptx::mma_commit(ptx::smem_u32(&empty_bar[stage]));
          if (++stage == nstage) { stage = 0; ph ^= 1u; }
          if (k % CHUNK == CHUNK - 1 || k == P.kb - 1) {
            ptx::mma_commit(ptx::smem_u32(&tfull_bar[acc]));
            if (++acc == 2) { acc = 0; aph ^= 1u; }
          }
        }
      }
      ptx::mma_commit(ptx::smem_u32(&drain_bar));
      int dummy = 0;
      ptx::mbar_wait(ptx::smem_u32(&drain_bar), 0, &dummy, DRAIN_NS);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;              // TMEM lane quarter this warp may read
    const int l = q * 32 + lane;         // row of the A operand
    auto& xp = x_part[q];
    T* y = static_cast<T*>(P.y);
    int acc = 0;
    uint32_t aph = 0;
    // A unit's scales: `load` fetches a chunk's while the last one is added, a unit's first ones before the last unit's
    // results are stored.
    const float *ws, *xs0, *xs1;             // of this lane's row of w, and of two rows of x
    bool more = false;                       // rows in the second 32
    float w[CHUNK], x0[CHUNK], x1[CHUNK];
    auto locate = [&](const Unit& u) {
      const int wrow = !SILU || l < 64 ? u.n0 + l : P.cols + u.n0 + l - 64;
      ws = P.w_scales + ((long)u.e * P.nb + min(wrow / KB, P.nb - 1)) * P.kb;
      xs0 = P.x_scales + (long)(u.row + min(lane, u.rows - 1)) * P.kb;
      xs1 = P.x_scales + (long)(u.row + min(lane + 32, u.rows - 1)) * P.kb;
      more = u.rows > 32;
    };
    auto load = [&](int k0) {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        const int k = min(k0 + i, P.kb - 1);
        w[i] = __ldg(ws + k);
        x0[i] = __ldg(xs0 + k);
        x1[i] = more ? __ldg(xs1 + k) : 0.0f;
      }
    };
    Unit u{};
    if ((int)blockIdx.x < total) {
      u = unit_at(blockIdx.x, G, expert_of, P, tiles);
      locate(u);
      load(0);
    }
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      float sum[MAXR];
#pragma unroll
      for (int j = 0; j < MAXR; ++j) sum[j] = 0.0f;
      bool ok = true;
      for (int k0 = 0; k0 < P.kb && ok; k0 += CHUNK) {
        float cw[CHUNK];
        __syncwarp();                      // the last chunk's have been read
#pragma unroll
        for (int i = 0; i < CHUNK; ++i) {
          cw[i] = w[i];
          xp[i][lane] = x0[i];
          if (more) xp[i][lane + 32] = x1[i];
        }
        __syncwarp();
        if (k0 + CHUNK < P.kb) load(k0 + CHUNK);
        // whole warps go on or stop
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * ACC_COLS);
#pragma unroll
        for (int c = 0; c < MAXR; c += 16) {
          if (c >= u.rows) continue;
          uint32_t v[CHUNK][16];
#pragma unroll
          for (int i = 0; i < CHUNK; ++i)
            if (k0 + i < P.kb) ptx::tmem_ld16(taddr + i * MAXR + c, v[i]);
#pragma unroll
          for (int i = 0; i < CHUNK; ++i) {
            if (k0 + i >= P.kb) continue;
            ptx::tmem_ld_wait16(v[i]);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 x = *reinterpret_cast<const float4*>(&xp[i][c + j]);
              sum[c + j] = fmaf(__uint_as_float(v[i][j]), x.x * cw[i], sum[c + j]);
              sum[c + j + 1] = fmaf(__uint_as_float(v[i][j + 1]), x.y * cw[i], sum[c + j + 1]);
              sum[c + j + 2] = fmaf(__uint_as_float(v[i][j + 2]), x.z * cw[i], sum[c + j + 2]);
              sum[c + j + 3] = fmaf(__uint_as_float(v[i][j + 3]), x.w * cw[i], sum[c + j + 3]);
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&tempty_bar[acc]));
        if (++acc == 2) { acc = 0; aph ^= 1u; }
      }
      // every epilogue warp sees the same outcome: the gate's exchange needs all four
      if (SILU) ok = !named_bar_or(1, 128, !ok);
      if (!ok) break;
      const int rows = u.rows, cols = u.cols;
      T* dst = y + (long)u.row * P.cols + u.n0;
      if (t + (int)gridDim.x < total) {
        u = unit_at(t + gridDim.x, G, expert_of, P, tiles);
        locate(u);
        load(0);
      }
#pragma unroll
      for (int c = 0; c < MAXR; c += 16) {
        if (c >= rows) continue;
        if (SILU) {
          if (l >= 64) {
#pragma unroll
            for (int j = 0; j < 16; ++j) up_part[l - 64][j] = sum[c + j];
          }
          ptx::named_bar_sync(1, 128);
        }
        if (l < cols) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < rows)
              dst[(long)(c + j) * P.cols + l] = from_float<T>(SILU ? mx::silu_fast(sum[c + j]) * up_part[l][j] : sum[c + j]);
        }
        if (SILU) ptx::named_bar_sync(1, 128);
      }
    }
    if (!*abort_p)
      grouped::zero_unowned(y, G, P.E, P.S, P.cols, (long)blockIdx.x * 128 + tid - 64, (long)gridDim.x * 128);
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
    ptx::tmem_dealloc(tmem_base, TMEM_COLS);
  }
  if (tid == 0 && P.status) {
    if (abort_flag) atomicOr(P.status, MOE_STATUS_TIMEOUT);
    if (G.bad && blockIdx.x == 0) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  }
}

template <bool SILU, class T>
int launch(const Fp8Args& a, cudaStream_t s) {
  const char* name = "fp8_grouped_few";
  if (int rc = ensure_smem_limit(fp8_few_kernel<SILU, T>, DSMEM, name)) return rc;
  CUtensorMap tw, tx;
  int rc;
  Params p{};
  p.cols = SILU ? a.N / 2 : a.N;
  p.f = grouped_few_columns(std::min(a.S, a.E), p.cols, SILU ? MAXF / 2 : MAXF);
  if ((rc = make_tmap_3d(&tw, a.w, 1, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E, KB, p.f))) return rc;
  if ((rc = make_tmap_3d(&tx, a.x, 1, (uint64_t)a.K, (uint64_t)a.S, 1, KB, BOX))) return rc;
  p.offsets = a.offsets;
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.S = a.S;
  p.E = a.E;
  p.kb = fp8::blocks(a.K);
  p.nb = fp8::blocks(a.N);
  p.y = a.y;
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(fp8_few_kernel<SILU, T>, num_sms(), THREADS, DSMEM, s, tw, tx, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

}  // namespace

int launch_fp8_few(const Fp8Args& a, cudaStream_t s) {
  if (a.out_dtype == MOE_F32) return a.silu ? launch<true, float>(a, s) : launch<false, float>(a, s);
  if (a.out_dtype == MOE_BF16) return a.silu ? launch<true, __nv_bfloat16>(a, s) : launch<false, __nv_bfloat16>(a, s);
  return a.silu ? launch<true, __half>(a, s) : launch<false, __half>(a, s);
}

}  // namespace moe
