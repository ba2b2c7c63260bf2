// Products grouped by expert where experts have few rows (decode): the weights are streamed
// once and everything else is small, so the bound is HBM.
//
//   y[p, n] = sum_k x[p, k] w[e, n, k]      bf16, float16, or 4-bit microscaled operands
//   (4-bit with the gate: silu(y[p, n]) y[p, N/2 + n])
//
// The operands change places: up to 128 rows of w are the MMA's M (A operand), the group's
// rows of x, 16 to 64 of them, its N; a TMEM lane then holds one output column of every row.
// One CTA per SM takes units of (expert, rows of x, f columns of y) by turns:
//   warp 0     TMA producer: per step 128 bytes of each of the unit's rows (one box of f rows of
//              w, boxes of 16 rows of x), through a ring whose stages are as large as the
//              launch's units need (their columns, the rows of the largest group), so that
//              there are up to 20 of them and about 160 KB of weights in flight per SM;
//   warp 1     MMA issuer (M = 128, N = 16 .. 64);
//   warps 2-5  epilogue: a warp stores 32 neighbouring columns of a row at a time;
//   warps 6-9  4-bit only: scales, each warp every fourth chunk of four steps, through a buffer
//              and a pair of barriers of its own, so that four chunks of loads are under way
//              without registers for more than one.
// f, the columns of a unit (a multiple of 16), is chosen on the host from the number of experts
// that can be active, min(S, E): M = 128 tiles of, say, 8 active experts with 2816 columns would
// be 176 units for 152 SMs, two rounds of which the second is nearly empty; 80 columns make 288.
// The box has f rows because TMA instructions are what limits a unit otherwise: with boxes of 16
// rows a step took 600 cycles whatever its size (33 GB/s an SM at f = 80).
// A group of more than 64 rows is several heads, whose units read the same weights at about the
// same time.
#include <algorithm>

#include "grouped.cuh"
#include "mxfp4_ptx.cuh"

namespace moe {
namespace {

constexpr int ROWB = 128;                // bytes of a row per step
constexpr int BOX = 16;                  // rows per TMA box
constexpr int BOX_BYTES = BOX * ROWB;
constexpr int MAXF = 128;                // MMA M
constexpr int MAXR = 64;                 // rows of x per unit (MMA N at most)
constexpr int MAXHEADS = MOE_MAX_EXPERTS + kFewRows * MOE_MAX_EXPERTS / MAXR;   // (expert, 64 rows) of a launch
constexpr int CHUNK = 4;                 // steps whose scales one warp loads together
constexpr uint64_t DRAIN_NS = 2000000000ull;

template <bool MX>
struct Cfg {
  static constexpr int A_READ = MAXF * ROWB;         // what an MMA reads of its A operand, whatever was loaded
  static constexpr int UP = A_READ / 2;              // with the gate: the up rows, after 64 rows of room for the gate's
  static constexpr int MAXSTAGE = 20;
  static constexpr int RING = (MX ? 176 : 208) * 1024;
  static constexpr int SF_WARPS = MX ? 4 : 0;
  static constexpr int SF_STEP = 4 * (int)mx::SF_ATOM;          // of one step: two atoms of A, two of B
  static constexpr int SF_OFF = RING, SF_BUF = CHUNK * SF_STEP;
  static constexpr int DSMEM = SF_OFF + SF_WARPS * SF_BUF + 1024;
  static constexpr int THREADS = (6 + SF_WARPS) * 32;
  static constexpr uint32_t SF_COL = 2 * MAXR;       // scales: two sets of 16 columns
  static constexpr uint32_t TMEM_COLS = MX ? 256 : 128;
};

struct Params {
  const int32_t* offsets;
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  int S, E, N, cols;    // rows of w; columns of y
  int f;                // columns per unit
  int steps;            // of 128 bytes along K
  int count, vec;       // 4-bit: scale bytes of a row, bytes read at a time (16, 4, 1)
  void* y;
  uint32_t idesc;       // without N
  int32_t* status;
  uint64_t wait_ns;
};

struct Unit {
  int e, row, rows, n0, cols;    // group row of its first row of x; columns [n0, n0 + cols)
};

// Unit t: head t / tiles (an expert's next 64 rows), column tile t % tiles. Every role looks its units
// up, and with short reductions that is what the MMA issuer waits for (a search over the experts and
// two divisions took 1000 of 3000 cycles a unit at K = 352), so the heads have a list.
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

__device__ __forceinline__ uint32_t word(const uint4& q, int i) { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }

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

template <bool MX, bool SILU, class T>
__global__ void __launch_bounds__(Cfg<MX>::THREADS, 1)
    grouped_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const Params P) {
  using C = Cfg<MX>;
  __shared__ __align__(8) uint64_t full_bar[C::MAXSTAGE], empty_bar[C::MAXSTAGE];
  __shared__ __align__(8) uint64_t sf_full[4], sf_empty[4];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int s_most;
  __shared__ grouped::Groups G;
  __shared__ uint16_t expert_of[MAXHEADS];
  __shared__ float up_part[SILU ? 64 : 1][17];      // up columns of 16 rows, on their way to the gate's warps
  extern __shared__ uint8_t dsmem_raw[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t dsmem = (ptx::smem_u32(dsmem_raw) + 1023u) & ~1023u;
  auto sf = [&](int b, int step) { return dsmem + (uint32_t)(C::SF_OFF + b * C::SF_BUF + step * C::SF_STEP); };
  volatile int* abort_p = &abort_flag;

  if (tid == 0) {
    for (int s = 0; s < C::MAXSTAGE; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&tfull_bar[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&tempty_bar[b]), 4);
    }
    for (int b = 0; b < 4; ++b) {
      ptx::mbar_init(ptx::smem_u32(&sf_full[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&sf_empty[b]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&drain_bar), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  if (warp == 1) ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), C::TMEM_COLS);
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
  // the ring: A, then B; an MMA reads A_READ bytes from a stage on, so the last stage has to end
  // that far inside the ring
  const int a_bytes = (SILU ? C::UP : 0) + f * ROWB;
  const int stage_bytes = a_bytes + (s_most + BOX - 1) / BOX * BOX_BYTES;
  const int nstage = min(C::MAXSTAGE, (C::RING - max(0, C::A_READ - stage_bytes)) / stage_bytes);
  auto st = [&](int s) { return dsmem + (uint32_t)(s * stage_bytes); };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Unit u = unit_at(t, G, expert_of, P, tiles);
        const int nb = (u.rows + BOX - 1) / BOX;
        for (int k = 0; k < P.steps; ++k) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb = ptx::smem_u32(&full_bar[stage]);
          ptx::mbar_arrive_expect_tx(fb, (uint32_t)((SILU ? 2 : 1) * f * ROWB + nb * BOX_BYTES));
          const int x = k * (MX ? ROWB : ROWB / 2);
          ptx::tma_load_3d(st(stage), &tmW, x, u.n0, u.e, fb);
          if (SILU) ptx::tma_load_3d(st(stage) + C::UP, &tmW, x, P.cols + u.n0, u.e, fb);
          for (int i = 0; i < nb; ++i)
            ptx::tma_load_3d(st(stage) + a_bytes + i * BOX_BYTES, &tmX, x, u.row + i * BOX, 0, fb);
          if (++stage == nstage) { stage = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (ptx::elect_one()) {
      int stage = 0, acc = 0, set = 0, turn = 0;   // turn: chunks of scales so far
      uint32_t ph = 0, aph = 0;
      for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const Unit u = unit_at(t, G, expert_of, P, tiles);
        const int n = (u.rows + BOX - 1) / BOX * BOX;
        const uint32_t idesc = P.idesc | ((uint32_t)(n >> 3) << 17);
        if (!ptx::mbar_wait(ptx::smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_p, P.wait_ns)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * MAXR);
        bool ok = true;
        for (int k = 0; k < P.steps; ++k) {
          if (!ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), ph, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          if (MX && k % CHUNK == 0 &&
              !ptx::mbar_wait(ptx::smem_u32(&sf_full[turn & 3]), (uint32_t)(turn >> 2) & 1u, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a0 = st(stage), b0 = a0 + a_bytes;
          if constexpr (MX) {
            const uint32_t sfa = tmem_base + C::SF_COL + (set ? 16u : 0u), sfb = sfa + 8;
            const uint32_t s0 = sf(turn & 3, k % CHUNK);
            set ^= 1;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              mx::copy_scales<1>(sfa + j * 4, mx::sdesc_scales(s0 + j * mx::SF_ATOM));
              mx::copy_scales<1>(sfb + j * 4, mx::sdesc_scales(s0 + (2 + j) * mx::SF_ATOM));
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mx::mma<1>(d_tmem, ptx::sdesc_k128(a0 + kk * 32), ptx::sdesc_k128(b0 + kk * 32),
                         idesc | mx::idesc_scales((kk & 1) * 2), sfa + (kk >> 1) * 4, sfb + (kk >> 1) * 4, (k | kk) != 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::mma_bf16(d_tmem, ptx::sdesc_k128(a0 + kk * 32), ptx::sdesc_k128(b0 + kk * 32), idesc, (k | kk) != 0);
          }
          ptx::mma_commit(ptx::smem_u32(&empty_bar[stage]));
          if (MX && (k % CHUNK == CHUNK - 1 || k == P.steps - 1)) {
            ptx::mma_commit(ptx::smem_u32(&sf_empty[turn & 3]));
            ++turn;
          }
          if (++stage == nstage) { stage = 0; ph ^= 1u; }
        }
        if (!ok) break;
        ptx::mma_commit(ptx::smem_u32(&tfull_bar[acc]));
        if (++acc == 2) { acc = 0; aph ^= 1u; }
      }
      ptx::mma_commit(ptx::smem_u32(&drain_bar));
      int dummy = 0;
      ptx::mbar_wait(ptx::smem_u32(&drain_bar), 0, &dummy, DRAIN_NS);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;              // TMEM lane quarter this warp may read
    const int l = q * 32 + lane;         // row of the A operand
    T* y = static_cast<T*>(P.y);
    int acc = 0;
    uint32_t aph = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Unit u = unit_at(t, G, expert_of, P, tiles);
      // every epilogue warp sees the same outcome: the gate's exchange needs all four
      bool ok = ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns);
      if (SILU) ok = !named_bar_or(1, 128, !ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * MAXR);
      for (int c = 0; c < u.rows; c += 16) {      // 16 rows of x
        uint32_t v[16];
        ptx::tmem_ld16(taddr + c, v);
        ptx::tmem_ld_wait();
        T* dst = y + (long)(u.row + c) * P.cols + u.n0;
        const int nr = min(16, u.rows - c);
        if (SILU) {
          if (l >= 64) {
#pragma unroll
            for (int j = 0; j < 16; ++j) up_part[l - 64][j] = __uint_as_float(v[j]);
          }
          ptx::named_bar_sync(1, 128);
          if (l < u.cols) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (j < nr) dst[(long)j * P.cols + l] = from_float<T>(mx::silu_fast(__uint_as_float(v[j])) * up_part[l][j]);
          }
          ptx::named_bar_sync(1, 128);
        } else if (l < u.cols) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < nr) dst[(long)j * P.cols + l] = from_float<T>(__uint_as_float(v[j]));
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&tempty_bar[acc]));
      if (++acc == 2) { acc = 0; aph ^= 1u; }
    }
    if (!*abort_p)
      grouped::zero_unowned(y, G, P.E, P.S, P.cols, (long)blockIdx.x * 128 + tid - 64, (long)gridDim.x * 128);
  } else if (MX) {
    // ------------------------------------------------------------ scales
    const int me = warp - 6;
    int turn = 0;                        // chunks so far, over all units
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Unit u = unit_at(t, G, expert_of, P, tiles);
      for (int k0 = 0; k0 < P.steps && ok; k0 += CHUNK, ++turn) {
        if ((turn & 3) != me) continue;
        // rows l, l + 32, l + 64, l + 96 of w and l, l + 32 of x; what the unit does not have is 0
        uint4 v[6][2];
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          const int r = lane + 32 * (i < 4 ? i : i - 4);
          const uint8_t* row = nullptr;
          const uint8_t* end = i < 4 ? P.w_scales + (long)P.E * P.N * P.count : P.x_scales + (long)P.S * P.count;
          if (i < 4) {
            const int c = SILU ? r & 63 : r;
            if (c < u.cols)
              row = P.w_scales + ((long)u.e * P.N + u.n0 + c + (SILU && r >= 64 ? P.cols : 0)) * P.count;
          } else if (r < u.rows) {
            row = P.x_scales + (long)(u.row + r) * P.count;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[i][h] = row != nullptr ? mx::scale16(row, k0 * 8 + h * 16, P.count, P.vec, end) : make_uint4(0, 0, 0, 0);
        }
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&sf_empty[me]), ((uint32_t)(turn >> 2) & 1u) ^ 1u,
                                                    abort_p, P.wait_ns));
        if (!ok) continue;
#pragma unroll
        for (int d = 0; d < CHUNK; ++d) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = d >> 1, wd = (d & 1) * 2 + j;      // word 2 d + j of the 32 bytes
            const uint32_t a = sf(me, d) + j * mx::SF_ATOM + lane * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(word(v[0][h], wd)),
                         "r"(word(v[1][h], wd)), "r"(word(v[2][h], wd)), "r"(word(v[3][h], wd))
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %3};" ::"r"(a + 2 * mx::SF_ATOM),
                         "r"(word(v[4][h], wd)), "r"(word(v[5][h], wd)), "r"(0)
                         : "memory");
          }
        }
        pair::fence_async_shared();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sf_full[me]));
      }
    }
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
    ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if (tid == 0 && P.status) {
    if (abort_flag) atomicOr(P.status, MOE_STATUS_TIMEOUT);
    if (G.bad && blockIdx.x == 0) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  }
}

template <bool MX, bool SILU, class T>
int launch(const CUtensorMap& w, const CUtensorMap& x, const Params& p, cudaStream_t s, const char* name) {
  if (int rc = ensure_smem_limit(grouped_few_kernel<MX, SILU, T>, Cfg<MX>::DSMEM, name)) return rc;
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(grouped_few_kernel<MX, SILU, T>, num_sms(), Cfg<MX>::THREADS, Cfg<MX>::DSMEM, s, w, x, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

template <bool SILU>
int launch_mx(int dtype, const CUtensorMap& w, const CUtensorMap& x, const Params& p, cudaStream_t s) {
  const char* name = "mxfp4_grouped_few";
  if (dtype == MOE_F32) return launch<true, SILU, float>(w, x, p, s, name);
  if (dtype == MOE_BF16) return launch<true, SILU, __nv_bfloat16>(w, x, p, s, name);
  return launch<true, SILU, __half>(w, x, p, s, name);
}

}  // namespace

// Columns per unit: the largest number of rounds times (columns + the cost of a unit, about that of
// 8 columns) is smallest; of equals the larger.
int grouped_few_columns(long heads, int cols, int most) {
  int best = most;
  long cost = 1L << 62;
  for (int f = most; f >= BOX; f -= BOX) {
    const long units = heads * ((cols + f - 1) / f), ctas = num_sms();
    const long c = (units + ctas - 1) / ctas * (f + 8);
    if (c < cost) {
      cost = c;
      best = f;
    }
  }
  return best;
}

int launch_grouped_few(const GroupedArgs& a, const void* x, const void* w, int cols, cudaStream_t s) {
  CUtensorMap tw, tx;
  int rc;
  const int f = grouped_few_columns(std::min(a.S, a.E), a.N, MAXF);
  if ((rc = make_tmap_3d(&tw, w, 2, (uint64_t)cols, (uint64_t)a.N, (uint64_t)a.E, ROWB / 2, f))) return rc;
  if ((rc = make_tmap_3d(&tx, x, 2, (uint64_t)cols, (uint64_t)a.S, 1, ROWB / 2, BOX))) return rc;
  Params p{};
  p.f = f;
  p.offsets = a.offsets;
  p.S = a.S;
  p.E = a.E;
  p.N = p.cols = a.N;
  p.steps = (a.K + ROWB / 2 - 1) / (ROWB / 2);
  p.y = a.y;
  p.idesc = ptx::idesc_bf16_f32(MAXF, 0);
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  if (a.dtype == MOE_BF16) return launch<false, false, __nv_bfloat16>(tw, tx, p, s, "grouped_gemm_few");
  p.idesc &= ~((1u << 7) | (1u << 10));   // A and B float16
  return launch<false, false, __half>(tw, tx, p, s, "grouped_gemm_few");
}

int launch_mxfp4_few(const Mxfp4Args& a, cudaStream_t s) {
  CUtensorMap tw, tx;
  int rc;
  const int f = grouped_few_columns(std::min(a.S, a.E), a.silu ? a.N / 2 : a.N, a.silu ? MAXF / 2 : MAXF);
  if ((rc = make_tmap_3d(&tw, a.w, 1, (uint64_t)a.K / 2, (uint64_t)a.N, (uint64_t)a.E, ROWB, f))) return rc;
  if ((rc = make_tmap_3d(&tx, a.x, 1, (uint64_t)a.K / 2, (uint64_t)a.S, 1, ROWB, BOX))) return rc;
  Params p{};
  p.f = f;
  p.offsets = a.offsets;
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.S = a.S;
  p.E = a.E;
  p.N = a.N;
  p.cols = a.silu ? a.N / 2 : a.N;
  p.steps = (a.K / 2 + ROWB - 1) / ROWB;
  p.count = a.K / 32;
  p.vec = mx::scale_vec(p.count);
  p.y = a.y;
  p.idesc = mx::idesc(MAXF, 0);
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  return a.silu ? launch_mx<true>(a.out_dtype, tw, tx, p, s) : launch_mx<false>(a.out_dtype, tw, tx, p, s);
}

}  // namespace moe
