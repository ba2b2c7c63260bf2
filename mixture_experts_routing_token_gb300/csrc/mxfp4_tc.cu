// Grouped product of 4-bit microscaled operands on SM pairs (tcgen05.mma.cta_group::2,
// kind::mxf4, M = 256 x N = 224 x K = 64, float32 accumulators in TMEM).
//
//   y[p, n] = sum over blocks b of 32 of 2^(sx + sw) sum in b of cx cw
// then, with the gate, silu(y[p, n]) y[p, N/2 + n] in the epilogue, so the [S, N] product
// is never written. Each SM of the pair loads its own 128 of the tile's 256 rows of x and
// half of its 224 rows of w per step of 256 of the reduction (128 bytes of codes a row, the
// layout 128-byte swizzled TMA writes); with the gate SM 0 holds 112 gate rows and SM 1 the
// matching 112 up rows, so a TMEM lane has both in columns j and 112 + j.
//
// N = 224: tensor memory has 512 columns, two accumulators of 256 would leave none for the
// scales (8 columns for A, 16 for B); two of 224 do, and keep the epilogue of one tile under
// the products of the next.
//
// The user holds scales as [rows, K / 32] bytes. tcgen05.cp wants them as atoms of 128 rows x 4
// scales, by tile, so a first kernel (mxfp4_scales_kernel) writes them in that order into the
// workspace: 1/17 of the operands' bytes, read and written once, after which a step's scales are
// one TMA box each. Warps that read them from global memory inside the product's own pipeline
// were slower (prompt 328 us with, 359 us with a deeper prefetch): with one row per lane their
// loads touch 32 lines an instruction, beside the epilogue's stores.
//
// Bound at prompt sizes: what an SM can take in. A step brings 33 KB (codes and scales) for about 490
// cycles of products and takes 550, 60 bytes a cycle; with the copies left out the same code took
// 224 us where it takes 252 (131072 rows, 64 experts of [2816, 2048] with the gate, on a cold GPU: 6.0
// PFLOP/s; under the power cap of a long run 287 us, 5.3). Half of a step's bytes are x, loaded again for
// every column tile. Prefetches of the next steps' weights into L2 made it slower (282 us).
// With the gate and N / 2 not a multiple of 8 each lane stores its row value by value, and that sets the
// pace: 1749 us at N / 2 = 1412, 248 at 1408.
#include <algorithm>

#include "grouped.cuh"
#include "mxfp4_ptx.cuh"

namespace moe {
namespace {

using namespace pair;

constexpr int BM = 128;                   // rows of x per SM
constexpr int BN = 224;                   // rows of w per tile
constexpr int HALF = BN / 2;              // per SM
constexpr int KB_BYTES = 128;             // bytes of codes per row and step (K = 256)
constexpr int NSTAGE = 6;
constexpr int A_BYTES = BM * KB_BYTES;
constexpr int B_BYTES = 14 * 1024;        // HALF rows
constexpr int SFA_OFF = A_BYTES + B_BYTES;
constexpr int SFB_OFF = SFA_OFF + 2 * (int)mx::SF_ATOM;
constexpr int STAGE = SFB_OFF + 4 * (int)mx::SF_ATOM;
constexpr int DSMEM = NSTAGE * STAGE + 1024;
constexpr int EPI_WARPS = 4;
constexpr int THREADS = (2 + EPI_WARPS) * 32;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SFA_COL = 2 * BN, SFB_COL = SFA_COL + 8;
constexpr uint64_t DRAIN_NS = 2000000000ull;
static_assert(B_BYTES == HALF * KB_BYTES && STAGE % 1024 == 0, "stage layout");
constexpr uint32_t SF_COLS = 24;          // one step's scales; two sets, taken in turn
static_assert(SFA_COL + 2 * SF_COLS <= TMEM_COLS, "tensor memory");

struct Params {
  const int32_t* offsets;
  int S, E;
  int steps;        // of 256 along K
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

__device__ __forceinline__ int mtiles(int rows) { return (rows + 2 * BM - 1) / (2 * BM); }

__device__ __forceinline__ Tile tile_at(int t, int& e, const grouped::Groups& G, const Params& P) {
  Tile d;
  e = grouped::find_from(G.start, e, t);
  d.e = e;
  d.g = G.span(d.e);
  const int local = t - G.start[d.e], mt = mtiles(d.g.rows());
  if (mt > P.NT) {
    d.m = grouped::quick_div(local, P.NT);
    d.n = local - d.m * P.NT;
  } else {
    d.n = grouped::quick_div(local, mt);
    d.m = local - d.n * mt;
  }
  return d;
}

// First row of w that block b (0 or 1, HALF rows) of tile n's B operand holds.
template <bool SILU>
__device__ __forceinline__ int w_row(int n, int b, const Params& P) {
  return SILU ? n * HALF + b * P.cols : n * BN + b * HALF;
}

template <bool SILU, class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmXS, const __grid_constant__ CUtensorMap tmWS,
                      const Params P) {
  __shared__ __align__(8) uint64_t full_bar[NSTAGE], empty_bar[NSTAGE];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ grouped::Groups G;
  extern __shared__ uint8_t dsmem_raw[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int cluster_id = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
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
      ptx::mbar_init(ptx::smem_u32(&tempty_bar[b]), 2 * EPI_WARPS);
    }
    ptx::mbar_init(ptx::smem_u32(&drain_bar), 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmX);
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmXS);
    ptx::prefetch_tmap(&tmWS);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     ptx::smem_u32(&tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();          // the offsets and operands may be the previous kernel's output
  pdl_trigger();
  if (warp == 2)
    grouped::group_list(P.offsets, P.E, P.S, [&](int rows) { return mtiles(rows) * P.NT; }, G);
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();      // barriers of both CTAs initialised before any cross-CTA signal
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int total = G.start[P.E];

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = cluster_id, e = 0; t < total && ok; t += nclusters) {
        const Tile ti = tile_at(t, e, G, P);
        const int a_row = ti.g.lo + ti.m * (2 * BM) + (int)rank * BM, b_row = w_row<SILU>(ti.n, (int)rank, P);
        const int a_atom = (grouped::quick_div(G.start[ti.e], P.NT) * 2 + ti.m * 2 + (int)rank) * P.steps * 2;
        const int b_atom = (ti.e * P.NT + ti.n) * P.steps * 4;
        for (int kb = 0; kb < P.steps; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = ptx::smem_u32(&full_bar[stage]);
          if (leader) ptx::mbar_arrive_expect_tx(fb_local, 2 * STAGE);
          const uint32_t fb = map_to_rank(fb_local, 0);
          tma_load_3d_pair(st(stage), &tmX, kb * KB_BYTES, a_row, 0, fb);
          tma_load_3d_pair(st(stage) + A_BYTES, &tmW, kb * KB_BYTES, b_row, ti.e, fb);
          tma_load_2d_pair(st(stage) + SFA_OFF, &tmXS, 0, a_atom + kb * 2, fb);
          tma_load_2d_pair(st(stage) + SFB_OFF, &tmWS, 0, b_atom + kb * 4, fb);
          if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    if (leader && ptx::elect_one()) {
      constexpr uint32_t IDESC = mx::idesc(2 * BM, BN);
      int stage = 0, acc = 0, set = 0;
      uint32_t ph = 0, aph = 0;
      for (int t = cluster_id, e = 0; t < total; t += nclusters) {
        if (!ptx::mbar_wait(ptx::smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_p, P.wait_ns)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
        bool ok = true;
        for (int kb = 0; kb < P.steps; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), ph, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a0 = st(stage), b0 = a0 + A_BYTES, sa = a0 + SFA_OFF, sb = a0 + SFB_OFF;
          // copies and MMAs of one thread execute in the order of issue
          const uint32_t sfa = tmem_base + SFA_COL + (set ? SF_COLS : 0u), sfb = sfa + (SFB_COL - SFA_COL);
          set ^= 1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mx::copy_scales<2>(sfa + j * 4, mx::sdesc_scales(sa + j * mx::SF_ATOM));
            mx::copy_scales<2>(sfb + j * 8, mx::sdesc_scales(sb + j * mx::SF_ATOM));
            mx::copy_scales<2>(sfb + j * 8 + 4, mx::sdesc_scales(sb + (2 + j) * mx::SF_ATOM));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mx::mma<2>(d_tmem, ptx::sdesc_k128(a0 + kk * 32), ptx::sdesc_k128(b0 + kk * 32),
                       IDESC | mx::idesc_scales((kk & 1) * 2), sfa + (kk >> 1) * 4, sfb + (kk >> 1) * 8, (kb | kk) != 0);
          commit_pair(ptx::smem_u32(&empty_bar[stage]), 0x3);
          if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
        }
        if (!ok) break;
        commit_pair(ptx::smem_u32(&tfull_bar[acc]), 0x3);
        if (++acc == 2) { acc = 0; aph ^= 1u; }
      }
      commit_pair(ptx::smem_u32(&drain_bar), 0x1);
      int dummy = 0;
      ptx::mbar_wait(ptx::smem_u32(&drain_bar), 0, &dummy, DRAIN_NS);
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;              // TMEM lane quarter this warp may read
    const int row = q * 32 + lane;
    T* y = static_cast<T*>(P.y);
    int acc = 0;
    uint32_t aph = 0;
    for (int t = cluster_id, e = 0; t < total; t += nclusters) {
      const Tile ti = tile_at(t, e, G, P);
      const int m = ti.m * (2 * BM) + (int)rank * BM + row;
      const bool mine = m < ti.g.rows();
      T* dst = y + ((long)ti.g.lo + m) * P.cols;
      if (!ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns)) break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      if (SILU) {
#pragma unroll 1
        for (int c = 0; c < HALF; c += 16) {
          uint32_t g[16], u[16];
          ptx::tmem_ld16(taddr + c, g);
          ptx::tmem_ld16(taddr + HALF + c, u);
          ptx::tmem_ld_wait();
          const int c0 = ti.n * HALF + c;
          if (mine && c0 < P.cols) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              g[i] = __float_as_uint(mx::silu_fast(__uint_as_float(g[i])) * __uint_as_float(u[i]));
            grouped::store_cols(dst, c0, P.cols, P.vec, g);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
          uint32_t v[32];
          ptx::tmem_ld32(taddr + c, v);
          ptx::tmem_ld_wait();
          const int c0 = ti.n * BN + c;
          if (P.vec > 0) {
            if (mine && c0 < P.cols) grouped::store_cols(dst, c0, P.cols, P.vec, v);
          } else if (m - lane < ti.g.rows() && c0 < P.cols) {
            grouped::store_turned(v, dst - (long)lane * P.cols, ti.g.rows() - (m - lane), c0, P.cols);
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&tempty_bar[acc]), 0));
      if (++acc == 2) { acc = 0; aph ^= 1u; }
    }
    if (!*abort_p)
      grouped::zero_unowned(y, G, P.E, P.S, P.cols, ((long)blockIdx.x * EPI_WARPS + warp - 2) * 32 + lane,
                            (long)gridDim.x * EPI_WARPS * 32);
  }

  if (*abort_p) {   // after a timeout, let copies in flight land before the shared memory is released
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 1000000ull) {
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                 : "memory");
  }
  if (tid == 0 && P.status) {
    if (abort_flag) atomicOr(P.status, MOE_STATUS_TIMEOUT);
    if (G.bad && blockIdx.x == 0) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  }
}

// ---- scales in tile order ------------------------------------------------------------

struct ScaleParams {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const int32_t* offsets;
  int S, E, N, NT;
  int steps, count;       // steps of 256 along K; scale bytes of a row (K / 32)
  int vec;                // bytes at a time that both can be read in: 16, 4 or 1
  int cols;               // of y (SILU: where the up rows start)
  uint4* x_atoms;         // [128-row blocks of x, steps, 2][32 lanes]
  uint4* w_atoms;         // [E, NT, steps, 2 blocks of 128 rows, 2][32 lanes]
};

// A warp writes four atoms (two steps) of one block of 128 rows: a lane reads 16 bytes of four
// rows, 32 apart, and writes its 16 bytes of each atom, so the writes are whole lines. Rows past
// a block's end (of the group, of the tile's 224) repeat a valid one; their results are not used.
template <bool SILU>
__global__ void __launch_bounds__(256) mxfp4_scales_kernel(const ScaleParams P) {
  __shared__ grouped::Groups G;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32)
    grouped::group_list(P.offsets, P.E, P.S, [](int rows) { return mtiles(rows) * 2; }, G);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int pairs = (P.steps + 1) / 2;
  const int x_blocks = G.start[P.E], w_blocks = P.E * P.NT * 2;
  const long units = (long)(x_blocks + w_blocks) * pairs, stride = (long)gridDim.x * (blockDim.x / 32);
  for (long u = (long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; u < units; u += stride) {
    const int block = (int)(u / pairs), step = (int)(u - (long)block * pairs) * 2;
    const uint8_t* rows[4];
    uint4* dst;
    int step_stride;        // uint4 between the atoms of one step and the next
    const uint8_t* end = block < x_blocks ? P.x_scales + (long)P.S * P.count : P.w_scales + (long)P.E * P.N * P.count;
    if (block < x_blocks) {
      const int e = grouped::find(G.start, P.E, block);
      const grouped::Span g = G.span(e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rows[i] = P.x_scales + (long)min(g.lo + (block - G.start[e]) * 128 + lane + 32 * i, P.S - 1) * P.count;
      dst = P.x_atoms + ((long)block * P.steps + step) * 2 * 32;
      step_stride = 2 * 32;
    } else {
      const int b = block - x_blocks, tile = b >> 1, e = tile / P.NT, n = tile - e * P.NT;
      if (G.start[e] == G.start[e + 1]) continue;     // no rows: no tile reads these
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = min((b & 1) * 128 + lane + 32 * i, BN - 1), h = r >= HALF;
        const int row = SILU ? n * HALF + r + h * (P.cols - HALF) : n * BN + r;
        rows[i] = P.w_scales + ((long)e * P.N + min(row, P.N - 1)) * P.count;
      }
      dst = P.w_atoms + (((long)tile * P.steps + step) * 4 + (b & 1) * 2) * 32;
      step_stride = 4 * 32;
    }
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mx::scale16(rows[i], step * 8, P.count, P.vec, end);
    dst[lane] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
    dst[32 + lane] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
    if (step + 1 < P.steps) {
      dst[step_stride + lane] = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
      dst[step_stride + 32 + lane] = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
    }
  }
}

int column_tiles(int N, bool silu) { return silu ? (N / 2 + HALF - 1) / HALF : (N + BN - 1) / BN; }
int k_steps(int K) { return (K / 2 + KB_BYTES - 1) / KB_BYTES; }
long x_atom_count(int S, int E, int steps) { return ((long)(S + 2 * BM - 1) / (2 * BM) + E) * 2 * steps * 2; }

template <bool SILU, class T>
int launch(const Mxfp4Args& a, cudaStream_t s) {
  const char* name = "mxfp4_grouped_gemm";
  if (int rc = ensure_smem_limit(mxfp4_pair_kernel<SILU, T>, DSMEM, name)) return rc;
  const int steps = k_steps(a.K), NT = column_tiles(a.N, SILU);
  const long xa = x_atom_count(a.S, a.E, steps), wa = (long)a.E * NT * steps * 4;
  Carver c(a.ws);
  uint4* x_atoms = c.take<uint4>((size_t)xa * 32);
  uint4* w_atoms = c.take<uint4>((size_t)wa * 32);
  {
    ScaleParams q{a.x_scales, a.w_scales, a.offsets, a.S, a.E, a.N, NT, steps, a.K / 32, mx::scale_vec(a.K / 32),
                  SILU ? a.N / 2 : a.N, x_atoms, w_atoms};
      ProfScope ps("mxfp4_scales", s);
    const long warps = (xa / (2 * steps) + wa / (2 * steps)) * ((steps + 1) / 2);
    const int grid = (int)std::max(1L, std::min((warps + 7) / 8, (long)num_sms() * 8));
    const cudaError_t e = launch_pdl(mxfp4_scales_kernel<SILU>, grid, 256, 0, s, q);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "mxfp4_scales: %s", cudaGetErrorString(e));
    if (int rc = check_launch("mxfp4_scales")) return rc;
  }
  CUtensorMap tx, tw, txs, tws;
  int rc;
  if ((rc = make_tmap_3d(&tx, a.x, 1, (uint64_t)a.K / 2, (uint64_t)a.S, 1, KB_BYTES, BM))) return rc;
  if ((rc = make_tmap_3d(&tw, a.w, 1, (uint64_t)a.K / 2, (uint64_t)a.N, (uint64_t)a.E, KB_BYTES, HALF))) return rc;
  if ((rc = make_tmap_atoms(&txs, x_atoms, (uint64_t)xa, 2))) return rc;
  if ((rc = make_tmap_atoms(&tws, w_atoms, (uint64_t)wa, 4))) return rc;
  Params p{};
  p.offsets = a.offsets;
  p.S = a.S;
  p.E = a.E;
  p.steps = steps;
  p.cols = SILU ? a.N / 2 : a.N;
  p.NT = NT;
  p.y = a.y;
  p.vec = grouped::store_width(a.y, p.cols, sizeof(T));
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  const long tiles = ((long)(a.S + 2 * BM - 1) / (2 * BM) + a.E) * p.NT;
  const int grid = 2 * (int)std::max(1L, std::min(tiles, (long)(num_sms() / 2)));
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(mxfp4_pair_kernel<SILU, T>, grid, THREADS, DSMEM, s, tx, tw, txs, tws, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

}  // namespace

size_t mxfp4_grouped_workspace(int S, int K, int N, int E, bool silu) {
  if (grouped_few_rows(S, E)) return 0;
  const int steps = k_steps(K);
  Carver c(nullptr);
  c.take<uint4>((size_t)x_atom_count(S, E, steps) * 32);
  c.take<uint4>((size_t)E * column_tiles(N, silu) * steps * 4 * 32);
  return align_up(c.used, 256);
}

int launch_mxfp4_grouped(const Mxfp4Args& a, cudaStream_t s) {
  if (grouped_few_rows(a.S, a.E)) return launch_mxfp4_few(a, s);
  if (a.out_dtype == MOE_F32) return a.silu ? launch<true, float>(a, s) : launch<false, float>(a, s);
  if (a.out_dtype == MOE_BF16) return a.silu ? launch<true, __nv_bfloat16>(a, s) : launch<false, __nv_bfloat16>(a, s);
  return a.silu ? launch<true, __half>(a, s) : launch<false, __half>(a, s);
}

}  // namespace moe
