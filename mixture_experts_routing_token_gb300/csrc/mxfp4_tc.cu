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
// Scales stay as the user holds them, [rows, K / 32] bytes: three warps per SM (A's rows, B's
// rows 0..127 and 128..223: both SMs need all of B's) read them four steps ahead into registers,
// write them into the ring's stage in the order tcgen05.cp expects, and arrive on the stage's
// full barrier beside the TMA bytes. Groups therefore start at any row, without a padded or
// reordered copy of the scales.
//
// Bound: the tensor cores and L2 at prompt sizes (a step moves 30 KB per SM for 448 cycles of
// products).
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
constexpr int SF_WARPS = 3;
constexpr int THREADS = (2 + EPI_WARPS + SF_WARPS) * 32;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SFA_COL = 2 * BN, SFB_COL = SFA_COL + 8;
constexpr uint64_t DRAIN_NS = 2000000000ull;
static_assert(B_BYTES == HALF * KB_BYTES && STAGE % 1024 == 0, "stage layout");
constexpr uint32_t SF_COLS = 24;          // one step's scales; two sets, taken in turn
static_assert(SFA_COL + 2 * SF_COLS <= TMEM_COLS, "tensor memory");

struct Params {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const int32_t* offsets;
  int S, E, N;      // N: rows of w
  int steps;        // of 256 along K
  int count;        // scale bytes of a row, K / 32
  int vec_x, vec_w; // how they can be read (16, 4 or 1 bytes at a time)
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

__device__ __forceinline__ Tile tile_at(int t, const int* start, const Params& P) {
  Tile d;
  d.e = grouped::find(start, P.E, t);
  d.g = grouped::span(P.offsets, d.e, P.S);
  const int local = t - start[d.e], mt = mtiles(d.g.rows());
  if (mt > P.NT) {
    d.m = local / P.NT;
    d.n = local - d.m * P.NT;
  } else {
    d.n = local / mt;
    d.m = local - d.n * mt;
  }
  return d;
}

// First row of w that block b (0 or 1, HALF rows) of tile n's B operand holds.
template <bool SILU>
__device__ __forceinline__ int w_row(int n, int b, const Params& P) {
  return SILU ? n * HALF + b * P.cols : n * BN + b * HALF;
}

// silu(z) = z / (1 + e^-z) with the approximate division (2 ulp; results below 2^-119 in
// magnitude, z < -87, become 0): with the IEEE division the epilogue took 12.9k cycles a tile,
// three and a half times the products.
__device__ __forceinline__ float silu_fast(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

template <bool SILU, class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const Params P) {
  __shared__ __align__(8) uint64_t full_bar[NSTAGE], empty_bar[NSTAGE];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, bad_flag;
  __shared__ int start[MOE_MAX_EXPERTS + 1];
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
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), 1 + 2 * SF_WARPS);
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
    grouped::tile_list(P.offsets, P.E, P.S, [&](int rows) { return mtiles(rows) * P.NT; }, start, &bad_flag);
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();      // barriers of both CTAs initialised before any cross-CTA signal
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int total = start[P.E];

  if (warp == 0) {
    // ------------------------------------------------------------ producer of codes (both CTAs)
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = cluster_id; t < total && ok; t += nclusters) {
        const Tile ti = tile_at(t, start, P);
        const int a_row = ti.g.lo + ti.m * (2 * BM) + (int)rank * BM, b_row = w_row<SILU>(ti.n, (int)rank, P);
        for (int kb = 0; kb < P.steps; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = ptx::smem_u32(&full_bar[stage]);
          if (leader) ptx::mbar_arrive_expect_tx(fb_local, 2 * (A_BYTES + B_BYTES));
          const uint32_t fb = map_to_rank(fb_local, 0);
          tma_load_3d_pair(st(stage), &tmX, kb * KB_BYTES, a_row, 0, fb);
          tma_load_3d_pair(st(stage) + A_BYTES, &tmW, kb * KB_BYTES, b_row, ti.e, fb);
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
      for (int t = cluster_id; t < total; t += nclusters) {
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
  } else if (warp < 2 + EPI_WARPS) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;              // TMEM lane quarter this warp may read
    const int row = q * 32 + lane;
    T* y = static_cast<T*>(P.y);
    int acc = 0;
    uint32_t aph = 0;
    for (int t = cluster_id; t < total; t += nclusters) {
      const Tile ti = tile_at(t, start, P);
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
              g[i] = __float_as_uint(silu_fast(__uint_as_float(g[i])) * __uint_as_float(u[i]));
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
          if (mine && c0 < P.cols) grouped::store_cols(dst, c0, P.cols, P.vec, v);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&tempty_bar[acc]), 0));
      if (++acc == 2) { acc = 0; aph ^= 1u; }
    }
    if (!*abort_p)
      grouped::zero_unowned(y, P.offsets, P.E, P.S, P.cols, ((long)blockIdx.x * EPI_WARPS + warp - 2) * 32 + lane,
                            (long)gridDim.x * EPI_WARPS * 32);
  } else {
    // ------------------------------------------------------------ scales (both CTAs)
    const int part = warp - 2 - EPI_WARPS;        // 0: A's rows; 1, 2: rows 0..127, 128..223 of the tile's B
    const uint32_t off = part == 0 ? SFA_OFF : SFB_OFF + (uint32_t)(part - 1) * 2 * mx::SF_ATOM;
    const int vec = part == 0 ? P.vec_x : P.vec_w;
    const uint8_t* rows[4];
    auto point = [&](int t) {                     // this lane's four rows of tile t (clamped: extra rows are not stored)
      const Tile ti = tile_at(t, start, P);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane + 32 * i;
        if (part == 0) {
          rows[i] = P.x_scales + (long)min(ti.g.lo + ti.m * (2 * BM) + (int)rank * BM + r, P.S - 1) * P.count;
        } else {
          const int b = min((part - 1) * 128 + r, BN - 1), h = b >= HALF;
          const int n = min(w_row<SILU>(ti.n, h, P) + b - h * HALF, P.N - 1);
          rows[i] = P.w_scales + ((long)ti.e * P.N + n) * P.count;
        }
      }
    };
    mx::ScaleRegs cur, next;
    int t = cluster_id, kb = 0, stage = 0;
    uint32_t ph = 0;
    if (t < total) {
      point(t);
      mx::load_scales(cur, rows, 0, P.count, vec);
    }
    bool ok = true;
    while (t < total && ok) {
      // request the next chunk, then hand over this one as stages come free
      int nt = t, nkb = kb + mx::CHUNK;
      if (nkb >= P.steps) {
        nkb = 0;
        nt = t + nclusters;
        if (nt < total) point(nt);
      }
      if (nt < total) mx::load_scales(next, rows, nkb, P.count, vec);
#pragma unroll
      for (int d = 0; d < mx::CHUNK; ++d) {
        if (kb + d < P.steps && ok) {
          ok = ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            mx::store_scales(cur, d, st(stage) + off, mx::SF_ATOM, lane);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&full_bar[stage]), 0));
            if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
          }
        }
      }
      cur = next;
      t = nt;
      kb = nkb;
    }
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
    if (bad_flag && blockIdx.x == 0) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  }
}

template <bool SILU, class T>
int launch(const Mxfp4Args& a, cudaStream_t s) {
  const char* name = "mxfp4_grouped_gemm";
  if (int rc = ensure_smem_limit(mxfp4_pair_kernel<SILU, T>, DSMEM, name)) return rc;
  CUtensorMap tx, tw;
  int rc;
  if ((rc = make_tmap_3d(&tx, a.x, 1, (uint64_t)a.K / 2, (uint64_t)a.S, 1, KB_BYTES, BM))) return rc;
  if ((rc = make_tmap_3d(&tw, a.w, 1, (uint64_t)a.K / 2, (uint64_t)a.N, (uint64_t)a.E, KB_BYTES, HALF))) return rc;
  Params p{};
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.offsets = a.offsets;
  p.S = a.S;
  p.E = a.E;
  p.N = a.N;
  p.steps = (a.K / 2 + KB_BYTES - 1) / KB_BYTES;
  p.count = a.K / 32;
  p.vec_x = mx::scale_vec(a.x_scales, p.count);
  p.vec_w = mx::scale_vec(a.w_scales, p.count);
  p.cols = SILU ? a.N / 2 : a.N;
  p.NT = SILU ? (p.cols + HALF - 1) / HALF : (p.cols + BN - 1) / BN;
  p.y = a.y;
  p.vec = grouped::store_width(a.y, p.cols, sizeof(T));
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  const long tiles = ((long)(a.S + 2 * BM - 1) / (2 * BM) + a.E) * p.NT;
  const int grid = 2 * (int)std::max(1L, std::min(tiles, (long)(num_sms() / 2)));
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(mxfp4_pair_kernel<SILU, T>, grid, THREADS, DSMEM, s, tx, tw, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

}  // namespace

int launch_mxfp4_grouped(const Mxfp4Args& a, cudaStream_t s) {
  if (a.out_dtype == MOE_F32) return a.silu ? launch<true, float>(a, s) : launch<false, float>(a, s);
  if (a.out_dtype == MOE_BF16) return a.silu ? launch<true, __nv_bfloat16>(a, s) : launch<false, __nv_bfloat16>(a, s);
  return a.silu ? launch<true, __half>(a, s) : launch<false, __half>(a, s);
}

}  // namespace moe
