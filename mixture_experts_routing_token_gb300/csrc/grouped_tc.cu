// Products grouped by expert on SM pairs, bf16 and float16 (tcgen05.mma.cta_group::2,
// M = 256 x N = 256 x K = 16, float32 accumulators in both SMs' TMEM).
//
//   ROWS   y[p, n]      = sum_k x[p, k] w[e, n, k]        A = x rows, B = w rows (both K-major)
//   GRADX  d_x[p, k]    = sum_n d_y[p, n] w[e, n, k]      A = d_y rows, B = w (MN-major)
//   GRADW  d_w[e, n, k] = sum over p of e of d_y[p, n] x[p, k]   A = d_y, B = x (both MN-major)
//
// Each SM of a 2-CTA cluster loads its own 128 of A's 256 rows and one half of B's 256
// per step of 64 of the reduction (32 KB per SM and step, six steps in flight) and holds
// its 128 rows x 256 columns of the result, twice, so the epilogue of a tile runs under
// the next tile's products. A tile is 256 rows of one expert (GRADW: 256 x 256 of its
// matrix). Bound by the tensor cores at prompt sizes; where experts have few rows, by
// the bytes of the weights.
//
// Edges need no copy of the operands:
//   - weights are a 3-D tensor [E, N, K], so what a box reads past an expert's last row
//     or column is zero fill, not the next expert;
//   - rows past a group's end inside a tile are the next expert's, but reach only their
//     own rows of the result, which are not stored;
//   - GRADW reduces over rows, so those rows have to count nothing even if they hold NaN.
//     Its last step of a group arrives on a barrier of the CTA's own; a warp (tail) clears
//     the rows past the end in shared memory (whole 128-byte lines, so the swizzle does
//     not matter) and only then hands the step to the MMA issuer.
//
// Barriers as in the FFN's pair kernel: full[s] in the leader CTA (the pair's bytes, and in
// GRADW one arrival of each CTA for a cleared step), empty[s] in both, tfull / tempty per
// accumulator. Every wait is bounded.
#include <algorithm>

#include "grouped.cuh"
#include "pair_ptx.cuh"

namespace moe {
namespace {

using namespace pair;

constexpr int BM = 128;                 // rows of A per SM (256 per pair)
constexpr int BK = 64;
constexpr int BN = 256;
constexpr int NSTAGE = 6;
constexpr int A_BYTES = BM * BK * 2;    // 16 KB
constexpr int B_BYTES = (BN / 2) * BK * 2;
constexpr int STAGE = A_BYTES + B_BYTES;
constexpr int DSMEM = NSTAGE * STAGE + 1024;
constexpr int EPI_WARPS = 4;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr uint64_t DRAIN_NS = 2000000000ull;    // issued MMAs and copies
constexpr uint32_t MN_BLOCK = 64 * BK * 2;      // bytes between the two 64-column boxes of an MN-major operand

enum { ROWS = 0, GRADX = 1, GRADW = 2 };

template <int MODE>
constexpr int threads() { return (2 + EPI_WARPS + (MODE == GRADW ? 1 : 0)) * 32; }

struct Params {
  const int32_t* offsets;
  int S, E;
  int R;            // length of the reduction (K: ROWS, N: GRADX); GRADW: the group's rows
  int M, C;         // GRADW: rows of an expert's result; columns of the result
  int MT, NT;       // tiles: GRADW rows, columns
  void* out;
  int vec;          // stores: 2 = 32-byte sectors, 1 = 16 bytes, 0 = single values
  uint32_t idesc;
  int32_t* status;
  uint64_t wait_ns;
};

struct Tile {
  int e, m, n, steps;
  grouped::Span g;
};

template <int MODE>
__device__ __forceinline__ int tiles_of(int rows, const Params& P) {
  return MODE == GRADW ? P.MT * P.NT : (rows + 2 * BM - 1) / (2 * BM) * P.NT;
}

// Tile t. Tiles of an expert that run together share the operand with fewer tiles, which
// stays in L2, while the other one is walked once.
template <int MODE>
__device__ __forceinline__ Tile tile_at(int t, const grouped::Groups& G, const Params& P) {
  Tile d;
  d.e = grouped::find(G.start, P.E, t);
  d.g = G.span(d.e);
  const int local = t - G.start[d.e];
  const int mt = MODE == GRADW ? P.MT : (d.g.rows() + 2 * BM - 1) / (2 * BM);
  if (mt > P.NT) {
    d.m = local / P.NT;
    d.n = local - d.m * P.NT;
  } else {
    d.n = local / mt;
    d.m = local - d.n * mt;
  }
  d.steps = ((MODE == GRADW ? d.g.rows() : P.R) + BK - 1) / BK;
  return d;
}

template <int MODE, class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads<MODE>(), 1)
    grouped_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const Params P) {
  __shared__ __align__(8) uint64_t full_bar[NSTAGE], empty_bar[NSTAGE], tail_bar[NSTAGE];
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
  auto sA = [&](int s) { return dsmem + (uint32_t)(s * STAGE); };
  auto sB = [&](int s) { return dsmem + (uint32_t)(s * STAGE + A_BYTES); };
  volatile int* abort_p = &abort_flag;

  if (tid == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), MODE == GRADW ? 2 : 1);
      ptx::mbar_init(ptx::smem_u32(&empty_bar[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&tail_bar[s]), 1);
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
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
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
    grouped::group_list(P.offsets, P.E, P.S, [&](int rows) { return tiles_of<MODE>(rows, P); }, G);
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
      for (int t = cluster_id; t < total; t += nclusters) {
        const Tile ti = tile_at<MODE>(t, G, P);
        const bool cut = MODE == GRADW && ti.g.rows() % BK != 0;
        for (int kb = 0; kb < ti.steps; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) goto producer_done;
          if (MODE == GRADW) {
            const int xa = ti.m * (2 * BM) + (int)rank * BM, xb = ti.n * BN + (int)rank * (BN / 2);
            const int y = ti.g.lo + kb * BK;
            if (cut && kb == ti.steps - 1) {
              const uint32_t tb = ptx::smem_u32(&tail_bar[stage]);
              ptx::mbar_arrive_expect_tx(tb, STAGE);
              ptx::tma_load_3d(sA(stage), &tmA, xa, y, 0, tb);
              ptx::tma_load_3d(sA(stage) + MN_BLOCK, &tmA, xa + 64, y, 0, tb);
              ptx::tma_load_3d(sB(stage), &tmB, xb, y, 0, tb);
              ptx::tma_load_3d(sB(stage) + MN_BLOCK, &tmB, xb + 64, y, 0, tb);
            } else {
              const uint32_t fb_local = ptx::smem_u32(&full_bar[stage]);
              if (leader) {
                ptx::mbar_arrive_expect_tx(fb_local, 2 * STAGE);
                ptx::mbar_arrive(fb_local);
              }
              const uint32_t fb = map_to_rank(fb_local, 0);
              tma_load_3d_pair(sA(stage), &tmA, xa, y, 0, fb);
              tma_load_3d_pair(sA(stage) + MN_BLOCK, &tmA, xa + 64, y, 0, fb);
              tma_load_3d_pair(sB(stage), &tmB, xb, y, 0, fb);
              tma_load_3d_pair(sB(stage) + MN_BLOCK, &tmB, xb + 64, y, 0, fb);
            }
          } else {
            const uint32_t fb_local = ptx::smem_u32(&full_bar[stage]);
            if (leader) ptx::mbar_arrive_expect_tx(fb_local, 2 * STAGE);
            const uint32_t fb = map_to_rank(fb_local, 0);
            tma_load_3d_pair(sA(stage), &tmA, kb * BK, ti.g.lo + ti.m * (2 * BM) + (int)rank * BM, 0, fb);
            if (MODE == ROWS) {
              tma_load_3d_pair(sB(stage), &tmB, kb * BK, ti.n * BN + (int)rank * (BN / 2), ti.e, fb);
            } else {
              const int x = ti.n * BN + (int)rank * (BN / 2);
              tma_load_3d_pair(sB(stage), &tmB, x, kb * BK, ti.e, fb);
              tma_load_3d_pair(sB(stage) + MN_BLOCK, &tmB, x + 64, kb * BK, ti.e, fb);
            }
          }
          if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
        }
      }
    producer_done:;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    if (leader && ptx::elect_one()) {
      constexpr int A_MN = MODE == GRADW, B_MN = MODE != ROWS;
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (int t = cluster_id; t < total; t += nclusters) {
        const Tile ti = tile_at<MODE>(t, G, P);
        if (ti.steps == 0) continue;   // nothing to add up: the epilogue writes zeros
        if (!ptx::mbar_wait(ptx::smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_p, P.wait_ns)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
        bool ok = true;
        for (int kb = 0; kb < ti.steps; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), ph, abort_p, P.wait_ns)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a0 = sA(stage), b0 = sB(stage);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = A_MN ? sdesc_mn128(a0 + kk * 2048, MN_BLOCK) : ptx::sdesc_k128(a0 + kk * 32);
            const uint64_t bd = B_MN ? sdesc_mn128(b0 + kk * 2048, MN_BLOCK) : ptx::sdesc_k128(b0 + kk * 32);
            mma_pair(d_tmem, ad, bd, P.idesc, (kb | kk) != 0);
          }
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
    T* out = static_cast<T*>(P.out);
    int acc = 0;
    uint32_t aph = 0;
    for (int t = cluster_id; t < total; t += nclusters) {
      const Tile ti = tile_at<MODE>(t, G, P);
      const int m = ti.m * (2 * BM) + (int)rank * BM + row;
      const bool mine = m < (MODE == GRADW ? P.M : ti.g.rows());
      T* dst = out + (MODE == GRADW ? (long)ti.e * P.M + m : (long)ti.g.lo + m) * P.C;
      if (ti.steps == 0) {
        uint32_t z[32] = {};
        if (mine)
          for (int c = ti.n * BN; c < min(P.C, (ti.n + 1) * BN); c += 32) grouped::store_cols(dst, c, P.C, P.vec, z);
        continue;
      }
      if (!ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns)) break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
#pragma unroll 1
      for (int c = 0; c < BN / 32; c += 2) {   // two 32-column chunks per TMEM wait
        uint32_t y[2][32];
        ptx::tmem_ld32(taddr + c * 32, y[0]);
        ptx::tmem_ld32(taddr + c * 32 + 32, y[1]);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = ti.n * BN + (c + h) * 32;
          if (mine && c0 < P.C) grouped::store_cols(dst, c0, P.C, P.vec, y[h]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&tempty_bar[acc]), 0));
      if (++acc == 2) { acc = 0; aph ^= 1u; }
    }
    if (MODE != GRADW && !*abort_p)
      grouped::zero_unowned(out, G, P.E, P.S, P.C, ((long)blockIdx.x * EPI_WARPS + warp - 2) * 32 + lane,
                            (long)gridDim.x * EPI_WARPS * 32);
  } else if (MODE == GRADW) {
    // ------------------------------------------------------------ tail (both CTAs): clears rows past a group's end
    int stage = 0;
    uint32_t tph = 0;                    // bit s: phase of tail_bar[s]
    for (int t = cluster_id; t < total; t += nclusters) {
      const Tile ti = tile_at<MODE>(t, G, P);
      if (ti.steps == 0) continue;
      const int s = (stage + ti.steps - 1) % NSTAGE;
      stage = (stage + ti.steps) % NSTAGE;
      const int keep = ti.g.rows() % BK;
      if (keep == 0) continue;
      if (!ptx::mbar_wait(ptx::smem_u32(&tail_bar[s]), (tph >> s) & 1u, abort_p, P.wait_ns)) break;
      tph ^= 1u << s;
      const int lines = (BK - keep) * 4, first = keep * 128;   // 128-byte lines to clear, in four boxes of 64
      for (int i = lane; i < lines * 8; i += 32) {
        const int line = i >> 3, box = line & 3;
        const uint32_t a = sA(s) + (uint32_t)(box * (int)MN_BLOCK + first + (line >> 2) * 128 + (i & 7) * 16);
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&full_bar[s]), 0));
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
    if (G.bad && blockIdx.x == 0) atomicOr(P.status, MOE_STATUS_BAD_INDEX);
  }
}
static_assert(A_BYTES == 2 * (int)MN_BLOCK && B_BYTES == 2 * (int)MN_BLOCK, "a stage is four boxes of 64 x 64");

template <int MODE, class T>
int launch(const CUtensorMap& a, const CUtensorMap& b, Params p, long most_tiles, cudaStream_t s, const char* name) {
  if (int rc = ensure_smem_limit(grouped_pair_kernel<MODE, T>, DSMEM, name)) return rc;
  const int grid = 2 * (int)std::max(1L, std::min(most_tiles, (long)(num_sms() / 2)));
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(grouped_pair_kernel<MODE, T>, grid, threads<MODE>(), DSMEM, s, a, b, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

template <int MODE>
int by_type(int dtype, const CUtensorMap& a, const CUtensorMap& b, Params& p, long most_tiles, cudaStream_t s,
            const char* name) {
  p.idesc = idesc_bf16_f32_major(2 * BM, BN, MODE == GRADW, MODE != ROWS);
  if (dtype == MOE_BF16) return launch<MODE, __nv_bfloat16>(a, b, p, most_tiles, s, name);
  p.idesc &= ~((1u << 7) | (1u << 10));   // A and B float16
  return launch<MODE, __half>(a, b, p, most_tiles, s, name);
}

Params params(const GroupedArgs& a, int R, int C, void* out) {
  Params p{};
  p.offsets = a.offsets;
  p.S = a.S;
  p.E = a.E;
  p.R = R;
  p.C = C;
  p.NT = (C + BN - 1) / BN;
  p.out = out;
  p.vec = grouped::store_width(out, C, 2);
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  return p;
}

long row_tiles(const GroupedArgs& a, int NT) { return ((long)(a.S + 2 * BM - 1) / (2 * BM) + a.E) * NT; }

// Rows whose bytes are not a multiple of 16 cannot be read by TMA: a copy with rows padded
// to one, zeros in between (an odd width is a small problem's; the copy is one pass over the
// operand at memory speed, against falling off the tensor cores).
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* __restrict__ src, long rows, int cols, int padded,
                                                       uint4* __restrict__ dst) {
  pdl_wait();
  pdl_trigger();
  const int P8 = padded / 8;
  const long n = rows * P8;
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x) {
    const long r = i / P8;
    const int c = (int)(i - r * P8) * 8;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? __ldg(src + r * cols + c + j) : 0u;
    dst[i] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

struct Mat {
  const void* p;
  int cols;      // of a row as stored (a multiple of 8)
};

int pad8(int c) { return (c + 7) / 8 * 8; }

// The matrix itself, or a padded copy of it in the workspace.
int padded(const void* src, long rows, int cols, Carver& c, Mat* m, cudaStream_t s) {
  *m = Mat{src, cols};
  if (cols % 8 == 0) return MOE_OK;
  m->cols = pad8(cols);
  uint16_t* dst = c.take<uint16_t>((size_t)rows * m->cols);
  m->p = dst;
  if (rows == 0) return MOE_OK;
  const long n = rows * (m->cols / 8);
  ProfScope ps("grouped_pad_rows", s);
  const int grid = (int)std::min((n + 255) / 256, (long)num_sms() * 16);
  const cudaError_t e = launch_pdl(pad_rows_kernel, grid, 256, 0, s, static_cast<const uint16_t*>(src), rows, cols,
                                   m->cols, reinterpret_cast<uint4*>(dst));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "grouped_pad_rows: %s", cudaGetErrorString(e));
  return check_launch("grouped_pad_rows");
}

}  // namespace

size_t grouped_tc_workspace(int S, int K, int N, int E, bool fwd) {
  Carver c(nullptr);
  if (K % 8 != 0) {
    c.take<uint16_t>((size_t)S * pad8(K));
    c.take<uint16_t>((size_t)E * N * pad8(K));
  }
  if (!fwd && N % 8 != 0) c.take<uint16_t>((size_t)S * pad8(N));
  return align_up(c.used, 256);
}

int launch_grouped_tc(const GroupedArgs& a, cudaStream_t s) {
  Carver c(a.ws);
  Mat x, w;
  int rc;
  if ((rc = padded(a.x, a.S, a.K, c, &x, s))) return rc;
  if ((rc = padded(a.w, (long)a.E * a.N, a.K, c, &w, s))) return rc;
  if (grouped_few_rows(a.S, a.E)) return launch_grouped_few(a, x.p, w.p, x.cols, s);
  CUtensorMap ta, tb;
  if ((rc = make_tmap_3d(&ta, x.p, 2, (uint64_t)x.cols, (uint64_t)a.S, 1, BK, BM))) return rc;
  if ((rc = make_tmap_3d(&tb, w.p, 2, (uint64_t)w.cols, (uint64_t)a.N, (uint64_t)a.E, BK, BN / 2))) return rc;
  Params p = params(a, a.K, a.N, a.y);
  return by_type<ROWS>(a.dtype, ta, tb, p, row_tiles(a, p.NT), s, "grouped_gemm");
}

int launch_grouped_tc_backward(const GroupedArgs& a, cudaStream_t s) {
  Carver c(a.ws);
  Mat dy, x, w;
  CUtensorMap ta, tb;
  int rc;
  if ((rc = padded(a.d_y, a.S, a.N, c, &dy, s))) return rc;
  if (a.d_x) {
    if ((rc = padded(a.w, (long)a.E * a.N, a.K, c, &w, s))) return rc;
    if ((rc = make_tmap_3d(&ta, dy.p, 2, (uint64_t)dy.cols, (uint64_t)a.S, 1, BK, BM))) return rc;
    if ((rc = make_tmap_3d(&tb, w.p, 2, (uint64_t)w.cols, (uint64_t)a.N, (uint64_t)a.E, 64, BK))) return rc;
    Params p = params(a, a.N, a.K, a.d_x);
    if ((rc = by_type<GRADX>(a.dtype, ta, tb, p, row_tiles(a, p.NT), s, "grouped_gemm_dx"))) return rc;
  }
  if (a.d_w) {
    if ((rc = padded(a.x, a.S, a.K, c, &x, s))) return rc;
    if ((rc = make_tmap_3d(&ta, dy.p, 2, (uint64_t)dy.cols, (uint64_t)a.S, 1, 64, BK))) return rc;
    if ((rc = make_tmap_3d(&tb, x.p, 2, (uint64_t)x.cols, (uint64_t)a.S, 1, 64, BK))) return rc;
    Params p = params(a, 0, a.K, a.d_w);
    p.M = a.N;
    p.MT = (a.N + 2 * BM - 1) / (2 * BM);
    if ((rc = by_type<GRADW>(a.dtype, ta, tb, p, (long)a.E * p.MT * p.NT, s, "grouped_gemm_dw"))) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
