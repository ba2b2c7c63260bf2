// Products grouped by expert on SM pairs, bf16, float16 and float32 (tcgen05.mma.cta_group::2,
// kind::f16, M = 256 x N = 256 x K = 16, float32 accumulators in both SMs' TMEM).
//
//   y[p, n]      = sum_k x[p, k] w[e, n, k]               A = x rows, B = w rows (both K-major)
//   d_x[p, k]    = sum_n d_y[p, n] w[e, n, k]             A = d_y rows, B = w (MN-major)
//   d_w[e, n, k] = sum over p of e of d_y[p, n] x[p, k]   A = d_y, B = x (both MN-major)
//
// The two gradients are the tiles of one launch, the ones with the longer reduction first: small
// problems fill the SMs better and pay one start (1554 rows, 16 experts of [714, 1000]: two launches
// took 28 us).
//
// Each SM of a 2-CTA cluster loads its own 128 of A's 256 rows and one half of B's 256
// per step of 64 of the reduction (32 KB per SM and step, six steps in flight) and holds
// its 128 rows x 256 columns of the result, twice, so the epilogue of a tile runs under
// the next tile's products. A tile is 256 rows of one expert (d_w: 256 x 256 of its
// matrix). Bound by the tensor cores at prompt sizes; where experts have few rows, by
// the bytes of the weights.
//
// Edges need no copy of the operands:
//   - weights are a 3-D tensor [E, N, K], so what a box reads past an expert's last row
//     or column is zero fill, not the next expert;
//   - rows past a group's end inside a tile are the next expert's, but reach only their
//     own rows of the result, which are not stored;
//   - d_w reduces over rows, so those rows have to count nothing even if they hold NaN.
//     Its last step of a group arrives on a barrier of the CTA's own; a warp (tail) clears
//     the rows past the end in shared memory (whole 128-byte lines, so the swizzle does
//     not matter) and only then hands the step to the MMA issuer.
//
// float32. A value is h + m + l, three bf16 parts of 8 bits each (all of its 24; a first kernel writes
// the parts into the workspace), and a product of two values the six
// products of parts hl + lh + mm + hm + mh + hh, each exact in float32; the three left out are below
// 2^-25 of it. The tensor cores add to an accumulator with truncation, 2^-24 of it on average and
// always toward zero, which a float32 result must not collect over a long reduction (measured on
// bf16 operands: 5e-7 at 512 terms, 9e-6 at 8192). So an accumulator holds two steps (K = 128, the
// small products first) and is then added in registers, rounded to nearest, by eight epilogue warps
// with 128 sums a thread, while the next two steps go into the other one. The parts are those of 2^16 times
// the value: every float32 is a multiple of 2^-149, bf16 ends at 2^-133, so the smallest keep all their
// bits; the sums take 2^-32 back on their way into the registers, in the addition (fma). Parts make no sense
// of infinities and NaN, and leading parts may be larger than their values by 2^-8, so that sums of their
// products leave float32's range where those of the values do not: below 2^44 a value (2^60 with the factor),
// 128 products stay below 2^127 (1 + 2^-8)^2. The first kernel flags what lies above, and then this one leaves
// everything to the kernel on the CUDA cores, which follows.
//
// Barriers as in the FFN's pair kernel: full[s] in the leader CTA (the pair's bytes, and in
// the gradients one arrival of each CTA for a cleared step), empty[s] in both, tfull / tempty per
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
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr uint64_t DRAIN_NS = 2000000000ull;    // issued MMAs and copies
constexpr uint32_t MN_BLOCK = 64 * BK * 2;      // bytes between the two 64-column boxes of an MN-major operand

template <class T>
constexpr bool is_f32() { return sizeof(T) == 4; }
template <class T>
constexpr int epi_warps() { return is_f32<T>() ? 8 : 4; }
template <bool GRAD, class T>
constexpr int threads() { return (2 + epi_warps<T>() + (GRAD ? 1 : 0)) * 32; }
// The ring and, for 16-bit results, the epilogue's buffers.
template <class T>
constexpr int dsmem_bytes() { return NSTAGE * STAGE + (is_f32<T>() ? 0 : 4 * 4096) + 1024; }

// One product over the groups.
struct Job {
  int R;            // length of the reduction; d_w: the group's rows (0 here)
  int C, NT;        // columns of the result, tiles of them
  int M, MT;        // d_w: rows of an expert's result, tiles of them
  void* out;        // null: not wanted
  int vec;          // stores: > 0 = rows are a multiple of 16 bytes, 0 = single values
  uint32_t idesc;
};

struct Params {
  const int32_t* offsets;
  int S, E;
  Job rows;         // y or d_x
  Job dw;           // d_w
  int dw_first;
  const int* flags;   // float32: grouped::any_flag
  int32_t* status;
  uint64_t wait_ns;
};

struct Tile {
  bool dw;
  int e, m, n, blocks;      // blocks: of 64 along the reduction
  grouped::Span g;
};

constexpr float kPartScale = 65536.0f, kSumScale = 1.0f / (65536.0f * 65536.0f);   // float32 in parts

// Steps of a tile: its blocks, in order; in float32 two blocks (or the odd last one) at a time, with
// six products of parts.
template <class T>
__device__ __forceinline__ int step_count(int blocks) { return is_f32<T>() ? 6 * blocks : blocks; }

struct Step {
  int block, pa, pb;        // parts of A and B
  bool first, last;         // of an accumulator
};

template <class T>
__device__ __forceinline__ Step step_at(int s, int blocks) {
  if (!is_f32<T>()) return Step{s, 0, 0, s == 0, s == blocks - 1};
  const int pairs = blocks >> 1;
  Step d;
  int p;
  if (s < pairs * 12) {
    const int c = s / 12, r = s - c * 12;
    p = r >> 1;
    d.block = 2 * c + (r & 1);
    d.first = r == 0;
    d.last = r == 11;
  } else {
    p = s - pairs * 12;
    d.block = blocks - 1;
    d.first = p == 0;
    d.last = p == 5;
  }
  d.pa = (0x010120 >> (4 * p)) & 3;     // h m h m l h, with
  d.pb = (0x001102 >> (4 * p)) & 3;     // h h m m h l, from the last to the first
  return d;
}

// Where a role is in the list of tiles: experts of its last tiles of either kind.
struct At {
  int e_rows = 0, e_dw = 0;
};

// Tile t. Tiles of an expert that run together share the operand with fewer tiles, which
// stays in L2, while the other one is walked once.
template <bool GRAD>
__device__ __forceinline__ Tile tile_at(int t, At& at, const grouped::Groups& G, int dw_tiles, const Params& P) {
  Tile d;
  const int row_tiles = G.start[P.E];
  d.dw = GRAD && (P.dw_first ? t < dw_tiles : t >= row_tiles);
  int mt, local;
  if (d.dw) {
    if (!P.dw_first) t -= row_tiles;
    const int per = P.dw.MT * P.dw.NT;
    while (t >= (at.e_dw + 1) * per) ++at.e_dw;
    d.e = at.e_dw;
    d.g = G.span(d.e);
    local = t - d.e * per;
    mt = P.dw.MT;
    d.blocks = (d.g.rows() + BK - 1) / BK;
  } else {
    if (P.dw_first) t -= dw_tiles;
    at.e_rows = grouped::find_from(G.start, at.e_rows, t);
    d.e = at.e_rows;
    d.g = G.span(d.e);
    local = t - G.start[d.e];
    mt = (d.g.rows() + 2 * BM - 1) / (2 * BM);
    d.blocks = (P.rows.R + BK - 1) / BK;
  }
  const int NT = d.dw ? P.dw.NT : P.rows.NT;
  if (mt > NT) {
    d.m = grouped::quick_div(local, NT);
    d.n = local - d.m * NT;
  } else {
    d.n = grouped::quick_div(local, mt);
    d.m = local - d.n * mt;
  }
  return d;
}

// GRAD = false: P.rows is y, tmA / tmB its operands. GRAD: P.rows is d_x (tmA, tmB), P.dw d_w (tmC, tmD).
// tmRows, tmDw: the outputs, where they are 16-bit and stored by TMA.
template <bool GRAD, class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads<GRAD, T>(), 1)
    grouped_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD,
                        const __grid_constant__ CUtensorMap tmRows, const __grid_constant__ CUtensorMap tmDw,
                        const Params P) {
  __shared__ __align__(8) uint64_t full_bar[NSTAGE], empty_bar[NSTAGE], tail_bar[NSTAGE];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ grouped::Groups G;
  __shared__ int skip;
  extern __shared__ uint8_t dsmem_raw[];
  constexpr bool F32 = is_f32<T>();
  constexpr int EPI_WARPS = epi_warps<T>();

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
      ptx::mbar_init(ptx::smem_u32(&full_bar[s]), GRAD ? 2 : 1);
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
    if (GRAD) {
      ptx::prefetch_tmap(&tmC);
      ptx::prefetch_tmap(&tmD);
    }
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
    grouped::group_list(P.offsets, P.E, P.S,
                        [&](int rows) { return P.rows.out ? (rows + 2 * BM - 1) / (2 * BM) * P.rows.NT : 0; }, G);
  if (F32 && warp == 3) {
    const int any = __any_sync(0xffffffffu, grouped::any_flag<32>(P.flags, lane));
    if (lane == 0) skip = any;
  }
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();      // barriers of both CTAs initialised before any cross-CTA signal
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int dw_tiles = GRAD && P.dw.out ? P.E * P.dw.MT * P.dw.NT : 0;
  const int total = F32 && skip ? 0 : G.start[P.E] + dw_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (ptx::elect_one()) {
      At at;
      int stage = 0;
      uint32_t ph = 0;
      for (int t = cluster_id; t < total; t += nclusters) {
        const Tile ti = tile_at<GRAD>(t, at, G, dw_tiles, P);
        const bool cut = ti.dw && ti.g.rows() % BK != 0;
        const int xb = ti.n * BN + (int)rank * (BN / 2);
        const int steps = step_count<T>(ti.blocks);
        for (int s = 0; s < steps; ++s) {
          if (!ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), ph ^ 1u, abort_p, P.wait_ns)) goto producer_done;
          const Step sp = step_at<T>(s, ti.blocks);
          if (cut && sp.block == ti.blocks - 1) {
            const int xa = ti.m * (2 * BM) + (int)rank * BM, y = ti.g.lo + sp.block * BK;
            const uint32_t tb = ptx::smem_u32(&tail_bar[stage]);
            ptx::mbar_arrive_expect_tx(tb, STAGE);
            ptx::tma_load_3d(sA(stage), &tmC, xa, y, sp.pa, tb);
            ptx::tma_load_3d(sA(stage) + MN_BLOCK, &tmC, xa + 64, y, sp.pa, tb);
            ptx::tma_load_3d(sB(stage), &tmD, xb, y, sp.pb, tb);
            ptx::tma_load_3d(sB(stage) + MN_BLOCK, &tmD, xb + 64, y, sp.pb, tb);
          } else {
            const uint32_t fb_local = ptx::smem_u32(&full_bar[stage]);
            if (leader) {
              ptx::mbar_arrive_expect_tx(fb_local, 2 * STAGE);
              if (GRAD) ptx::mbar_arrive(fb_local);
            }
            const uint32_t fb = map_to_rank(fb_local, 0);
            if (GRAD && ti.dw) {
              const int xa = ti.m * (2 * BM) + (int)rank * BM, y = ti.g.lo + sp.block * BK;
              tma_load_3d_pair(sA(stage), &tmC, xa, y, sp.pa, fb);
              tma_load_3d_pair(sA(stage) + MN_BLOCK, &tmC, xa + 64, y, sp.pa, fb);
              tma_load_3d_pair(sB(stage), &tmD, xb, y, sp.pb, fb);
              tma_load_3d_pair(sB(stage) + MN_BLOCK, &tmD, xb + 64, y, sp.pb, fb);
            } else {
              const int k = sp.block * BK, mat = ti.e + sp.pb * P.E;
              tma_load_3d_pair(sA(stage), &tmA, k, ti.g.lo + ti.m * (2 * BM) + (int)rank * BM, sp.pa, fb);
              if (GRAD) {
                tma_load_3d_pair(sB(stage), &tmB, xb, k, mat, fb);
                tma_load_3d_pair(sB(stage) + MN_BLOCK, &tmB, xb + 64, k, mat, fb);
              } else {
                tma_load_3d_pair(sB(stage), &tmB, k, xb, mat, fb);
              }
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
      At at;
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (int t = cluster_id; t < total; t += nclusters) {
        const Tile ti = tile_at<GRAD>(t, at, G, dw_tiles, P);
        const uint32_t idesc = ti.dw ? P.dw.idesc : P.rows.idesc;
        const int steps = step_count<T>(ti.blocks);   // 0: the epilogue writes zeros
        bool ok = true;
        uint32_t d_tmem = 0;
        for (int s = 0; s < steps; ++s) {
          const Step sp = step_at<T>(s, ti.blocks);
          if (sp.first) {
            ok = ptx::mbar_wait(ptx::smem_u32(&tempty_bar[acc]), aph ^ 1u, abort_p, P.wait_ns);
            if (!ok) break;
            ptx::tc_fence_after();
            d_tmem = tmem_base + (uint32_t)(acc * BN);
          }
          ok = ptx::mbar_wait(ptx::smem_u32(&full_bar[stage]), ph, abort_p, P.wait_ns);
          if (!ok) break;
          // a step that the tail warps cleared, the other CTA's among them
          if (GRAD && ti.dw && sp.block == ti.blocks - 1 && ti.g.rows() % BK != 0)
            acquire_cluster(ptx::smem_u32(&full_bar[stage]), ph);
          ptx::tc_fence_after();
          const uint32_t a0 = sA(stage), b0 = sB(stage);
          // descriptors of the step's first MMA; K-major operands advance 32 bytes a K = 16, MN-major 2 KB
          const bool a_mn = GRAD && ti.dw;
          const uint64_t ad = a_mn ? sdesc_mn128(a0, MN_BLOCK) : ptx::sdesc_k128(a0);
          const uint64_t bd = GRAD ? sdesc_mn128(b0, MN_BLOCK) : ptx::sdesc_k128(b0);
          const uint32_t a_step = (a_mn ? 2048u : 32u) >> 4, b_step = (GRAD ? 2048u : 32u) >> 4;
          // d_w: no steps past the group's last row, of which the tail warp clears less then: 64 rows, 16
          // experts of [2048, 2048], 31 us instead of 37 (float32, six products a block: 4% slower, not done)
          const int left = GRAD && !F32 && ti.dw ? ti.g.rows() - sp.block * BK : BK;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            if (kk * 16 < left) mma_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc, !sp.first || kk != 0);
          commit_pair(ptx::smem_u32(&empty_bar[stage]), 0x3);
          if (++stage == NSTAGE) { stage = 0; ph ^= 1u; }
          if (sp.last) {
            commit_pair(ptx::smem_u32(&tfull_bar[acc]), 0x3);
            if (++acc == 2) { acc = 0; aph ^= 1u; }
          }
        }
        if (!ok) break;
      }
      commit_pair(ptx::smem_u32(&drain_bar), 0x1);
      int dummy = 0;
      ptx::mbar_wait(ptx::smem_u32(&drain_bar), 0, &dummy, DRAIN_NS);
    }
  } else if (warp < 2 + EPI_WARPS) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;              // TMEM lane quarter this warp may read
    const int row = q * 32 + lane;
    const uint32_t sbuf = dsmem + NSTAGE * STAGE + (uint32_t)q * 4096u;
    At at;
    int acc = 0;
    uint32_t aph = 0;
    bool zeroed = false;      // the buffer holds zeros
    for (int t = cluster_id; t < total; t += nclusters) {
      const Tile ti = tile_at<GRAD>(t, at, G, dw_tiles, P);
      const Job& J = ti.dw ? P.dw : P.rows;
      const int m = ti.m * (2 * BM) + (int)rank * BM + row;
      const int nrows = (ti.dw ? J.M : ti.g.rows()) - (m - lane);     // of this warp's 32 (from lane 0 on)
      const bool mine = lane < nrows;
      T* dst = static_cast<T*>(J.out) + (ti.dw ? (long)ti.e * J.M + m : (long)ti.g.lo + m) * J.C;
      if (ti.blocks == 0) {
        // d_w of an expert without rows: a buffer of zeros sent as often as the tile asks (18 rows, 113 experts of
        // [512, 2048], 41 us; by the stretch 46), or this warp's share of the zeros as one stretch of memory
        // (4 rows, 32 experts of [714, 1030], 24 us; by the tile's rows 45; float32 by the
        // tile's rows: the stretch cost its other tiles 8%)
        if (!F32 && J.vec > 0) {
          if (!zeroed) {
            if (lane == 0) ptx::tma_store_wait_read();
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 8; ++p)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sbuf + lane * 128 + p * 16), "r"(0) : "memory");
            fence_async_shared();
            __syncwarp();
            zeroed = true;
          }
          if (lane == 0 && nrows > 0)
            for (int c = ti.n * BN; c < min(J.C, (ti.n + 1) * BN); c += 64) ptx::tma_store_3d(&tmDw, sbuf, c, m, ti.e);
        } else if constexpr (F32) {
          T* row0 = dst - (long)lane * J.C;
          if (warp < 6)
            for (int r = 0; r < min(32, nrows); ++r)
              for (int c = ti.n * BN + lane; c < min(J.C, (ti.n + 1) * BN); c += 32) row0[(long)r * J.C + c] = from_float<T>(0.0f);
        } else {
          constexpr int W = 2 * EPI_WARPS;
          const long all = (long)J.M * J.C, shares = (long)J.MT * J.NT * W;
          const long share = ((all + shares - 1) / shares + 7) / 8 * 8;
          const long from = ((long)(ti.m * J.NT + ti.n) * W + (int)rank * EPI_WARPS + warp - 2) * share;
          if (from < all) grouped::zero_values(static_cast<T*>(J.out) + ti.e * all + from, (int)min(share, all - from));
        }
        continue;
      }
      zeroed = false;
      if constexpr (F32) {
        // this warp's 128 of the 256 columns, over the accumulators of the tile
        const int half = (warp - 2) >> 2;
        float sum[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
        bool ok = true;
        for (int left = (ti.blocks + 1) >> 1; left > 0; --left) {
          ok = ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + half * 128);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t y[32];
            ptx::tmem_ld32(taddr + c * 32, y);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c * 32 + j] = fmaf(__uint_as_float(y[j]), kSumScale, sum[c * 32 + j]);
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&tempty_bar[acc]), 0));
          if (++acc == 2) { acc = 0; aph ^= 1u; }
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t y[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(sum[c * 32 + j]);
          const int c0 = ti.n * BN + half * 128 + c * 32;
          if (J.vec > 0) {
            if (mine && c0 < J.C) grouped::store_cols(dst, c0, J.C, J.vec, y);
          } else if (nrows > 0 && c0 < J.C) {
            grouped::store_turned(y, dst - (long)lane * J.C, nrows, c0, J.C);
          }
        }
        continue;
      }
      if (!ptx::mbar_wait(ptx::smem_u32(&tfull_bar[acc]), aph, abort_p, P.wait_ns)) break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
#pragma unroll 1
      for (int c = 0; c < BN; c += 64) {
        uint32_t y[2][32];
        ptx::tmem_ld32(taddr + c, y[0]);
        ptx::tmem_ld32(taddr + c + 32, y[1]);
        ptx::tmem_ld_wait();
        const int c0 = ti.n * BN + c;
        if (nrows <= 0 || c0 >= J.C) continue;
        uint32_t words[32];
        grouped::pack_words<T, 32>(y[0], words);
        grouped::pack_words<T, 32>(y[1], words + 16);
        T* row0 = dst - (long)lane * J.C;
        if (J.vec > 0) {
          // d_w: the tensor's own edge ends the rows; y, d_x: the group does, so a box needs all of its 32
          grouped::store_rows(sbuf, words, ti.dw ? &tmDw : &tmRows, c0, ti.dw ? m - lane : ti.g.lo + m - lane, ti.dw ? ti.e : 0,
                              ti.dw || nrows >= 32, row0, nrows, J.C);
        } else {
          grouped::store_ragged(sbuf, words, row0, nrows, c0, J.C);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(map_to_rank(ptx::smem_u32(&tempty_bar[acc]), 0));
      if (++acc == 2) { acc = 0; aph ^= 1u; }
    }
    if (lane == 0) ptx::tma_store_wait();
    if (P.rows.out != nullptr && !*abort_p)
      grouped::zero_unowned(static_cast<T*>(P.rows.out), G, P.E, P.S, P.rows.C,
                            ((long)blockIdx.x * EPI_WARPS + warp - 2) * 32 + lane, (long)gridDim.x * EPI_WARPS * 32);
  } else if (GRAD) {
    // ------------------------------------------------------------ tail (both CTAs): clears rows past a group's end
    At at;
    int stage = 0;
    uint32_t tph = 0;                    // bit s: phase of tail_bar[s]
    for (int t = cluster_id; t < total; t += nclusters) {
      const Tile ti = tile_at<GRAD>(t, at, G, dw_tiles, P);
      const int first = stage, keep = ti.g.rows() % BK;
      stage = (stage + step_count<T>(ti.blocks)) % NSTAGE;
      if (!ti.dw || keep == 0) continue;
      bool ok = true;
      for (int p = 0; p < (F32 ? 6 : 1) && ok; ++p) {      // the last block's steps
        const int at_step = !F32 ? ti.blocks - 1 : ti.blocks & 1 ? (ti.blocks - 1) * 6 + p : (ti.blocks - 2) * 6 + 2 * p + 1;
        const int s = (first + at_step) % NSTAGE;
        ok = ptx::mbar_wait(ptx::smem_u32(&tail_bar[s]), (tph >> s) & 1u, abort_p, P.wait_ns);
        if (!ok) break;
        tph ^= 1u << s;
        // 128-byte lines to clear, in four boxes of 64: the MMAs' rows past the group's
        const int lines = (F32 ? BK - keep : (16 - keep % 16) % 16) * 4;
        for (int i = lane; i < lines * 8; i += 32) {
          const int line = i >> 3, box = line & 3;
          const uint32_t a = sA(s) + (uint32_t)(box * (int)MN_BLOCK + (keep + (line >> 2)) * 128 + (i & 7) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) arrive_remote_release(map_to_rank(ptx::smem_u32(&full_bar[s]), 0));
      }
      if (!ok) break;
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

template <bool GRAD, class T>
int launch(const CUtensorMap (&m)[4], const GroupedArgs& a, const Params& p, long most_tiles, cudaStream_t s, const char* name) {
  if (int rc = ensure_smem_limit(grouped_pair_kernel<GRAD, T>, dsmem_bytes<T>(), name)) return rc;
  const int grid = 2 * (int)std::max(1L, std::min(most_tiles, (long)(num_sms() / 2)));
  CUtensorMap rows = m[0], dw = m[0];      // not used where the job is not wanted or not stored by TMA
  if (!is_f32<T>()) {
    int rc;
    if (p.rows.out && p.rows.vec && (rc = make_tmap_3d(&rows, p.rows.out, 2, (uint64_t)p.rows.C, (uint64_t)a.S, 1, 64, 32)))
      return rc;
    if (p.dw.out && p.dw.vec &&
        (rc = make_tmap_3d(&dw, p.dw.out, 2, (uint64_t)p.dw.C, (uint64_t)p.dw.M, (uint64_t)a.E, 64, 32)))
      return rc;
  }
  ProfScope ps(name, s);
  const cudaError_t e = launch_pdl(grouped_pair_kernel<GRAD, T>, grid, threads<GRAD, T>(), dsmem_bytes<T>(), s, m[0], m[1],
                                   m[2], m[3], rows, dw, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

Job job(int dtype, int R, int C, void* out, int a_mn, int b_mn) {
  Job j{};
  j.R = R;
  j.C = C;
  j.NT = (C + BN - 1) / BN;
  j.out = out;
  j.vec = grouped::store_width(out, C, dtype == MOE_F32 ? 4 : 2);
  j.idesc = idesc_bf16_f32_major(2 * BM, BN, a_mn, b_mn);
  if (dtype == MOE_F16) j.idesc &= ~((1u << 7) | (1u << 10));   // A and B float16
  return j;
}

long row_tiles(const GroupedArgs& a, int NT) { return ((long)(a.S + 2 * BM - 1) / (2 * BM) + a.E) * NT; }

struct Mat {
  const void* p;
  int cols;      // of a row as stored (a multiple of 8)
};

int pad8(int c) { return (c + 7) / 8 * 8; }

// Rows whose bytes are not a multiple of 16 cannot be read by TMA: copies with rows padded to one,
// zeros in between (the copy is one pass over the operand at
// memory speed, against falling off the tensor cores).
struct Pad {
  const uint16_t* src;
  uint4* dst;
  long n;               // pieces of 8 columns
  int cols, pieces;     // columns; pieces of a row
  int per;              // rows of an expert's matrix (0: not by expert)
  uintptr_t end;        // of the matrix
};

// The experts that have rows, in shared memory: nothing reads the weights of the others, and a few
// tokens reach few experts. (A group needs offsets[e] < offsets[e + 1], whatever the list is like.)
struct Live {
  uint16_t expert[MOE_MAX_EXPERTS];
  int count;
  int lo, hi;       // the rows that some group owns (off[0] and off[E] of grouped::group_list)
};

// Whole block.
__device__ __forceinline__ void live_list(const int32_t* offsets, int E, int S, Live& live) {
  if (threadIdx.x < 32) {
    int n = 0, top = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + (int)threadIdx.x;
      const int a = e < E ? __ldg(offsets + e) : 0, b = e < E ? __ldg(offsets + e + 1) : 0;
      const bool on = a < b;
      top = max(top, max(a, b));
      const unsigned m = __ballot_sync(0xffffffffu, on);
      if (on) live.expert[n + __popc(m & ((1u << threadIdx.x) - 1u))] = (uint16_t)e;
      n += __popc(m);
      if (e == 0) live.lo = min(max(a, 0), S);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (threadIdx.x == 0) {
      live.count = n;
      live.hi = min(top, S);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ long div_by(long n, int d) {
  return n < (1L << 31) ? (long)((uint32_t)n / (uint32_t)d) : n / d;
}

// Pieces of a matrix that some group reads: rows that one owns, or, where it is by expert, those of live experts.
__device__ __forceinline__ long live_pieces(int pieces, int per, const Live& live) {
  return (long)(per ? (long)live.count * per : live.hi - live.lo) * pieces;
}

// Row and piece of the i-th of them.
__device__ __forceinline__ long piece_row(long i, int pieces, int per, const Live& live, int& piece) {
  long r = div_by(i, pieces);
  piece = (int)(i - r * pieces);
  if (per) {
    const long k = div_by(r, per);
    return r + (live.expert[k] - k) * per;
  }
  return r + live.lo;
}

// Eight 16-bit values from p on, of which the first `count` are wanted (zeros else), as words: two aligned
// 16-byte loads, shifted by whole words and then by half of one, where both lie before `end`. 8192 rows,
// 8 experts of [2047, 1001]: 63 us, with eight single loads a piece 66.
__device__ __forceinline__ uint4 load_any(const uint16_t* p, int count, uintptr_t end) {
  uint32_t v[4];
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), base = a & ~(uintptr_t)15;
  if (base + 32 <= end) {
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(base)), hi = __ldg(reinterpret_cast<const uint4*>(base) + 1);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int by = (int)(a - base);
    uint32_t two[6], one[5];
#pragma unroll
    for (int j = 0; j < 6; ++j) two[j] = by & 8 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) one[j] = by & 4 ? two[j + 1] : two[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = by & 2 ? __byte_perm(one[j], one[j + 1], 0x5432) : one[j];
      if (count < 2 * j + 2) v[j] = count > 2 * j ? v[j] & 0xffffu : 0u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = (2 * j < count ? (uint32_t)__ldg(p + 2 * j) : 0u) | (2 * j + 1 < count ? (uint32_t)__ldg(p + 2 * j + 1) << 16 : 0u);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

struct PadParams {
  const int32_t* offsets;
  int E, S;
  Pad m[3];
  int count;
};

__global__ void __launch_bounds__(256) pad_rows_kernel(const PadParams P) {
  __shared__ Live live;
  pdl_wait();
  pdl_trigger();
  live_list(P.offsets, P.E, P.S, live);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k >= P.count) break;
    const Pad M = P.m[k];
    const long n = live_pieces(M.pieces, M.per, live);
    for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x) {
      int piece;
      const long r = piece_row(i, M.pieces, M.per, live, piece);
      const int c = piece * 8;
      M.dst[r * M.pieces + piece] = load_any(M.src + r * M.cols + c, M.cols - c, M.end);
    }
  }
}

// The matrix itself, or the place of its padded copy in the workspace (made by launch_pads).
void padded(PadParams& p, const void* src, long rows, int cols, int per, Carver& c, Mat* m) {
  *m = Mat{src, cols};
  if (cols % 8 == 0) return;
  m->cols = pad8(cols);
  uint16_t* dst = c.take<uint16_t>((size_t)rows * m->cols);
  m->p = dst;
  const int pieces = m->cols / 8;
  p.m[p.count++] = Pad{static_cast<const uint16_t*>(src), reinterpret_cast<uint4*>(dst), rows * pieces, cols, pieces, per,
                     reinterpret_cast<uintptr_t>(src) + (uintptr_t)rows * cols * 2};
}

int launch_pads(const PadParams& p, cudaStream_t s) {
  if (p.count == 0) return MOE_OK;
  long n = 0;
  for (int i = 0; i < p.count; ++i) n = std::max(n, p.m[i].n);
  const int grid = (int)std::max(1L, std::min((n + 255) / 256, (long)num_sms() * 16));
  ProfScope ps("grouped_pad_rows", s);
  const cudaError_t e = launch_pdl(pad_rows_kernel, grid, 256, 0, s, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "grouped_pad_rows: %s", cudaGetErrorString(e));
  return check_launch("grouped_pad_rows");
}

// ---- float32 operands in parts ---------------------------------------------------------

struct Split {
  const float* src;
  uint4* dst;           // [3 parts, rows, padded columns] bf16
  long n;               // pieces of 8 columns of one part
  int cols, pieces;     // columns; pieces of a row
  int per;              // rows of an expert's matrix (0: not by expert)
};

struct SplitParams {
  const int32_t* offsets;
  int E, S;
  Split m[3];
  int count;
  int* flags;           // grouped::kFlagWords, one per block and zeros
};

__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// 2^16 x = h + m + l, each rounded to nearest from what is left. Bound by memory: 4 bytes in, 6 out. Rows that no group
// owns stay out: they may never have been written, and what they hold must not choose the kernel.
__global__ void __launch_bounds__(256) split_kernel(const SplitParams P) {
  __shared__ Live live;
  pdl_wait();
  pdl_trigger();
  live_list(P.offsets, P.E, P.S, live);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k >= P.count) break;
    const Split M = P.m[k];
    const long n = live_pieces(M.pieces, M.per, live);
    for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long)gridDim.x * blockDim.x) {
      int piece;
      const long r = piece_row(i, M.pieces, M.per, live, piece);
      const int c = piece * 8;
      const float* p = M.src + r * M.cols + c;
      float v[8];
      if ((M.cols & 3) == 0 && c + 8 <= M.cols) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < M.cols ? __ldg(p + j) : 0.0f;
      }
      uint32_t q[3][4] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        bad |= (__float_as_uint(v[j]) & 0x7fffffffu) >= 0x55800000u;     // 2^44 and above, infinity, NaN
        float left = v[j] * kPartScale;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint32_t bits = bf16_bits(left);
          q[part][j >> 1] |= bits << (16 * (j & 1));
          left -= __uint_as_float(bits << 16);       // exact
        }
      }
#pragma unroll
      for (int part = 0; part < 3; ++part)
        M.dst[part * M.n + r * M.pieces + piece] = make_uint4(q[part][0], q[part][1], q[part][2], q[part][3]);
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) P.flags[blockIdx.x] = any;
  if (blockIdx.x == 0)
    for (int i = gridDim.x + threadIdx.x; i < grouped::kFlagWords; i += blockDim.x) P.flags[i] = 0;
}

void add_split(SplitParams& p, const void* src, long rows, int cols, int per, Carver& c, Mat* m) {
  const int pc = pad8(cols);
  uint16_t* dst = c.take<uint16_t>((size_t)3 * rows * pc);
  *m = Mat{dst, pc};
  p.m[p.count++] = Split{static_cast<const float*>(src), reinterpret_cast<uint4*>(dst), rows * (pc / 8), cols, pc / 8, per};
}

int launch_split(SplitParams& p, Params* out, cudaStream_t s) {
  long n = 0;
  for (int i = 0; i < p.count; ++i) n = std::max(n, p.m[i].n);
  const int grid = (int)std::max(1L, std::min((n + 255) / 256, (long)grouped::kFlagWords));
  out->flags = p.flags;
  ProfScope ps("grouped_split", s);
  const cudaError_t e = launch_pdl(split_kernel, grid, 256, 0, s, p);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "grouped_split: %s", cudaGetErrorString(e));
  return check_launch("grouped_split");
}

size_t split_bytes(Carver& c, long rows, int cols) {
  c.take<uint16_t>((size_t)3 * rows * pad8(cols));
  return c.used;
}

}  // namespace

size_t grouped_tc_workspace(int dtype, int S, int K, int N, int E, bool fwd) {
  Carver c(nullptr);
  if (dtype == MOE_F32) {
    if (!grouped_f32_uses_tensor_cores(S, K, N, E, !fwd)) return grouped_simt_workspace(S, K, N, E, fwd);
    c.take<int>(grouped::kFlagWords);
    split_bytes(c, S, K);
    split_bytes(c, (long)E * N, K);
    if (!fwd) split_bytes(c, S, N);
    return align_up(c.used, 256);
  }
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
  Params p{a.offsets, a.S, a.E, job(a.dtype, a.K, a.N, a.y, 0, 0), Job{}, 0, nullptr, a.status, wait_limit_ns()};
  const bool f32 = a.dtype == MOE_F32;
  if (f32) {
    SplitParams q{};
    q.offsets = a.offsets;
    q.E = a.E;
    q.S = a.S;
    q.flags = c.take<int>(grouped::kFlagWords);
    add_split(q, a.x, a.S, a.K, 0, c, &x);
    add_split(q, a.w, (long)a.E * a.N, a.K, a.N, c, &w);
    if ((rc = launch_split(q, &p, s))) return rc;
  } else {
    PadParams q{a.offsets, a.E, a.S, {}, 0};
    padded(q, a.x, a.S, a.K, 0, c, &x);
    padded(q, a.w, (long)a.E * a.N, a.K, a.N, c, &w);
    if ((rc = launch_pads(q, s))) return rc;
    if (grouped_few_rows(a.S, a.E)) return launch_grouped_few(a, x.p, w.p, x.cols, s);
  }
  const uint64_t parts = f32 ? 3 : 1;
  CUtensorMap m[4];
  if ((rc = make_tmap_3d(&m[0], x.p, 2, (uint64_t)x.cols, (uint64_t)a.S, parts, BK, BM))) return rc;
  if ((rc = make_tmap_3d(&m[1], w.p, 2, (uint64_t)w.cols, (uint64_t)a.N, parts * (uint64_t)a.E, BK, BN / 2))) return rc;
  m[2] = m[3] = m[0];      // not read
  const long tiles = row_tiles(a, p.rows.NT);
  if (f32) {
    if ((rc = launch<false, float>(m, a, p, tiles, s, "grouped_gemm"))) return rc;
    return launch_grouped_simt(a, p.flags, s);
  }
  return a.dtype == MOE_BF16 ? launch<false, __nv_bfloat16>(m, a, p, tiles, s, "grouped_gemm")
                             : launch<false, __half>(m, a, p, tiles, s, "grouped_gemm");
}

int launch_grouped_tc_backward(const GroupedArgs& a, cudaStream_t s) {
  Carver c(a.ws);
  Mat dy{}, x{}, w{};
  CUtensorMap m[4] = {};
  int rc;
  Params p{a.offsets, a.S, a.E, Job{}, Job{}, 0, nullptr, a.status, wait_limit_ns()};
  const bool f32 = a.dtype == MOE_F32;
  const uint64_t parts = f32 ? 3 : 1;
  if (f32) {
    SplitParams q{};
    q.offsets = a.offsets;
    q.E = a.E;
    q.S = a.S;
    q.flags = c.take<int>(grouped::kFlagWords);
    add_split(q, a.d_y, a.S, a.N, 0, c, &dy);
    if (a.d_w) add_split(q, a.x, a.S, a.K, 0, c, &x);
    if (a.d_x) add_split(q, a.w, (long)a.E * a.N, a.K, a.N, c, &w);
    if ((rc = launch_split(q, &p, s))) return rc;
  } else {
    PadParams q{a.offsets, a.E, a.S, {}, 0};
    padded(q, a.d_y, a.S, a.N, 0, c, &dy);
    if (a.d_x) padded(q, a.w, (long)a.E * a.N, a.K, a.N, c, &w);
    if (a.d_w) padded(q, a.x, a.S, a.K, 0, c, &x);
    if ((rc = launch_pads(q, s))) return rc;
  }
  long tiles = 0;
  if (a.d_x) {
    if ((rc = make_tmap_3d(&m[0], dy.p, 2, (uint64_t)dy.cols, (uint64_t)a.S, parts, BK, BM))) return rc;
    if ((rc = make_tmap_3d(&m[1], w.p, 2, (uint64_t)w.cols, (uint64_t)a.N, parts * (uint64_t)a.E, 64, BK))) return rc;
    p.rows = job(a.dtype, a.N, a.K, a.d_x, 0, 1);
    tiles += row_tiles(a, p.rows.NT);
  }
  if (a.d_w) {
    if ((rc = make_tmap_3d(&m[2], dy.p, 2, (uint64_t)dy.cols, (uint64_t)a.S, parts, 64, BK))) return rc;
    if ((rc = make_tmap_3d(&m[3], x.p, 2, (uint64_t)x.cols, (uint64_t)a.S, parts, 64, BK))) return rc;
    p.dw = job(a.dtype, 0, a.K, a.d_w, 1, 1);
    p.dw.M = a.N;
    p.dw.MT = (a.N + 2 * BM - 1) / (2 * BM);
    tiles += (long)a.E * p.dw.MT * p.dw.NT;
  }
  if (!a.d_x) m[0] = m[1] = m[2];      // not read
  if (!a.d_w) m[2] = m[3] = m[0];
  p.dw_first = a.S / a.E > a.N;
  const char* name = "grouped_gemm_backward";
  if (f32) {
    if ((rc = launch<true, float>(m, a, p, tiles, s, name))) return rc;
    if (a.d_x && (rc = launch_grouped_simt_dx(a, p.flags, s))) return rc;
    return a.d_w ? launch_grouped_simt_dw(a, p.flags, s) : MOE_OK;
  }
  return a.dtype == MOE_BF16 ? launch<true, __nv_bfloat16>(m, a, p, tiles, s, name)
                             : launch<true, __half>(m, a, p, tiles, s, name);
}

}  // namespace moe
