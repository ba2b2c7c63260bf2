// Rows grouped by expert: what the kernels over caller-given group offsets share.
//
// offsets [E + 1] (device) says that expert e owns rows offsets[e] .. offsets[e + 1] - 1
// of a matrix of S rows. The values come from the caller and are read on the device
// only, so every kernel clamps them: a group is cut to [0, S) and one that ends before
// it starts is empty. All indexing then stays in bounds whatever the words hold.
#pragma once
#include "common.cuh"

namespace moe {
namespace grouped {

struct Span {
  int lo, hi;
  __device__ __forceinline__ int rows() const { return hi - lo; }
};

__device__ __forceinline__ Span span(const int32_t* offsets, int e, int S) {
  const int lo = min(max(__ldg(offsets + e), 0), S);
  return Span{lo, max(lo, min(__ldg(offsets + e + 1), S))};
}

// Whole warp: start[e] = sum over e' < e of tiles(rows of e'), start[E] = the total.
// Also reports (bad != null) whether the offsets are not an ascending list in [0, S].
template <class Tiles>
__device__ __forceinline__ void tile_list(const int32_t* offsets, int E, int S, Tiles tiles, int* start, int* bad) {
  const int lane = threadIdx.x & 31;
  const int per = (E + 31) / 32;
  const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
  int run = 0, wrong = 0;
  for (int e = e0; e < e1; ++e) {
    const int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
    wrong |= a < 0 || b < a || b > S;
    run += tiles(span(offsets, e, S).rows());
  }
  int incl = run;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  int acc = incl - run;
  for (int e = e0; e < e1; ++e) {
    start[e] = acc;
    acc += tiles(span(offsets, e, S).rows());
  }
  if (lane == 31) start[E] = incl;
  wrong = __any_sync(0xffffffffu, wrong);
  if (bad != nullptr && lane == 0) *bad = wrong;
}

// The expert whose tiles hold t: start[e] <= t < start[e + 1].
__device__ __forceinline__ int find(const int* start, int E, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Rows that no group owns (before offsets[0], from offsets[E] on) are zero in row
// outputs. Thread `i` of `n` writes its share of them.
template <class T>
__device__ __forceinline__ void zero_unowned(T* out, const int32_t* offsets, int E, int S, long cols, long i, long n) {
  const int first = min(max(__ldg(offsets), 0), S);
  const int last = max(first, min(__ldg(offsets + E), S));
  for (long j = i; j < (long)first * cols; j += n) out[j] = from_float<T>(0.0f);
  for (long j = (long)last * cols + i; j < (long)S * cols; j += n) out[j] = from_float<T>(0.0f);
}

// Two values of a 16-bit type in one word.
template <class T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// How rows of `cols` values are stored: 2 = 32-byte sectors, 1 = 16 bytes, 0 = single values.
inline int store_width(const void* out, long cols, int bytes) {
  if (cols * bytes % 32 == 0 && aligned(out, 32)) return 2;
  return cols * bytes % 16 == 0 && aligned(out, 16) ? 1 : 0;
}

// W (16 or 32) columns of one row from column c on (of `cols`): float32 sums (as bits), rounded once.
template <class T, int W>
__device__ __forceinline__ void store_cols(T* row, int c, int cols, int vec, const uint32_t (&y)[W]) {
  if (vec > 0 && c + W <= cols) {
    constexpr int Q = W * (int)sizeof(T) / 4;
    uint32_t q[Q];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < Q; ++i) q[i] = y[i];
    } else {
#pragma unroll
      for (int i = 0; i < Q; ++i) q[i] = pack_pair<T>(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
    }
    uint32_t* p = reinterpret_cast<uint32_t*>(row + c);
    if (vec == 2) {
#pragma unroll
      for (int i = 0; i < Q / 8; ++i) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = q[8 * i + j];
        st_v8(p + 8 * i, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < Q / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (c + i < cols) row[c + i] = from_float<T>(__uint_as_float(y[i]));
  }
}

}  // namespace grouped
}  // namespace moe
