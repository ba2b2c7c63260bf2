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

}  // namespace grouped
}  // namespace moe
