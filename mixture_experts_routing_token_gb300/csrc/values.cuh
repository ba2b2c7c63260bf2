// Eight or sixteen neighbouring values of a row between memory and float32 registers.
#pragma once
#include "grouped.cuh"

namespace moe {

// 16 bytes of memory that the kernel may write as well (SAME), or that nobody writes while it runs (the read-only path).
template <bool SAME, class V>
__device__ __forceinline__ V load16b(const V* p) {
  if constexpr (SAME) return *p;
  else return __ldg(p);
}

template <bool SAME = false>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = load16b<SAME>(reinterpret_cast<const float4*>(p)), b = load16b<SAME>(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <bool SAME = false>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = load16b<SAME>(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <bool SAME = false>
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 q = load16b<SAME>(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// 16 values of one row as whole 32-byte sectors (or 16-byte halves where the output is not so aligned).
template <class T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16], bool sectors) {
  constexpr int Q = 4 * (int)sizeof(T);     // words
  uint32_t q[Q];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < Q; ++j) q[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < Q; ++j) q[j] = grouped::pack_pair<T>(v[2 * j], v[2 * j + 1]);
  }
  uint32_t* d = reinterpret_cast<uint32_t*>(p);
#pragma unroll
  for (int j = 0; j < Q / 8; ++j) {
    if (sectors) {
      uint32_t w[8];
#pragma unroll
      for (int l = 0; l < 8; ++l) w[l] = q[8 * j + l];
      st_v8(d + 8 * j, w);
    } else {
      reinterpret_cast<uint4*>(d)[2 * j] = make_uint4(q[8 * j], q[8 * j + 1], q[8 * j + 2], q[8 * j + 3]);
      reinterpret_cast<uint4*>(d)[2 * j + 1] = make_uint4(q[8 * j + 4], q[8 * j + 5], q[8 * j + 6], q[8 * j + 7]);
    }
  }
}

// Eight values of one row, rounded to T: 16 bytes, or one 32-byte sector.
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(grouped::pack_pair<T>(v[0], v[1]), grouped::pack_pair<T>(v[2], v[3]),
                                              grouped::pack_pair<T>(v[4], v[5]), grouped::pack_pair<T>(v[6], v[7]));
  }
}

}  // namespace moe
