// Rows grouped by expert: what the kernels over caller-given group offsets share.
//
// offsets [E + 1] (device) says that expert e owns rows offsets[e] .. offsets[e + 1] - 1
// of a matrix of S rows. The values come from the caller and are read on the device
// only, so every kernel first makes them an ascending list in [0, S] (each entry cut to
// [0, S] and raised to the largest before it). Groups are then disjoint and all indexing
// stays in bounds, whatever the words hold.
#pragma once
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace grouped {

struct Span {
  int lo, hi;
  __device__ __forceinline__ int rows() const { return hi - lo; }
};

// In shared memory.
struct Groups {
  int off[MOE_MAX_EXPERTS + 1];     // the ascending offsets
  int start[MOE_MAX_EXPERTS + 1];   // tiles of the experts before e; start[E]: all tiles
  int bad;                          // the caller's offsets were not an ascending list in [0, S]

  __device__ __forceinline__ Span span(int e) const { return Span{off[e], off[e + 1]}; }
};

// Whole warp: fills G; tiles(rows) is the tile count of a group. A lane takes four neighbouring
// entries, so up to 127 experts are one load latency and two scans, which every kernel here waits
// for before its first tile. Returns (in every lane) the rows of the largest group.
template <class Tiles>
__device__ __forceinline__ int group_list(const int32_t* offsets, int E, int S, Tiles tiles, Groups& G) {
  const int lane = threadIdx.x & 31;
  int top = 0, last = 0, wrong = 0, sum = 0, most = 0;    // over all entries before this turn
  for (int i0 = 0; i0 <= E; i0 += 128) {
    const int i = i0 + 4 * lane;
    int v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i + u <= E ? __ldg(offsets + i + u) : 0;
    int raw = __shfl_up_sync(0xffffffffu, v[3], 1);
    if (lane == 0) raw = last;
    last = __shfl_sync(0xffffffffu, v[3], 31);
    int up = 0;                                       // largest of the lane's entries, then of all up to it
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i + u > E) continue;
      wrong |= v[u] < 0 || v[u] > S || (i + u > 0 && v[u] < raw);
      raw = v[u];
      up = max(up, min(max(v[u], 0), S));
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) up = max(up, __shfl_up_sync(0xffffffffu, up, d));
    int before = __shfl_up_sync(0xffffffffu, up, 1);  // offset of the entry before the lane's
    before = max(top, lane == 0 ? 0 : before);
    top = max(top, __shfl_sync(0xffffffffu, up, 31));
    int off[4], count[4], total = 0;                  // count[u]: tiles of the lane's groups up to entry u
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      off[u] = max(before, i + u <= E ? min(max(v[u], 0), S) : 0);
      if (i + u > 0 && i + u <= E) {                  // the group that ends here; one without rows may have tiles
        most = max(most, off[u] - before);
        total += tiles(off[u] - before);
      }
      count[u] = total;
      before = off[u];
    }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u <= E) {
        G.off[i + u] = off[u];
        G.start[i + u] = sum + incl - total + count[u];      // the tiles of groups 0 .. i + u - 1
      }
    sum += __shfl_sync(0xffffffffu, incl, 31);
  }
  wrong = __any_sync(0xffffffffu, wrong);
  if (lane == 0) G.bad = wrong;
#pragma unroll
  for (int d = 16; d; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
  return most;
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

// The same for a t that grows from call to call; `e` is the last answer (0 at first).
__device__ __forceinline__ int find_from(const int* start, int e, int t) {
  while (start[e + 1] <= t) ++e;
  return e;
}

// n / d for n >= 0, d > 0. The float32 quotient of (n + 1/2) is off by less than 2^-22 of itself, the
// true one at least 1/(2 d) from the next integer, so below 2^21 its whole part is exact; a tenth of
// the integer division's cycles, which the roles would wait for at every tile.
__device__ __forceinline__ int quick_div(int n, int d) {
  return n < (1 << 21) ? (int)__fdividef((float)n + 0.5f, (float)d) : n / d;
}

// Rows that no group owns (before the first offset, from the last one on) are zero in row
// outputs. Thread `i` of `n` writes its share of them.
template <class T>
__device__ __forceinline__ void zero_unowned(T* out, const Groups& G, int E, int S, long cols, long i, long n) {
  for (long j = i; j < (long)G.off[0] * cols; j += n) out[j] = from_float<T>(0.0f);
  for (long j = (long)G.off[E] * cols + i; j < (long)S * cols; j += n) out[j] = from_float<T>(0.0f);
}

// float32 products in parts: one word per block of the kernel that makes the parts, not 0 where it
// met a value that parts do not stand for (kFlagWords in all). Thread `i` of `n` looks at its share,
// all loads under way together.
constexpr int kFlagWords = 1024;
template <int N>
__device__ __forceinline__ int any_flag(const int* flags, int i) {
  int any = 0;
#pragma unroll
  for (int j = 0; j < kFlagWords / 4 / N; ++j) {
    const int4 q = __ldg(reinterpret_cast<const int4*>(flags) + i + j * N);
    any |= q.x | q.y | q.z | q.w;
  }
  return any;
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

// 32 columns of a warp's 32 rows (row l's in lane l's y) where rows are not a multiple of 16 bytes:
// the lanes exchange the block's transpose (five rounds of shuffles), then each store instruction
// writes neighbouring columns of one row. Lanes storing their own rows value by value touched 32
// lines with every instruction.
template <class T>
__device__ __forceinline__ void store_turned(uint32_t (&y)[32], T* row0, int count, int c, int cols) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 16; s; s >>= 1) {
    const bool hi = lane & s;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j & s) continue;
      const uint32_t give = hi ? y[j] : y[j + s];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, give, s);
      if (hi) y[j] = got; else y[j + s] = got;
    }
  }
  if (c + lane < cols) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < count) row0[(long)j * cols + c + lane] = from_float<T>(__uint_as_float(y[j]));
  }
}

// Rows of an accumulator, one per lane, to the output through 4 KB of shared memory of the warp's
// own (1024-byte aligned): `q` holds 64 packed 16-bit columns. A box of 32 whole rows goes out as one
// TMA store of tensor `m` at (x, y, z), which runs on while the warp reads its next columns; rows that
// end before (count < 32, the next group follows) are read back and stored with ordinary
// instructions, four rows of 128 bytes each. Measured at K = 128, where the epilogue sets the pace,
// float16 output of 270 MB: 65 us, with ordinary stores alone 93. Needs rows that are a multiple of
// 16 bytes, 16-byte aligned. The 16-byte pieces lie in the order of the tensor's 128-byte swizzle,
// with which neither side meets bank conflicts.
template <class T>
__device__ __forceinline__ void store_rows(uint32_t buf, const uint32_t (&q)[32], const CUtensorMap* m, int x, int y, int z,
                                           bool whole, T* row0, int count, int cols) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) ptx::tma_store_wait_read();      // the last box has left the buffer
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 8; ++p)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((p ^ (lane & 7)) << 4)),
                 "r"(q[4 * p]), "r"(q[4 * p + 1]), "r"(q[4 * p + 2]), "r"(q[4 * p + 3])
                 : "memory");
  if (whole) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) ptx::tma_store_3d(m, buf, x, y, z);
    return;
  }
  __syncwarp();
  const int p = lane & 7, col = x + p * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(buf + r * 128 + ((p ^ (r & 7)) << 4))
                 : "memory");
    // cols is a multiple of 8: whole pieces
    if (col < cols && r < count) *reinterpret_cast<uint4*>(row0 + (long)r * cols + col) = v;
  }
  __syncwarp();
}

// The same for rows that are not a multiple of 16 bytes, which start anywhere between two pieces of memory: eight lanes take
// a row and store its whole pieces, each out of the two in the buffer that hold its values, shifted in registers; the up to
// seven values before the first and behind the last of them leave in words and single values, a row a lane. 16000
// float16 rows, K = 136, 4093 columns: 80 us; 109 where a whole warp read a row back and stored it in words of 4 bytes, 139
// where the lanes exchanged the block by shuffles and stored single values. 22676 8-bit rows, K = 128, 8121 bf16 columns:
// 177 us, with words 238 (39 instructions a row and 64 columns, of which the epilogue's warps are short).
// `count` > 0 rows, columns from c0 on.
template <class T>
__device__ __forceinline__ void store_ragged(uint32_t buf, const uint32_t (&q)[32], T* row0, int count, int c0, int cols) {
  const int lane = threadIdx.x & 31, p = lane & 7;
  __syncwarp();                                   // the last columns have been read
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((i ^ (lane & 7)) << 4)),
                 "r"(q[4 * i]), "r"(q[4 * i + 1]), "r"(q[4 * i + 2]), "r"(q[4 * i + 3])
                 : "memory");
  __syncwarp();
  const int left = min(64, cols - c0);            // values of a row
  uint16_t* const first = reinterpret_cast<uint16_t*>(row0) + c0;
  auto before = [](const uint16_t* row) { return (int)(reinterpret_cast<uintptr_t>(row) >> 1) & 7; };
#pragma unroll 2
  for (int r0 = 0; r0 < 32; r0 += 4) {
    if (r0 >= count) break;
    const int r = r0 + (lane >> 3);
    uint16_t* row = first + (long)r * cols;
    const int d = before(row), x = 8 * p - d;     // the values x .. x + 7, of the pieces p - 1 and p
    uint32_t w[8];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(buf + r * 128 + ((((p - 1) & 7) ^ (r & 7)) << 4))
                 : "memory");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "r"(buf + r * 128 + ((p ^ (r & 7)) << 4))
                 : "memory");
    const uint32_t shift = 16 - 2 * d;            // bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = shift & 16 ? w[i + 4] : w[i];
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
    if (r < count && x >= 0 && x + 8 <= left) *reinterpret_cast<uint4*>(row + x) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane < count) {
    uint16_t* row = first + (long)lane * cols;
    const int d = before(row);
    const int head = min((8 - d) & 7, left);                   // values before the first whole piece
    const int tail = max(head, ((left + d) & ~7) - d);         // the first one behind the last
    auto value = [&](int v) {
      uint32_t b;
      asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                   : "=r"(b)
                   : "r"(buf + lane * 128 + (((v >> 3) ^ (lane & 7)) << 4) + (v & 7) * 2)
                   : "memory");
      return b;
    };
    auto some = [&](int v, int end) {                          // up to seven of them
      if (v < end && (reinterpret_cast<uintptr_t>(row + v) & 2)) {
        row[v] = (uint16_t)value(v);
        ++v;
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (v + 1 < end) {
          *reinterpret_cast<uint32_t*>(row + v) = value(v) | value(v + 1) << 16;
          v += 2;
        }
      if (v < end) row[v] = (uint16_t)value(v);
    };
    some(0, head);
    some(tail, left);
  }
}

// Whole warp: n >= 0 neighbouring values to zero, 16 bytes a lane between the first and the last boundary.
template <class T>
__device__ __forceinline__ void zero_values(T* p, int n) {
  const int lane = threadIdx.x & 31;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), e = a + (uintptr_t)n * sizeof(T);
  const uintptr_t first = min((a + 15) & ~(uintptr_t)15, e), last = max(first, e & ~(uintptr_t)15);
  for (uintptr_t u = first + lane * 16; u < last; u += 512) *reinterpret_cast<uint4*>(u) = make_uint4(0, 0, 0, 0);
  const uintptr_t head = a + lane * sizeof(T), tail = last + lane * sizeof(T);      // under 16 bytes each
  if (head < first) *reinterpret_cast<T*>(head) = from_float<T>(0.0f);
  if (tail < e) *reinterpret_cast<T*>(tail) = from_float<T>(0.0f);
}

// W float32 sums (as bits) as words of T.
template <class T, int W>
__device__ __forceinline__ void pack_words(const uint32_t (&y)[W], uint32_t* q) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = y[i];
  } else {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) q[i] = pack_pair<T>(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
  }
}

}  // namespace grouped
}  // namespace moe
