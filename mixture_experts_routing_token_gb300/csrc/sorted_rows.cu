// Gradients of sorting rows by expert and of the weighted sum that brings them back, and both forward steps for
// the types and widths that the layer's own kernels do not take (float16, rows that are not a multiple of 16 bytes).
//
// pos(s) is the sorted row of slot s = t k + j (the inverse of reverse_indices over the rows p < offsets[E]); slots
// that the align step dropped have none.
//   copy      x[pos(s)] = hidden[t]                 d_hidden[t] = sum_j d_x[pos(t k + j)]
//   sum       out[t] = sum_j w[t, j] y[pos(t k + j)]
//             d_y[pos(s)] = w[t, j] d_out[t],       d_w[t, j] = <d_out[t], y[pos(s)]>
// All in token order: a CTA takes neighbouring tokens, so that d_out and every sorted row move once (in sorted order
// d_out would be read k times over). Sums in float32, j ascending, one rounding; a slot without a row adds nothing.
// Bound by memory.
//
// The inverse comes from a first kernel (a word per slot in the workspace), which writes the slots that have a row and
// leaves the others as they were: a reader takes an entry p only if p is a routed row and reverse[p] is the slot, so
// that whatever else the buffer holds, no index leaves the arrays and no slot takes another one's row. With few slots each
// CTA of the one launch looks through reverse_indices itself instead.
#include <algorithm>
#include <type_traits>

#include "values.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Loads of sorted rows that a thread has under way: of 2, 4 or 8 slots (K), the least that are k or more. Measured, us, both
// gradients with 8 / 4 / 2 slots at a time, bf16 rows of 2048: k = 8, 8192 tokens 158 / 160 / 162 (500 tokens of 512 values
// 10.8 / 11.7 / 14.0), k = 4, 16384 tokens 185 / 153 / 161, k = 3, 8192 tokens 89 / 72 / 77 (before every slot's entry was
// looked up in reverse_indices again, which made 157, 158 and 74 of 155, 155 and 73).
constexpr int kFlight = 8;
// Whether the CTAs look for their slots themselves. Measured, us, both gradients of bf16 rows of 512, from Python / in a
// graph, with the first kernel and its workspace, and without: 4000 slots of 500 tokens 26.5 / 11.7 and 13.5 / 10.7, 8000
// slots of 1000 tokens 27.5 / 12.4 and 14.3 / 14.8, of 8000 tokens 27.2 / 22.2 and 30.5 / 31.2. At the rule's upper end,
// with / without: 8 slots of 1025 / 1024 tokens 26 / 12.3 and 16 / 15.4, 4 of 2049 / 2048 25 / 15.3 and 21 / 20.3, 1 of 2049 /
// 2048 25 / 11.7 and 13 / 10.3: chosen for calls from Python; in a graph the first kernel is the faster one there.
bool each_looks(int T, int k) { return (long)T * k <= 2048 || ((long)T * k <= 8192 && T <= 2048); }
// Rows in windows: two slots at a time, a piece each, in registers for four CTAs an SM. Measured, us, 8192 tokens x 8 of 2047
// bf16 values, combine backward / gather backward: 151 / 83; with five CTAs 222 / 93, four slots and three CTAs 167 / 90,
// as many registers as it likes 202 / 109; single values instead of windows 244 / 199. At 2046 values 148 / 82, in words of 4
// bytes together 259.
constexpr int kCtas = 4;
constexpr int kMinGroup = 4;            // threads of a token at least
constexpr int kSlotsPerCta = kThreads / kMinGroup * MOE_MAX_TOPK;

// 16 bytes of neighbouring values as they lie in memory.
template <class T>
struct Piece {
  static constexpr int V = 16 / (int)sizeof(T);
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void values(float (&v)[V]) const {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(q[i]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(q + i));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(q[i] << 16);
        v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else store8(p, v);
  }
};

// Rows that are not a multiple of 16 bytes start anywhere between two pieces of memory, each at a place of its own. The row
// that is written sets the pieces: the first may begin up to V - 1 values before the row, the last end after it. A row
// that is read is shifted against them and comes as the two pieces that hold the values (the second one is the next
// thread's first and comes out of L1).
template <class T>
__device__ __forceinline__ int values_before(const T* row) { return (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T); }

// A piece of the array from `first` (which is at the start of one) to `last`; zeros outside.
template <class T>
__device__ __forceinline__ Piece<T> piece_inside(const T* p, const T* first, const T* last) {
  constexpr int V = Piece<T>::V;
  Piece<T> r;
  if (p >= first && p + V <= last) {
    r.load(p);
  } else {
    __align__(16) T v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p >= first && p + i < last ? p[i] : from_float<T>(0.0f);
    r.w = *reinterpret_cast<const uint4*>(v);
  }
  return r;
}

template <class T>
struct Window {
  Piece<T> lo, hi;
  uint32_t shift;          // bytes
  __device__ __forceinline__ void load(const T* p, const T* first, const T* last) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    shift = (uint32_t)(at & 15);
    const T* q = reinterpret_cast<const T*>(at - shift);
    lo = piece_inside(q, first, last);
    if (shift) hi = piece_inside(q + Piece<T>::V, first, last);
  }
  __device__ __forceinline__ Piece<T> get() const {
    uint32_t w[8] = {lo.w.x, lo.w.y, lo.w.z, lo.w.w, hi.w.x, hi.w.y, hi.w.z, hi.w.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
    }
    Piece<T> r;
    r.w = make_uint4(w[0], w[1], w[2], w[3]);
    return r;
  }
};

// Values i .. i + V - 1 of a row of H, those that there are.
template <class T>
__device__ __forceinline__ void store_inside(T* row, int i, int H, const float (&v)[Piece<T>::V]) {
  constexpr int V = Piece<T>::V;
  if (i >= 0 && i + V <= H) {
    Piece<T>::store(row + i, v);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (i + q >= 0 && i + q < H) row[i + q] = from_float<T>(v[q]);
  }
}

struct Args {
  const int32_t* reverse;
  const int32_t* offsets;
  int32_t* pos;         // null: the CTA looks through reverse
  int T, k, E;
  int H;
  const float* weights; // [T, k], or null: 1
  int32_t* status;
};

__device__ __forceinline__ int routed(const Args& a) { return min(max(__ldg(a.offsets + a.E), 0), a.T * a.k); }

__global__ void __launch_bounds__(kThreads) slot_positions_kernel(const Args a) {
  pdl_wait();
  pdl_trigger();
  const int S = a.T * a.k, n = routed(a);
  for (long p = (long)blockIdx.x * kThreads + threadIdx.x; p < n; p += (long)gridDim.x * kThreads) {
    const int s = __ldg(a.reverse + p);
    if (s >= 0 && s < S) a.pos[s] = (int)p;
  }
}

// The sorted rows of the CTA's slots [s0, s0 + count) to shared memory, -1 where there is none; reports what is wrong
// with the routing.
__device__ __forceinline__ void take_positions(const Args& a, int s0, int count, int* pos) {
  const int S = a.T * a.k, n = routed(a);
  if (a.pos == nullptr) {
    for (int i = threadIdx.x; i < count; i += kThreads) pos[i] = -1;
    __syncthreads();
    for (int p0 = threadIdx.x; p0 < n; p0 += 8 * kThreads) {
      int s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = p0 + i * kThreads < n ? __ldg(a.reverse + p0 + i * kThreads) : -1;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s[i] >= s0 && s[i] - s0 < count) pos[s[i] - s0] = p0 + i * kThreads;
    }
  } else {
    for (int i = threadIdx.x; i < count; i += kThreads) {
      int p = __ldcg(a.pos + s0 + i);
      if (p < 0 || p >= n || __ldg(a.reverse + p) != s0 + i) p = -1;
      pos[i] = p;
    }
  }
  if (a.status != nullptr) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(a.offsets + a.E) != n) atomicOr(a.status, MOE_STATUS_BAD_INDEX);
    for (long p = (long)blockIdx.x * kThreads + threadIdx.x; p < n; p += (long)gridDim.x * kThreads) {
      const int s = __ldg(a.reverse + p);
      if (s < 0 || s >= S) atomicOr(a.status, MOE_STATUS_BAD_INDEX);
    }
  }
  __syncthreads();
}

// out[t] = sum_j w[t, j] src[pos(t, j)]. G threads take a token, K of its slots and kFlight / K pieces at a time.
// WHOLE: rows are a multiple of 16 bytes and begin at one.
template <class T, bool WHOLE, int K>
__global__ void __launch_bounds__(kThreads, WHOLE ? 0 : kCtas)
    sum_rows_kernel(const Args a, const T* __restrict__ src, T* __restrict__ out, int G) {
  constexpr int V = Piece<T>::V, U = WHOLE ? kFlight / K : 1;
  __shared__ int pos[kSlotsPerCta];
  pdl_wait();
  pdl_trigger();
  const int tokens = kThreads / G, t0 = blockIdx.x * tokens;
  take_positions(a, t0 * a.k, min(tokens, a.T - t0) * a.k, pos);
  const int local = threadIdx.x / G, t = t0 + local;
  if (t >= a.T) return;
  const int* at = pos + local * a.k;
  const float* w = a.weights ? a.weights + (long)t * a.k : nullptr;
  T* row = out + (long)t * a.H;
  const int before = WHOLE ? 0 : values_before(row);
  const int pieces = (a.H + before + V - 1) / V;
  for (int c0 = threadIdx.x % G; c0 < pieces; c0 += U * G) {
    float sum[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < V; ++q) sum[u][q] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += K) {
      std::conditional_t<WHOLE, Piece<T>, Window<T>> y[K][U];
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j0 + j < a.k && at[j0 + j] >= 0 && c0 + u * G < pieces) {
            const T* p = src + (long)at[j0 + j] * a.H + (c0 + u * G) * V - before;
            if constexpr (WHOLE) y[j][u].load(p);
            else y[j][u].load(p, src, src + (long)a.T * a.k * a.H);
          }
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j0 + j < a.k && at[j0 + j] >= 0) {
          const float wj = w ? __ldg(w + j0 + j) : 1.0f;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[V];
            if constexpr (WHOLE) y[j][u].values(v);
            else y[j][u].get().values(v);
#pragma unroll
            for (int q = 0; q < V; ++q) sum[u][q] += wj * v[q];
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u * G >= pieces) continue;
      if constexpr (WHOLE) Piece<T>::store(row + (c0 + u * G) * V, sum[u]);
      else store_inside(row, (c0 + u * G) * V - before, a.H, sum[u]);
    }
  }
}

// d_y[pos(t, j)] = w[t, j] d_out[t] and d_w[t, j] = <d_out[t], y[pos(t, j)]>; either may be null.
// 16-bit rows with registers for three CTAs an SM: both gradients, us, as many registers as it likes / this: 8192 tokens x 8
// of 2048 values 159 / 156, 1200 x 8 of 2048 41 / 38, 1712 x 6 of 2224 48 / 43; float32 rows of 2304, 606 x 6, 29 / 34.
template <class T, bool WHOLE, int K>
__global__ void __launch_bounds__(kThreads, !WHOLE ? kCtas : sizeof(T) == 2 ? 3 : 0)
    sum_rows_backward_kernel(const Args a, const T* __restrict__ d_out, const T* __restrict__ y, T* __restrict__ d_y,
                             float* __restrict__ d_w, int G) {
  constexpr int V = Piece<T>::V, U = WHOLE ? kFlight / K : 1;
  __shared__ int pos[kSlotsPerCta];
  __shared__ float part[kThreads / 32][K];
  pdl_wait();
  pdl_trigger();
  const int tokens = kThreads / G, t0 = blockIdx.x * tokens;
  take_positions(a, t0 * a.k, min(tokens, a.T - t0) * a.k, pos);
  const int local = threadIdx.x / G, me = threadIdx.x % G, t = t0 + local;
  const bool in = t < a.T;
  const int* at = pos + (in ? local : 0) * a.k;
  const float* w = a.weights + (long)(in ? t : 0) * a.k;
  for (int j0 = 0; j0 < a.k; j0 += K) {
    float dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) dot[j] = 0.0f;
    if constexpr (WHOLE) {
      const int pieces = a.H / V;
      for (int c0 = me; in && c0 < pieces; c0 += U * G) {
        Piece<T> d[U], r[K][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c0 + u * G < pieces) d[u].load(d_out + (long)t * a.H + (c0 + u * G) * V);
        if (d_w != nullptr) {
#pragma unroll
          for (int j = 0; j < K; ++j)
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (j0 + j < a.k && at[j0 + j] >= 0 && c0 + u * G < pieces)
                r[j][u].load(y + (long)at[j0 + j] * a.H + (c0 + u * G) * V);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c0 + u * G >= pieces) continue;
          float dv[V];
          d[u].values(dv);
#pragma unroll
          for (int j = 0; j < K; ++j) {
            if (j0 + j >= a.k || at[j0 + j] < 0) continue;
            if (d_w != nullptr) {
              float v[V];
              r[j][u].values(v);
#pragma unroll
              for (int q = 0; q < V; ++q) dot[j] += dv[q] * v[q];
            }
            if (d_y != nullptr) {
              const float wj = __ldg(w + j0 + j);
              float o[V];
#pragma unroll
              for (int q = 0; q < V; ++q) o[q] = wj * dv[q];
              Piece<T>::store(d_y + (long)at[j0 + j] * a.H + (c0 + u * G) * V, o);
            }
          }
        }
      }
    } else {
      // the sorted row sets the pieces; d_out comes shifted to each, out of L1 after the first
      const T* const d_row = d_out + (long)(in ? t : 0) * a.H;
      const int pieces = (a.H - 1) / V + 2;      // of a row, wherever it lies
      for (int c = me; in && c < pieces; c += G) {
        Window<T> d[K];
        Piece<T> r[K];
        int x[K];              // first value, H: nothing to do
#pragma unroll
        for (int j = 0; j < K; ++j) {
          x[j] = a.H;
          if (j0 + j >= a.k || at[j0 + j] < 0) continue;
          const long row = (long)at[j0 + j] * a.H;
          const int i = c * V - (int)(row & (V - 1));
          if (i >= a.H) continue;
          x[j] = i;
          if (d_w != nullptr) r[j] = piece_inside(y + row + i, y, y + (long)a.T * a.k * a.H);
          d[j].load(d_row + i, d_out, d_out + (long)a.T * a.H);
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int i = x[j];
          if (i >= a.H) continue;
          float dv[V];
          d[j].get().values(dv);
          if (d_w != nullptr) {
            float v[V];
            r[j].values(v);
            if (i >= 0 && i + V <= a.H) {
#pragma unroll
              for (int q = 0; q < V; ++q) dot[j] += dv[q] * v[q];
            } else {           // what lies beside the row may be anything
#pragma unroll
              for (int q = 0; q < V; ++q)
                if (i + q >= 0 && i + q < a.H) dot[j] += dv[q] * v[q];
            }
          }
          if (d_y != nullptr) {
            const float wj = __ldg(w + j0 + j);
            float o[V];
#pragma unroll
            for (int q = 0; q < V; ++q) o[q] = wj * dv[q];
            store_inside(d_y + (long)at[j0 + j] * a.H, i, a.H, o);
          }
        }
      }
    }
    if (d_w == nullptr) continue;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      for (int s = min(G, 32) / 2; s; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
      if (G > 32 && lane == 0) part[warp][j] = dot[j];
    }
    if (G > 32) __syncthreads();
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (!in || me != j % G || j0 + j >= a.k) continue;
      float sum = dot[j];
      if (G > 32) {
        sum = 0.0f;
        for (int i = 0; i < G / 32; ++i) sum += part[warp + i][j];
      }
      d_w[(long)t * a.k + j0 + j] = sum;
    }
    if (G > 32) __syncthreads();
  }
}

// out[p] = src[ids[p]] for the routed rows, rows of any width (zeros where there is no such row). With registers for four
// CTAs an SM: 131072 of 16384 bf16 rows of 2047, us, as many registers as it likes / this: 157 / 142.
template <class T>
__global__ void __launch_bounds__(kThreads, kCtas)
    gather_any_rows_kernel(const T* __restrict__ src, const int32_t* __restrict__ ids, const int32_t* __restrict__ offsets, int E,
                           int rows, int S, int H, T* __restrict__ out) {
  constexpr int V = Piece<T>::V, U = 4;
  pdl_wait();
  pdl_trigger();
  const int n = min(max(__ldg(offsets + E), 0), S), lane = threadIdx.x & 31;
  for (long p = (long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; p < n; p += (long)gridDim.x * (kThreads / 32)) {
    const int t = __ldg(ids + p);
    T* to = out + p * H;
    if (t < 0 || t >= rows) {
      for (long i = lane; i < H; i += 32) to[i] = from_float<T>(0.0f);
      continue;
    }
    const T* from = src + (long)t * H;
    for (long i = lane * V - values_before(to); i < H; i += U * 32 * V) {
      Window<T> w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * 32 * V < H) w[u].load(from + i + u * 32 * V, src, src + (long)rows * H);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long x = i + u * 32 * V;
        if (x >= H) continue;
        __align__(16) T v[V];
        *reinterpret_cast<uint4*>(v) = w[u].get().w;
        if (x >= 0 && x + V <= H) {
          *reinterpret_cast<uint4*>(to + x) = *reinterpret_cast<const uint4*>(v);
        } else {
#pragma unroll
          for (int q = 0; q < V; ++q)
            if (x + q >= 0 && x + q < H) to[x + q] = v[q];
        }
      }
    }
  }
}

// ---- host -----------------------------------------------------------------------------------------

int done(cudaError_t e, const char* name) {
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

int positions(Args& a, cudaStream_t s) {
  const long S = (long)a.T * a.k;
  if (each_looks(a.T, a.k)) {
    a.pos = nullptr;
    return MOE_OK;
  }
  ProfScope ps("slot_positions", s);
  const int grid = (int)std::min((long)num_sms() * 4, (S + kThreads - 1) / kThreads);
  return done(launch_pdl(slot_positions_kernel, grid, kThreads, 0, s, a), "slot_positions");
}

// CTAs of `tokens` each (a power of two); T may be the largest int.
unsigned ctas(int T, int tokens) { return (unsigned)(((long)T + tokens - 1) / tokens); }

// Threads of a token, a power of two: no more than it has pieces, and no more than give every SM five CTAs.
int threads_per_token(int pieces, int T) {
  int g = kMinGroup;
  while (g < kThreads && g < pieces && (g < 32 || (long)T * g < 5L * kThreads * num_sms())) g *= 2;
  return g;
}

// Whether rows are whole pieces of 16 bytes (arrays start at one).
template <class T>
bool whole(const Args& a) { return a.H % Piece<T>::V == 0; }

// Pieces of a row at most.
template <class T, bool WHOLE>
int pieces_of(int H) { return WHOLE ? H / Piece<T>::V : (H - 1) / Piece<T>::V + 2; }

template <class T, bool WHOLE, int K>
int sum_as(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  const int G = threads_per_token(pieces_of<T, WHOLE>(a.H), a.T), tokens = kThreads / G;
  ProfScope ps(name, s);
  return done(launch_pdl(sum_rows_kernel<T, WHOLE, K>, ctas(a.T, tokens), kThreads, 0, s, a,
                         static_cast<const T*>(src), static_cast<T*>(out), G),
              name);
}
template <class T>
int sum(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  if (!whole<T>(a)) return sum_as<T, false, 2>(a, src, out, name, s);
  if (a.k <= 2) return sum_as<T, true, 2>(a, src, out, name, s);
  return a.k <= 4 ? sum_as<T, true, 4>(a, src, out, name, s) : sum_as<T, true, 8>(a, src, out, name, s);
}

template <class T, bool WHOLE, int K>
int sum_backward_as(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  const char* name = "ep_combine_backward";
  const int G = threads_per_token(pieces_of<T, WHOLE>(a.H), a.T), tokens = kThreads / G;
  ProfScope ps(name, s);
  return done(launch_pdl(sum_rows_backward_kernel<T, WHOLE, K>, ctas(a.T, tokens), kThreads, 0, s, a,
                         static_cast<const T*>(d_out), static_cast<const T*>(y), static_cast<T*>(d_y), d_w, G),
              name);
}
template <class T>
int sum_backward(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  if (!whole<T>(a)) return sum_backward_as<T, false, 2>(a, d_out, y, d_y, d_w, s);
  if (a.k <= 2) return sum_backward_as<T, true, 2>(a, d_out, y, d_y, d_w, s);
  return a.k <= 4 ? sum_backward_as<T, true, 4>(a, d_out, y, d_y, d_w, s) : sum_backward_as<T, true, 8>(a, d_out, y, d_y, d_w, s);
}

Args args(const SortedRows& r, const float* weights) {
  return Args{r.reverse, r.offsets, static_cast<int32_t*>(r.ws), r.T, r.k, r.E, r.H, weights, r.status};
}

}  // namespace

size_t sorted_rows_workspace(int T, int k) { return each_looks(T, k) ? 0 : align_up((size_t)T * k * sizeof(int32_t), 256); }

int launch_sum_sorted_rows(const SortedRows& r, const float* weights, const void* src, void* out, const char* name, cudaStream_t s) {
  Args a = args(r, weights);
  if (int rc = positions(a, s)) return rc;
  if (r.dtype == MOE_F32) return sum<float>(a, src, out, name, s);
  if (r.dtype == MOE_BF16) return sum<__nv_bfloat16>(a, src, out, name, s);
  return sum<__half>(a, src, out, name, s);
}

int launch_sum_sorted_rows_backward(const SortedRows& r, const float* weights, const void* d_out, const void* y, void* d_y,
                                    float* d_weights, cudaStream_t s) {
  Args a = args(r, weights);
  if (int rc = positions(a, s)) return rc;
  if (r.dtype == MOE_F32) return sum_backward<float>(a, d_out, y, d_y, d_weights, s);
  if (r.dtype == MOE_BF16) return sum_backward<__nv_bfloat16>(a, d_out, y, d_y, d_weights, s);
  return sum_backward<__half>(a, d_out, y, d_y, d_weights, s);
}

int launch_gather_any_rows(const void* src, const int32_t* ids, const int32_t* offsets, int elem_bytes, int T, int H, int E, int S,
                           void* out, cudaStream_t s) {
  const char* name = "gather_rows";
  const int grid = (int)std::max(1L, std::min((long)num_sms() * 8, ((long)S + 7) / 8));
  ProfScope ps(name, s);
  if (elem_bytes == 4)
    return done(launch_pdl(gather_any_rows_kernel<float>, grid, kThreads, 0, s, static_cast<const float*>(src), ids, offsets, E, T, S, H,
                           static_cast<float*>(out)),
                name);
  return done(launch_pdl(gather_any_rows_kernel<__half>, grid, kThreads, 0, s, static_cast<const __half*>(src), ids, offsets, E, T, S, H,
                         static_cast<__half*>(out)),
              name);
}

}  // namespace moe
