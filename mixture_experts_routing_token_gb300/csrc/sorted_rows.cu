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
// leaves the others as they were: a reader takes an entry p only if reverse[p] is the slot (asked only if some slot was
// dropped) and p is a routed row, so that whatever else the buffer holds, no index leaves the arrays. With few slots
// each CTA of the one launch looks through reverse_indices itself instead.
#include <algorithm>
#include <type_traits>

#include "values.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 8;              // loads of sorted rows that a thread has under way
// Whether the CTAs look for their slots themselves. Measured, us, both gradients of bf16 rows of 512, from Python / in a
// graph, with the first kernel and its workspace, and without: 4000 slots of 500 tokens 26.5 / 11.7 and 13.5 / 10.7, 8000
// slots of 1000 tokens 27.5 / 12.4 and 14.3 / 14.8, of 8000 tokens 27.2 / 22.2 and 30.5 / 31.2.
bool each_looks(int T, int k) { return (long)T * k <= 2048 || ((long)T * k <= 8192 && T <= 2048); }
constexpr int kMinGroup = 4;            // threads of a token at least
constexpr int kSlotsPerCta = kThreads / kMinGroup * MOE_MAX_TOPK;

// B bytes of neighbouring values as they lie in memory: 16, or 4 or 2 where rows are not a multiple of more.
template <int B>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

template <class T, int B>
struct Piece {
  static constexpr int V = B / (int)sizeof(T);
  using W = typename Word<B>::type;
  W w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const W*>(p)); }
  __device__ __forceinline__ void values(float (&v)[V]) const {
    if constexpr (sizeof(T) == 4) {
      if constexpr (B == 16) {
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
      } else {
        v[0] = __uint_as_float(w);
      }
    } else if constexpr (B == 2) {
      v[0] = to_float(*reinterpret_cast<const T*>(&w));
    } else {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(q + i));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        } else {
          v[2 * i] = __uint_as_float(q[i] << 16);
          v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
      if constexpr (B == 16) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      else *p = v[0];
    } else if constexpr (B == 2) {
      *p = from_float<T>(v[0]);
    } else if constexpr (B == 4) {
      *reinterpret_cast<uint32_t*>(p) = grouped::pack_pair<T>(v[0], v[1]);
    } else {
      store8(p, v);
    }
  }
};

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
      if (p < 0 || p >= n || (n < S && __ldg(a.reverse + p) != s0 + i)) p = -1;
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
template <class T, int B, int K>
__global__ void __launch_bounds__(kThreads) sum_rows_kernel(const Args a, const T* __restrict__ src, T* __restrict__ out, int G) {
  using P = Piece<T, B>;
  constexpr int U = kFlight / K;
  __shared__ int pos[kSlotsPerCta];
  pdl_wait();
  pdl_trigger();
  const int tokens = kThreads / G, t0 = blockIdx.x * tokens;
  take_positions(a, t0 * a.k, min(tokens, a.T - t0) * a.k, pos);
  const int local = threadIdx.x / G, t = t0 + local;
  if (t >= a.T) return;
  const int* at = pos + local * a.k;
  const float* w = a.weights ? a.weights + (long)t * a.k : nullptr;
  const int pieces = a.H / P::V;
  for (int c0 = threadIdx.x % G; c0 < pieces; c0 += U * G) {
    float sum[U][P::V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < P::V; ++q) sum[u][q] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += K) {
      P y[K][U];
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j0 + j < a.k && at[j0 + j] >= 0 && c0 + u * G < pieces)
            y[j][u].load(src + (long)at[j0 + j] * a.H + (c0 + u * G) * P::V);
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j0 + j < a.k && at[j0 + j] >= 0) {
          const float wj = w ? __ldg(w + j0 + j) : 1.0f;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[P::V];
            y[j][u].values(v);
#pragma unroll
            for (int q = 0; q < P::V; ++q) sum[u][q] += wj * v[q];
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * G < pieces) P::store(out + (long)t * a.H + (c0 + u * G) * P::V, sum[u]);
  }
}

// d_y[pos(t, j)] = w[t, j] d_out[t] and d_w[t, j] = <d_out[t], y[pos(t, j)]>; either may be null.
template <class T, int B, int K>
__global__ void __launch_bounds__(kThreads)
    sum_rows_backward_kernel(const Args a, const T* __restrict__ d_out, const T* __restrict__ y, T* __restrict__ d_y,
                             float* __restrict__ d_w, int G) {
  using P = Piece<T, B>;
  constexpr int U = kFlight / K;
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
  const int pieces = a.H / P::V;
  for (int j0 = 0; j0 < a.k; j0 += K) {
    float dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) dot[j] = 0.0f;
    for (int c0 = me; in && c0 < pieces; c0 += U * G) {
      P d[U], r[K][U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * G < pieces) d[u].load(d_out + (long)t * a.H + (c0 + u * G) * P::V);
      if (d_w != nullptr) {
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (j0 + j < a.k && at[j0 + j] >= 0 && c0 + u * G < pieces)
              r[j][u].load(y + (long)at[j0 + j] * a.H + (c0 + u * G) * P::V);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + u * G >= pieces) continue;
        float dv[P::V];
        d[u].values(dv);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          if (j0 + j >= a.k || at[j0 + j] < 0) continue;
          if (d_w != nullptr) {
            float v[P::V];
            r[j][u].values(v);
#pragma unroll
            for (int q = 0; q < P::V; ++q) dot[j] += dv[q] * v[q];
          }
          if (d_y != nullptr) {
            const float wj = __ldg(w + j0 + j);
            float o[P::V];
#pragma unroll
            for (int q = 0; q < P::V; ++q) o[q] = wj * dv[q];
            P::store(d_y + (long)at[j0 + j] * a.H + (c0 + u * G) * P::V, o);
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

// out[p] = src[ids[p]] for the routed rows, rows of any width: 2 or 4 bytes at a time.
template <class W>
__global__ void __launch_bounds__(kThreads)
    gather_any_rows_kernel(const W* __restrict__ src, const int32_t* __restrict__ ids, const int32_t* __restrict__ offsets, int E,
                           int T, int S, int H, W* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int n = min(max(__ldg(offsets + E), 0), S), lane = threadIdx.x & 31;
  for (long p = (long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; p < n; p += (long)gridDim.x * (kThreads / 32)) {
    const int t = __ldg(ids + p);
    if (t < 0 || t >= T) continue;
    const W* from = src + (long)t * H;
    W* to = out + p * H;
    for (int c = lane; c < H; c += 32) to[c] = __ldg(from + c);
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

// Threads of a token, a power of two: no more than it has pieces, and no more than give every SM five CTAs.
int threads_per_token(int pieces, int T) {
  int g = kMinGroup;
  while (g < kThreads && g < pieces && (g < 32 || (long)T * g < 5L * kThreads * num_sms())) g *= 2;
  return g;
}

// Bytes of a row that are read at a time.
int piece_bytes(long row_bytes) { return row_bytes % 16 == 0 ? 16 : row_bytes % 4 == 0 ? 4 : 2; }

template <class T, int B, int K>
int sum_as(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  const int G = threads_per_token(a.H / Piece<T, B>::V, a.T), tokens = kThreads / G;
  ProfScope ps(name, s);
  return done(launch_pdl(sum_rows_kernel<T, B, K>, (unsigned)((a.T + tokens - 1) / tokens), kThreads, 0, s, a, static_cast<const T*>(src),
                         static_cast<T*>(out), G),
              name);
}
template <class T, int B>
int sum_of(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  return a.k <= 2 ? sum_as<T, B, 2>(a, src, out, name, s) : sum_as<T, B, kFlight>(a, src, out, name, s);
}
template <class T>
int sum(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  const int b = piece_bytes((long)a.H * (int)sizeof(T));
  if (b == 16) return sum_of<T, 16>(a, src, out, name, s);
  if constexpr (sizeof(T) == 2)
    if (b == 2) return sum_of<T, 2>(a, src, out, name, s);
  return sum_of<T, 4>(a, src, out, name, s);
}

template <class T, int B, int K>
int sum_backward_as(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  const char* name = "ep_combine_backward";
  const int G = threads_per_token(a.H / Piece<T, B>::V, a.T), tokens = kThreads / G;
  ProfScope ps(name, s);
  return done(launch_pdl(sum_rows_backward_kernel<T, B, K>, (unsigned)((a.T + tokens - 1) / tokens), kThreads, 0, s, a,
                         static_cast<const T*>(d_out), static_cast<const T*>(y), static_cast<T*>(d_y), d_w, G),
              name);
}
template <class T, int B>
int sum_backward_of(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  return a.k <= 2 ? sum_backward_as<T, B, 2>(a, d_out, y, d_y, d_w, s) : sum_backward_as<T, B, kFlight>(a, d_out, y, d_y, d_w, s);
}
template <class T>
int sum_backward(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  const int b = piece_bytes((long)a.H * (int)sizeof(T));
  if (b == 16) return sum_backward_of<T, 16>(a, d_out, y, d_y, d_w, s);
  if constexpr (sizeof(T) == 2)
    if (b == 2) return sum_backward_of<T, 2>(a, d_out, y, d_y, d_w, s);
  return sum_backward_of<T, 4>(a, d_out, y, d_y, d_w, s);
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
    return done(launch_pdl(gather_any_rows_kernel<uint32_t>, grid, kThreads, 0, s, static_cast<const uint32_t*>(src), ids, offsets, E,
                           T, S, H, static_cast<uint32_t*>(out)),
                name);
  return done(launch_pdl(gather_any_rows_kernel<uint16_t>, grid, kThreads, 0, s, static_cast<const uint16_t*>(src), ids, offsets, E, T,
                         S, H, static_cast<uint16_t*>(out)),
              name);
}

}  // namespace moe
