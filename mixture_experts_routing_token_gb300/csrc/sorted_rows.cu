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

#include "values.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 8;               // slots of a token whose rows are under way together
constexpr int kScanSlots = 2048;        // up to this many slots a CTA finds its own (see above)
constexpr int kSlotsPerCta = kThreads / 32 * MOE_MAX_TOPK;

// V neighbouring values: 16 bytes, or one where rows are not a multiple of that.
template <class T, bool VEC>
struct Piece {
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  float v[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (!VEC) {
      v[0] = to_float(__ldg(p));
    } else if constexpr (sizeof(T) == 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p));
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      load8(p, v);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (!VEC) {
      *p = from_float<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
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
    for (int p = threadIdx.x; p < n; p += kThreads) {
      const int i = __ldg(a.reverse + p) - s0;
      if (i >= 0 && i < count) pos[i] = p;
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

// out[t] = sum_j w[t, j] src[pos(t, j)]. G threads take a token.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) sum_rows_kernel(const Args a, const T* __restrict__ src, T* __restrict__ out, int G) {
  using P = Piece<T, VEC>;
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
  for (int c = threadIdx.x % G; c < pieces; c += G) {
    P sum;
#pragma unroll
    for (int q = 0; q < P::V; ++q) sum.v[q] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += kGroup) {
      P y[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (j0 + j < a.k && at[j0 + j] >= 0) y[j].load(src + (long)at[j0 + j] * a.H + c * P::V);
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (j0 + j < a.k && at[j0 + j] >= 0) {
          const float wj = w ? __ldg(w + j0 + j) : 1.0f;
#pragma unroll
          for (int q = 0; q < P::V; ++q) sum.v[q] += wj * y[j].v[q];
        }
    }
    sum.store(out + (long)t * a.H + c * P::V);
  }
}

// d_y[pos(t, j)] = w[t, j] d_out[t] and d_w[t, j] = <d_out[t], y[pos(t, j)]>; either may be null.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    sum_rows_backward_kernel(const Args a, const T* __restrict__ d_out, const T* __restrict__ y, T* __restrict__ d_y,
                             float* __restrict__ d_w, int G) {
  using P = Piece<T, VEC>;
  __shared__ int pos[kSlotsPerCta];
  __shared__ float part[kThreads / 32][kGroup];
  pdl_wait();
  pdl_trigger();
  const int tokens = kThreads / G, t0 = blockIdx.x * tokens;
  take_positions(a, t0 * a.k, min(tokens, a.T - t0) * a.k, pos);
  const int local = threadIdx.x / G, t = t0 + local;
  const bool in = t < a.T;
  const int* at = pos + (in ? local : 0) * a.k;
  const float* w = a.weights + (long)(in ? t : 0) * a.k;
  const int pieces = a.H / P::V;
  for (int j0 = 0; j0 < a.k; j0 += kGroup) {
    float dot[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) dot[j] = 0.0f;
    for (int c = threadIdx.x % G; in && c < pieces; c += G) {
      P d, r[kGroup];
      d.load(d_out + (long)t * a.H + c * P::V);
      if (d_w != nullptr) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
          if (j0 + j < a.k && at[j0 + j] >= 0) r[j].load(y + (long)at[j0 + j] * a.H + c * P::V);
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
          if (j0 + j < a.k && at[j0 + j] >= 0) {
#pragma unroll
            for (int q = 0; q < P::V; ++q) dot[j] += d.v[q] * r[j].v[q];
          }
      }
      if (d_y != nullptr) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
          if (j0 + j < a.k && at[j0 + j] >= 0) {
            const float wj = __ldg(w + j0 + j);
            P o;
#pragma unroll
            for (int q = 0; q < P::V; ++q) o.v[q] = wj * d.v[q];
            o.store(d_y + (long)at[j0 + j] * a.H + c * P::V);
          }
      }
    }
    if (d_w == nullptr) continue;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
#pragma unroll
      for (int s = 16; s; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (in && threadIdx.x % G < kGroup && j0 + threadIdx.x % G < a.k) {
      float sum = 0.0f;
      for (int i = 0; i < G / 32; ++i) sum += part[warp + i][lane];
      d_w[(long)t * a.k + j0 + lane] = sum;
    }
    __syncthreads();
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
  if (S <= kScanSlots) {
    a.pos = nullptr;
    return MOE_OK;
  }
  ProfScope ps("slot_positions", s);
  const int grid = (int)std::min((long)num_sms() * 4, (S + kThreads - 1) / kThreads);
  return done(launch_pdl(slot_positions_kernel, grid, kThreads, 0, s, a), "slot_positions");
}

// Threads of a token: as many as it has pieces, a power of two between a warp and the CTA.
int threads_per_token(int pieces) {
  int g = 32;
  while (g < kThreads && g < pieces) g *= 2;
  return g;
}

template <class T>
bool by_16_bytes(int H, std::initializer_list<const void*> rows) {
  if ((long)H * (int)sizeof(T) % 16 != 0) return false;
  for (const void* p : rows)
    if (!aligned(p, 16)) return false;
  return true;
}

template <class T, bool VEC>
int sum_as(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  const int G = threads_per_token(a.H / Piece<T, VEC>::V), tokens = kThreads / G;
  ProfScope ps(name, s);
  return done(launch_pdl(sum_rows_kernel<T, VEC>, (unsigned)((a.T + tokens - 1) / tokens), kThreads, 0, s, a, static_cast<const T*>(src),
                         static_cast<T*>(out), G),
              name);
}
template <class T>
int sum(const Args& a, const void* src, void* out, const char* name, cudaStream_t s) {
  return by_16_bytes<T>(a.H, {src, out}) ? sum_as<T, true>(a, src, out, name, s) : sum_as<T, false>(a, src, out, name, s);
}

template <class T, bool VEC>
int sum_backward_as(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  const char* name = "ep_combine_backward";
  const int G = threads_per_token(a.H / Piece<T, VEC>::V), tokens = kThreads / G;
  ProfScope ps(name, s);
  return done(launch_pdl(sum_rows_backward_kernel<T, VEC>, (unsigned)((a.T + tokens - 1) / tokens), kThreads, 0, s, a,
                         static_cast<const T*>(d_out), static_cast<const T*>(y), static_cast<T*>(d_y), d_w, G),
              name);
}
template <class T>
int sum_backward(const Args& a, const void* d_out, const void* y, void* d_y, float* d_w, cudaStream_t s) {
  return by_16_bytes<T>(a.H, {d_out, y, d_y}) ? sum_backward_as<T, true>(a, d_out, y, d_y, d_w, s)
                                              : sum_backward_as<T, false>(a, d_out, y, d_y, d_w, s);
}

Args args(const SortedRows& r, const float* weights) {
  return Args{r.reverse, r.offsets, static_cast<int32_t*>(r.ws), r.T, r.k, r.E, r.H, weights, r.status};
}

}  // namespace

size_t sorted_rows_workspace(int T, int k) { return (long)T * k <= kScanSlots ? 0 : align_up((size_t)T * k * sizeof(int32_t), 256); }

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
