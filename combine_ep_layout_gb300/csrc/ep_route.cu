// ep_route.cu -- the router: scores to top-k expert ids and weights, and the
// gradient of the scores (include/ep_gb300_moe.h states the formulas).
//
// One warp serves one token.  Lane l holds the V = ceil(E / 32) consecutive
// scores [l V, l V + V) as 32-bit keys whose unsigned order is the scores'
// order (0 = not choosable), so that the lowest lane and then the lowest slot
// among equal keys is the lowest expert id.  Each of the K rounds takes the
// warp's largest key with one redux, finds the first lane that holds it, and
// that lane drops it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_moe_kernels.hpp"

namespace epg {
namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

template <class T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Order-preserving key of a score: larger score, larger key; -0 equals +0;
// 0 for -inf and NaN, which are never chosen.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  const uint32_t k = u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  return z > -INFINITY ? k : 0u;
}

__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// exp(z - peak) for z <= peak; a +inf peak leaves 1 for the +inf scores and 0
// for the others (the limit).  Masked scores (not > -inf) give 0.
__device__ __forceinline__ float exp_below(float z, float peak) {
  if (!(z > -INFINITY)) return 0.0f;
  return z == peak ? 1.0f : expf(z - peak);
}

__device__ __forceinline__ float sigmoid(float z) {
  return z > -INFINITY ? 1.0f / (1.0f + expf(-z)) : 0.0f;
}

// sigmoid(z) * exp(-min(peak, 0)) for z <= peak: scores that are all far below
// zero keep their ratios instead of vanishing together.
__device__ __forceinline__ float sigmoid_scaled(float z, float peak) {
  if (!(z > -INFINITY)) return 0.0f;
  if (peak >= 0.0f) return sigmoid(z);
  return expf(z - peak) / (1.0f + expf(z));
}

// The V scores of a lane as floats (-inf past the end of the row).
template <class T, int V>
__device__ __forceinline__ void load_row(const T* row, int experts, int lane, bool vec, float (&z)[V]) {
  constexpr int kPer = 16 / sizeof(T);
  const int j0 = lane * V;
  if constexpr (V % kPer == 0) {
    if (vec && j0 + V <= experts) {
#pragma unroll
      for (int v = 0; v < V; v += kPer) {
        const uint4 q = *reinterpret_cast<const uint4*>(row + j0 + v);
        const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
        for (int i = 0; i < kPer; ++i) z[v + i] = as_float(e[i]);
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) z[v] = j0 + v < experts ? as_float(row[j0 + v]) : -INFINITY;
}

// Peak of a row (-inf when nothing is choosable) from its lane-held scores.
template <int V>
__device__ __forceinline__ float row_peak(const float (&z)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) m = max(m, key_of(z[v]));
  m = __reduce_max_sync(kAll, m);
  return m ? value_of(m) : -INFINITY;
}

template <int V>
__device__ __forceinline__ float row_exp_sum(const float (&z)[V], float peak) {
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) s += exp_below(z[v], peak);
  return warp_sum(s);
}

template <class T, int V, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteParams p, bool vec) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.n) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.row_stride;
  float z[V];
  load_row<T, V>(row, p.experts, lane, vec, z);
  const bool whole = !p.sigmoid && (BIAS || !p.renorm);   // the softmax's full sum is needed
  const float peak = row_peak(z);
  const float sum = whole ? row_exp_sum(z, peak) : 1.0f;
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int j = lane * V + v;
    if constexpr (BIAS) {
      const float f = p.sigmoid ? sigmoid(z[v]) : exp_below(z[v], peak) / sum;
      key[v] = j < p.experts && z[v] > -INFINITY ? key_of(f + p.bias[j]) : 0u;
    } else {
      key[v] = key_of(z[v]);
    }
  }
  int chosen = -1;                                        // lane k: the k-th expert
  for (int k = 0; k < p.topk; ++k) {
    uint32_t best = 0;
    int slot = 0;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] >= best) best = key[v], slot = v;
    const uint32_t top = __reduce_max_sync(kAll, best);
    if (top == 0) break;
    const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
    const int id = __shfl_sync(kAll, lane * V + slot, src);
    if (lane == k) chosen = id;
    if (lane == src) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == slot) key[v] = 0;
    }
  }
  const float zk = chosen >= 0 ? as_float(row[chosen]) : -INFINITY;
  float f;
  if (p.sigmoid) {
    // the largest chosen score: with a selection bias not the first one
    uint32_t m = __reduce_max_sync(kAll, key_of(zk));
    f = p.renorm ? sigmoid_scaled(zk, m ? value_of(m) : 0.0f) : sigmoid(zk);
  } else if (p.renorm) {
    uint32_t m = __reduce_max_sync(kAll, key_of(zk));
    f = exp_below(zk, m ? value_of(m) : -INFINITY);
  } else {
    f = sum > 0.0f ? exp_below(zk, peak) / sum : 0.0f;
  }
  if (p.renorm) {
    const float tot = warp_sum(f);
    f = tot > 0.0f ? f / tot : 0.0f;
  }
  if (lane < p.topk) {
    p.idx[t * p.topk + lane] = chosen;
    p.weights[t * p.topk + lane] = chosen >= 0 ? f * p.scale : 0.0f;
  }
}

template <class T, int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteParams p, bool vec) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.n) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.row_stride;
  T* out = static_cast<T*>(p.grad) + t * p.grad_stride;
  int64_t id = -1;
  float g = 0.0f, zk = -INFINITY;
  if (lane < p.topk) {
    id = p.idx_in[t * p.topk + lane];
    if (id < 0 || id >= p.experts) id = -1;
    if (id >= 0) {
      g = p.grad_w[t * p.topk + lane] * p.scale;
      zk = as_float(row[id]);
    }
  }
  const bool full = !p.sigmoid && !p.renorm;              // the gradient reaches every expert
  float d, spread = 0.0f, peak = 0.0f, inv = 0.0f;
  if (full) {
    float z[V];
    load_row<T, V>(row, p.experts, lane, vec, z);
    peak = row_peak(z);
    const float sum = row_exp_sum(z, peak);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float fk = exp_below(zk, peak) * inv;
    spread = warp_sum(id >= 0 ? g * fk : 0.0f);
    d = fk * (g - spread);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = lane * V + v;
      if (j < p.experts)
        out[j] = from_float<T>(z[v] > -INFINITY ? -spread * exp_below(z[v], peak) * inv : 0.0f);
    }
  } else {
    for (int j = lane; j < p.experts; j += 32) out[j] = from_float<T>(0.0f);
    const uint32_t m = __reduce_max_sync(kAll, key_of(zk));
    const float top = m ? value_of(m) : -INFINITY;
    const float s = p.sigmoid ? sigmoid(zk) : 0.0f;
    float f = !p.renorm ? s : p.sigmoid ? sigmoid_scaled(zk, m ? top : 0.0f) : exp_below(zk, top);
    if (p.renorm) {
      const float tot = warp_sum(f);
      f = tot > 0.0f ? f / tot : 0.0f;
      const float mean = warp_sum(id >= 0 ? g * f : 0.0f);
      d = f * (g - mean);
    } else {
      d = f * g;
    }
    if (p.sigmoid) d *= 1.0f - s;
  }
  __syncwarp();                                           // the row's writes come before the K entries'
  if (id >= 0) out[id] = from_float<T>(zk > -INFINITY ? d : 0.0f);
}

bool aligned16(const void* p, int64_t stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride_bytes)) & 15u) == 0;
}

template <class T, int V>
cudaError_t launch_v(const RouteParams& p, bool backward, cudaStream_t s) {
  const bool vec = aligned16(p.logits, p.row_stride * static_cast<int64_t>(sizeof(T)));
  const unsigned grid = static_cast<unsigned>((p.n + kWarps - 1) / kWarps);
  if (backward)
    route_backward_kernel<T, V><<<grid, kWarps * 32, 0, s>>>(p, vec);
  else if (p.bias)
    route_kernel<T, V, true><<<grid, kWarps * 32, 0, s>>>(p, vec);
  else
    route_kernel<T, V, false><<<grid, kWarps * 32, 0, s>>>(p, vec);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch(const RouteParams& p, bool backward, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  if (p.experts <= 32) return launch_v<T, 1>(p, backward, s);
  if (p.experts <= 64) return launch_v<T, 2>(p, backward, s);
  if (p.experts <= 128) return launch_v<T, 4>(p, backward, s);
  if (p.experts <= 256) return launch_v<T, 8>(p, backward, s);
  if (p.experts <= 512) return launch_v<T, 16>(p, backward, s);
  if (p.experts <= 1024) return launch_v<T, 32>(p, backward, s);
  return launch_v<T, 64>(p, backward, s);
}

}  // namespace

cudaError_t LaunchRoute(const RouteParams& p, cudaStream_t s) {
  return p.bf16 ? launch<__nv_bfloat16>(p, false, s) : launch<float>(p, false, s);
}

cudaError_t LaunchRouteBackward(const RouteParams& p, cudaStream_t s) {
  return p.bf16 ? launch<__nv_bfloat16>(p, true, s) : launch<float>(p, true, s);
}

}  // namespace epg
