// ep_route.cu -- the router: scores to top-k expert ids and weights, and the
// gradient of the scores (include/ep_gb300_moe.h states the formulas).
//
// One warp serves one token.  Lane l holds the V = ceil(E / 32) consecutive keys
// [l V, l V + V) (-inf: not choosable).  Bound by instructions, not by reading the
// scores, so the K choices are not K searches of the row:
//   1. the K-th largest (K rounded up to 8 or 16) of the 32 lane maxima is a bound that at least K keys
//      reach (one redux.max a step);
//   2. the keys that reach it -- K and a few, typically -- are gathered into
//      the first lanes through shared memory;
//   3. K steps take the largest of one key a lane, the lowest id among equals.
// Rows where more than 32 keys reach the bound (many equal scores) are searched K
// times.
//
// Measured: 32768 tokens of 256 fp32 scores, top-8, 14.3 us (2.6 TB/s), 357 instructions
// a token at 68% of the issue slots while busy; a search of the row for each choice
// took 26.7 us.  The gradient: 16384 x 128 bf16 together with the router 12.4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_kernels.hpp"
#include "ep_moe_kernels.hpp"
#include "ep_route.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

using namespace route;

constexpr int kWarps = 8;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (sizeof(T) == 4)
    return v;
  else
    return __float2bfloat16_rn(v);
}

// The V scores of a lane as floats; -inf past the end of the row and for NaN.
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
        for (int i = 0; i < kPer; ++i) z[v + i] = fmaxf(as_float(e[i]), -INFINITY);
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) z[v] = j0 + v < experts ? fmaxf(as_float(row[j0 + v]), -INFINITY) : -INFINITY;
}

// z becomes exp(z - peak); their sum over the row.
template <int V>
__device__ __forceinline__ float exp_row(float (&z)[V], float peak) {
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    z[v] = exp_below(z[v], peak);
    s += z[v];
  }
  return warp_sum(s);
}

template <class T, int V, int KT, bool BIAS>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteParams p, bool vec) {
  __shared__ int slots[kWarps][32];
  allow_dependent_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  grid_dependency_wait();
  if (t >= p.n) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.row_stride;
  float key[V];
  load_row<T, V>(row, p.experts, lane, vec, key);
  const bool whole = !p.sigmoid && (BIAS || !p.renorm);   // the softmax's full sum is needed
  float peak = 0.0f, sum = 1.0f;
  if (whole) {
    peak = warp_max(lane_max(key));
    float e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = key[v];
    sum = exp_row(e, peak);
  }
  auto biased = [&](float z, int j) {
    const float f = p.sigmoid ? sigmoid(z) : exp_below(z, peak) / sum;
    return z > -INFINITY ? fmaxf(f + p.bias[j], -INFINITY) : -INFINITY;
  };
  if constexpr (BIAS) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane * V + v < p.experts) key[v] = biased(key[v], lane * V + v);
  }
  float zk = -INFINITY;
  const int chosen = choose<V, KT, false>(
      key, p.topk, lane, slots[warp],
      [&](int j) {
        const float z = fmaxf(as_float(row[j]), -INFINITY);
        return BIAS ? biased(z, j) : z;
      },
      zk);
  if constexpr (BIAS) zk = chosen >= 0 ? as_float(row[chosen]) : -INFINITY;
  const float f = p.renorm || p.sigmoid ? chosen_weight(zk, p.sigmoid, p.renorm)
                  : sum > 0.0f          ? exp_below(zk, peak) / sum
                                        : 0.0f;
  if (lane < p.topk) {
    p.idx[t * p.topk + lane] = chosen;
    p.weights[t * p.topk + lane] = chosen >= 0 ? f * p.scale : 0.0f;
  }
}

// A lane's V values of an output row.
template <class T, int V>
__device__ __forceinline__ void store_row(T* row, int experts, int lane, bool vec, const float (&z)[V]) {
  constexpr int kPer = 16 / sizeof(T);
  const int j0 = lane * V;
  if constexpr (V % kPer == 0) {
    if (vec && j0 + V <= experts) {
#pragma unroll
      for (int v = 0; v < V; v += kPer) {
        uint4 q;
        T* e = reinterpret_cast<T*>(&q);
#pragma unroll
        for (int i = 0; i < kPer; ++i) e[i] = from_float<T>(z[v + i]);
        *reinterpret_cast<uint4*>(row + j0 + v) = q;
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (j0 + v < experts) row[j0 + v] = from_float<T>(z[v]);
}

// The gradient where it reaches every expert (softmax, not renormalised): a warp a
// token, as in the router.
template <class T, int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteParams p, bool vec, bool vec_out) {
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (t >= p.n) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.row_stride;
  T* out = static_cast<T*>(p.grad) + t * p.grad_stride;
  int64_t id = -1;
  float g = 0.0f, zk = -INFINITY, z[V];
  if (lane < p.topk) {
    id = p.idx_in[t * p.topk + lane];
    if (id < 0 || id >= p.experts) id = -1;
  }
  load_row<T, V>(row, p.experts, lane, vec, z);
  if (id >= 0) {
    g = p.grad_w[t * p.topk + lane] * p.scale;
    zk = fmaxf(as_float(row[id]), -INFINITY);
  }
  const float peak = warp_max(lane_max(z));
  const float sum = exp_row(z, peak);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  const float fk = exp_below(zk, peak) * inv;
  const float spread = warp_sum(id >= 0 ? g * fk : 0.0f);
#pragma unroll
  for (int v = 0; v < V; ++v) z[v] = z[v] > 0.0f ? -spread * z[v] * inv : 0.0f;
  store_row<T, V>(out, p.experts, lane, vec_out, z);
  __syncwarp();                                           // the row's writes come before the K entries'
  if (id >= 0) out[id] = from_float<T>(zk > -INFINITY ? fk * (g - spread) : 0.0f);
}

// The gradient where it stays with the chosen experts: GL (8 or 16, at least topk)
// lanes a token, several tokens a warp; zeros for the rows, then the entries.
template <class T, int GL>
__global__ void __launch_bounds__(kWarps * 32) route_backward_chosen_kernel(RouteParams p, bool vec_out) {
  constexpr int kTokens = 32 / GL, kPer = 16 / sizeof(T);
  allow_dependent_grids();
  const int lane = threadIdx.x & 31, k = lane % GL;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
  const int64_t t = t0 + lane / GL;
  grid_dependency_wait();
  if (t0 >= p.n) return;
  auto group_max = [](float v) {
#pragma unroll
    for (int d = GL / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
  };
  auto group_sum = [](float v) {
#pragma unroll
    for (int d = GL / 2; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
  };
  int64_t id = -1;
  float g = 0.0f, zk = -INFINITY;
  if (t < p.n && k < p.topk) {
    id = p.idx_in[t * p.topk + k];
    if (id < 0 || id >= p.experts) id = -1;
    if (id >= 0) {
      g = p.grad_w[t * p.topk + k] * p.scale;
      zk = fmaxf(as_float(static_cast<const T*>(p.logits)[t * p.row_stride + id]), -INFINITY);
    }
  }
  for (int r = 0; r < kTokens && t0 + r < p.n; ++r) {
    T* row = static_cast<T*>(p.grad) + (t0 + r) * p.grad_stride;
    int j0 = 0;
    if (vec_out) {
      for (int j = lane * kPer; j + kPer <= p.experts; j += 32 * kPer) *reinterpret_cast<uint4*>(row + j) = make_uint4(0, 0, 0, 0);
      j0 = p.experts / kPer * kPer;
    }
    for (int j = j0 + lane; j < p.experts; j += 32) row[j] = from_float<T>(0.0f);
  }
  const float s = p.sigmoid ? sigmoid(zk) : 0.0f;
  float d = s * g;
  if (p.renorm) {
    const float top = group_max(zk);
    float f = p.sigmoid ? sigmoid_scaled(zk, top) : exp_below(zk, top);
    const float tot = group_sum(f);
    f = tot > 0.0f ? f / tot : 0.0f;
    d = f * (g - group_sum(id >= 0 ? g * f : 0.0f));
  }
  if (p.sigmoid) d *= sigmoid(-zk);                       // 1 - s, with all its bits where s is near 1
  __syncwarp();                                           // the rows' writes come before the entries'
  if (id >= 0) static_cast<T*>(p.grad)[t * p.grad_stride + id] = from_float<T>(zk > -INFINITY ? d : 0.0f);
}

bool aligned16(const void* p, int64_t stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride_bytes)) & 15u) == 0;
}

template <class T, int V>
cudaError_t launch_v(const RouteParams& p, bool backward, cudaStream_t s) {
  const int64_t size = static_cast<int64_t>(sizeof(T));
  const bool vec = aligned16(p.logits, p.row_stride * size);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.n + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  static const bool pdl = PdlEnabled();
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (backward) {
    const bool vec_out = aligned16(p.grad, p.grad_stride * size);
    if (!p.sigmoid && !p.renorm) return cudaLaunchKernelEx(&cfg, route_backward_kernel<T, V>, p, vec, vec_out);
    const int tokens = p.topk <= 8 ? 4 : 2;
    cfg.gridDim = dim3(static_cast<unsigned>((p.n + kWarps * tokens - 1) / (kWarps * tokens)));
    return tokens == 4 ? cudaLaunchKernelEx(&cfg, route_backward_chosen_kernel<T, 8>, p, vec_out)
                       : cudaLaunchKernelEx(&cfg, route_backward_chosen_kernel<T, 16>, p, vec_out);
  }
  if (p.topk <= 8)
    return p.bias ? cudaLaunchKernelEx(&cfg, route_kernel<T, V, 8, true>, p, vec)
                  : cudaLaunchKernelEx(&cfg, route_kernel<T, V, 8, false>, p, vec);
  return p.bias ? cudaLaunchKernelEx(&cfg, route_kernel<T, V, 16, true>, p, vec)
                : cudaLaunchKernelEx(&cfg, route_kernel<T, V, 16, false>, p, vec);
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
