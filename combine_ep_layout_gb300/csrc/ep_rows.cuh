// ep_rows.cuh -- a warp's row of router scores: lane l holds the V consecutive ones
// [l V, l V + V).  Shared by the router and the balance losses.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace epg {
namespace rows {

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

inline bool aligned16(const void* p, int64_t stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride_bytes)) & 15u) == 0;
}

}  // namespace rows
}  // namespace epg
