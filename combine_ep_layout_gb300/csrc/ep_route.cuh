// ep_route.cuh -- one warp's part of the router: the choice of K among a row's keys
// and the weights of what was chosen.  Shared by the router's kernel and the MoE
// layer, which routes a few tokens itself.
#pragma once

#include <cstdint>
#include <type_traits>

namespace epg {
namespace route {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// exp(z - peak) for z <= peak; a +inf peak leaves 1 for the +inf scores and 0
// for the others (the limit).  Masked scores (-inf) give 0.
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

// Largest score of a row (-inf when nothing is choosable).
template <int V>
__device__ __forceinline__ float lane_max(const float (&z)[V]) {
  float m = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
  return m;
}

// The keys lie lane V + v (consecutive in a lane) or 32 v + lane (STRIDED).  Lane k
// (< topk <= KT): the id of the k-th largest key, the lower id first among
// equals, and the key; -1 and -inf where fewer keys are above -inf.  key_of(id)
// gives any key of the row, `slots` are 32 of the warp's own.  The steps are KT
// whatever topk is, so that they unroll: more of them only lower the bound and fill
// lanes that nobody reads.
template <int V, int KT, bool STRIDED, class KeyOf>
__device__ __forceinline__ int choose(float (&key)[V], int topk, int lane, int* slots, KeyOf key_of, float& chosen_key) {
  auto id_of = [&](int v) { return STRIDED ? 32 * v + lane : lane * V + v; };
  float val = key[0];
  int id = lane;
  if constexpr (V > 1) {
    float top = lane_max(key), bound = 0.0f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      bound = warp_max(top);
      if (top == bound) top = -INFINITY;
    }
    // -inf where fewer than KT lanes hold a key: then every key counts
    bound = fmaxf(bound, __int_as_float(0xff7fffff));
    using Mask = std::conditional_t<(V > 32), uint64_t, uint32_t>;
    Mask mine = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] >= bound) mine |= Mask{1} << v;
    int n = 0;
    const unsigned below = (1u << lane) - 1u;
    // lanes with more to give: two or three turns for the usual K and a few keys
    for (unsigned who; n <= 32 && (who = __ballot_sync(kAll, mine != 0)) != 0; n += __popc(who)) {
      const int at = n + __popc(who & below);
      if (mine != 0 && at < 32) slots[at] = id_of((V > 32 ? __ffsll(static_cast<long long>(mine)) : __ffs(static_cast<int>(mine))) - 1);
      mine &= mine - 1;
    }
    if (n > 32) {   // more keys than lanes: search the row K times
      int chosen = -1;
      for (int i = 0; i < topk; ++i) {
        float best = -INFINITY;
        int slot = 0;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if (key[v] >= best) best = key[v], slot = v;
        const float m = warp_max(best);
        if (!(m > -INFINITY)) break;
        const int j = static_cast<int>(__reduce_min_sync(kAll, best == m ? static_cast<unsigned>(id_of(slot)) : 0xffffffffu));
        if (lane == i) chosen = j, chosen_key = m;
        if (id_of(slot) == j) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v == slot) key[v] = -INFINITY;
        }
      }
      return chosen;
    }
    __syncwarp();
    id = lane < n ? slots[lane] : -1;
    val = lane < n ? key_of(id) : -INFINITY;
  }
  int chosen = -1;
#pragma unroll
  for (int k = 0; k < KT; ++k) {
    const float m = warp_max(val);
    const int j = static_cast<int>(__reduce_min_sync(kAll, val == m ? static_cast<unsigned>(id) : 0xffffffffu));
    if (lane == k) chosen = j, chosen_key = m;
    if (id == j) val = -INFINITY;
  }
  if (lane >= topk || !(chosen_key > -INFINITY)) chosen = -1, chosen_key = -INFINITY;
  return chosen;
}

// The weights of chosen scores (lane k: zk, -inf: none) that need no other score:
// renormalised, or a sigmoid's own.
__device__ __forceinline__ float chosen_weight(float zk, bool is_sigmoid, bool renorm) {
  if (!renorm) return sigmoid(zk);
  const float top = warp_max(zk);   // with a selection bias not the first one
  const float f = is_sigmoid ? sigmoid_scaled(zk, top) : exp_below(zk, top);
  const float tot = warp_sum(f);
  return tot > 0.0f ? f / tot : 0.0f;
}

}  // namespace route
}  // namespace epg
