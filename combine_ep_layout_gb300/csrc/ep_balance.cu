// ep_balance.cu -- the router's training losses and their gradient
// (include/ep_gb300_balance.h states the formulas).
//
// Bound by reading the scores once; a score costs one exp (sigmoid: two).
//
// Forward, two launches: each block of the first takes a run of consecutive
// tokens, a warp a token at a time, and keeps a column of sums in every lane; for each
// sequence that its run touches it writes one row of sums (probabilities, counts,
// live tokens, squared lse).  The second adds those rows, 32 experts a block, and the last of its
// blocks adds the losses.  The pairs (block, sequence) with tokens form a staircase, so
// block + sequence numbers their rows.  Every sum has a fixed order; only whole numbers go
// through atomics.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_balance_kernels.hpp"
#include "ep_kernels.hpp"
#include "ep_route.cuh"
#include "ep_rows.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

using namespace route;
using namespace rows;

constexpr int kWarps = 8;

// A lane's scores of a row.  VEC: V consecutive ones; else every 32nd, which rows that are not
// 16-byte aligned are read by in whole sectors.
template <bool VEC, int V>
__device__ __forceinline__ int expert_of(int lane, int v) {
  return VEC ? lane * V + v : 32 * v + lane;
}

template <class T, int V, bool VEC>
__device__ __forceinline__ void load_scores(const T* row, int experts, int lane, float (&z)[V]) {
  if constexpr (VEC) {
    load_row<T, V>(row, experts, lane, true, z);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = 32 * v + lane;
      z[v] = j < experts ? fmaxf(as_float(row[j]), -INFINITY) : -INFINITY;
    }
  }
}

// z becomes p; returns lse, -inf where every score is masked.  SIGMOID: soft gets exp(z - peak),
// not_s gets 1 - sigmoid(z).
template <int V, bool SIGMOID, bool GRAD>
__device__ __forceinline__ float probabilities(float (&z)[V], float (&soft)[V], float (&not_s)[V]) {
  const float peak = warp_max(lane_max(z));
  float whole = 0.0f, part = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float e = exp_below(z[v], peak);
    whole += e;
    if constexpr (SIGMOID) {
      // scaled by exp(-peak) where every score is below zero, so that ratios survive
      const float t = expf(-fabsf(z[v])), inv = 1.0f / (1.0f + t);
      const float s = peak < 0.0f ? e * inv : z[v] >= 0.0f ? inv : t * inv;
      if constexpr (GRAD) soft[v] = e, not_s[v] = z[v] >= 0.0f ? t * inv : inv;
      z[v] = z[v] > -INFINITY ? s : 0.0f;
      part += z[v];
    } else {
      z[v] = e;
    }
  }
  whole = warp_sum(whole);
  if constexpr (SIGMOID) part = warp_sum(part);
  const float inv = whole > 0.0f ? 1.0f / whole : 0.0f;
  const float inv_p = SIGMOID ? (part > 0.0f ? 1.0f / part : 0.0f) : inv;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    z[v] *= inv_p;
    if constexpr (SIGMOID && GRAD) soft[v] *= inv;
  }
  return whole > 0.0f ? peak + logf(whole) : -INFINITY;
}

__device__ __forceinline__ int offset_at(const BalanceParams& p, int g) {
  return p.offsets ? min(max(p.offsets[g], 0), p.n) : (g ? p.n : 0);
}

// The first sequence that ends behind token t.
__device__ __forceinline__ int sequence_of(const BalanceParams& p, int t) {
  int lo = 0, hi = p.sequences;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offset_at(p, mid + 1) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__host__ __device__ __forceinline__ int run_of(int n, int blocks) { return (n + blocks - 1) / blocks; }

template <class T, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32) balance_sums_kernel(BalanceParams p) {
  extern __shared__ float shared[];                  // [kWarps][E] sums, [E] counts
  __shared__ float zz[kWarps];
  __shared__ int live_of[kWarps];
  allow_dependent_grids();
  int* cnt = reinterpret_cast<int*>(shared + kWarps * p.experts);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = run_of(p.n, p.blocks), start = static_cast<int>(blockIdx.x) * run, end = min(start + run, p.n);
  grid_dependency_wait();
  for (int at = start, g; at < end && (g = sequence_of(p, at)) < p.sequences;) {
    const int from = max(at, offset_at(p, g)), to = min(end, offset_at(p, g + 1));
    at = max(to, at + 1);
    if (from >= to) continue;
    for (int e = threadIdx.x; e < p.experts; e += kWarps * 32) cnt[e] = 0;
    __syncthreads();
    float acc[V], squares = 0.0f;
    int live = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    for (int t = from + warp; t < to; t += kWarps) {
      float z[V], none[V];
      load_scores<T, V, VEC>(static_cast<const T*>(p.logits) + t * p.row_stride, p.experts, lane, z);
      int64_t id = -1;
      if (lane < p.topk) id = p.idx[static_cast<int64_t>(t) * p.topk + lane];
      const bool valid = id >= 0 && id < p.experts;
      if (!__any_sync(kAll, valid)) continue;
      if (valid) atomicAdd(cnt + id, 1);
      const float lse = probabilities<V, SIGMOID, false>(z, none, none);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += z[v];
      squares += lse > -INFINITY ? lse * lse : 0.0f;
      ++live;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = expert_of<VEC, V>(lane, v);
      if (j < p.experts) shared[warp * p.experts + j] = acc[v];
    }
    if (lane == 0) zz[warp] = squares, live_of[warp] = live;
    __syncthreads();
    float* out = p.sums + (static_cast<int64_t>(blockIdx.x) + g) * (2 * p.experts + 2);
    for (int e = threadIdx.x; e < p.experts; e += kWarps * 32) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += shared[w * p.experts + e];
      out[e] = s;
      out[p.experts + e] = __int_as_float(cnt[e]);
    }
    if (threadIdx.x == 0) {
      float s = 0.0f;
      int k = 0;
      for (int w = 0; w < kWarps; ++w) s += zz[w], k += live_of[w];
      out[2 * p.experts] = __int_as_float(k);
      out[2 * p.experts + 1] = s;
    }
    __syncthreads();
  }
}

__device__ __forceinline__ float ld(const float* p) { return ld_coherent(p); }

// Sum over the block, in thread 0 (in a fixed order).
__device__ __forceinline__ float block_sum(float v, float* shared) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x == 0)
    for (int w = 0; w < kWarps; ++w) s += shared[w];
  return s;
}

// grid: the column blocks of each sequence in turn
__global__ void __launch_bounds__(kWarps * 32) balance_final_kernel(BalanceParams p) {
  __shared__ float sums[kWarps][32], red[kWarps];
  __shared__ int cnts[kWarps][32], lives[kWarps];
  __shared__ bool last;
  allow_dependent_grids();
  const int columns = (p.experts + kBalanceColumns - 1) / kBalanceColumns;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = static_cast<int>(blockIdx.x) / columns, column = static_cast<int>(blockIdx.x) % columns;
  const int e = column * kBalanceColumns + lane;
  grid_dependency_wait();
  const int run = run_of(p.n, p.blocks), from = offset_at(p, g), to = offset_at(p, g + 1), words = 2 * p.experts + 2;
  // the blocks that have tokens of this sequence
  const int b0 = to > from ? from / run : 0, b1 = to > from ? (to - 1) / run + 1 : 0;
  float sum = 0.0f, squares = 0.0f;
  int count = 0, live = 0;
#pragma unroll 4
  for (int b = b0 + warp; b < b1; b += kWarps) {
    const float* row = p.sums + (static_cast<int64_t>(b) + g) * words;
    if (e < p.experts) sum += ld(row + e), count += __float_as_int(ld(row + p.experts + e));
    live += __float_as_int(ld(row + 2 * p.experts));
    squares += ld(row + 2 * p.experts + 1);
  }
  sums[warp][lane] = sum, cnts[warp][lane] = count;
  if (lane == 0) lives[warp] = live, red[warp] = squares;
  __syncthreads();
  if (warp == 0) {
    sum = squares = 0.0f, count = live = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sums[w][lane], count += cnts[w][lane], live += lives[w], squares += red[w];
    if (e < p.experts) {
      p.counts[static_cast<int64_t>(g) * p.experts + e] = count;
      p.prob_sums[static_cast<int64_t>(g) * p.experts + e] = sum;
    }
    const float share = live ? static_cast<float>(p.experts) / (static_cast<float>(p.topk) * p.sequences) / live / live : 0.0f;
    const float dot = warp_sum(e < p.experts ? static_cast<float>(count) * sum : 0.0f) * share;
    if (lane == 0) {
      float* part = p.parts + 2 * static_cast<int64_t>(blockIdx.x);
      part[0] = dot;
      part[1] = column ? 0.0f : squares;
      if (column == 0) p.tokens[g] = live;
      __threadfence();
      last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float loss = 0.0f, z = 0.0f;
  int total = 0;
  for (int64_t i = threadIdx.x; i < gridDim.x; i += kWarps * 32) loss += ld(p.parts + 2 * i), z += ld(p.parts + 2 * i + 1);
  for (int i = threadIdx.x; i < p.sequences; i += kWarps * 32) total += ld_coherent(p.tokens + i);
  loss = block_sum(loss, red);
  z = block_sum(z, red);
  total = __reduce_add_sync(kAll, total);
  __syncthreads();
  if (lane == 0) lives[warp] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    total = 0;
    for (int w = 0; w < kWarps; ++w) total += lives[w];
    p.loss[0] = loss;
    p.loss[1] = total ? z / total : 0.0f;
    p.tokens[p.sequences] = total;
    *p.ticket = 0;
  }
}

template <class T, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32) balance_backward_kernel(BalanceParams p) {
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (t >= p.n) return;
  const int g = sequence_of(p, t);
  if (g >= p.sequences || t < offset_at(p, g)) return;
  float z[V], soft[V], not_s[V], d[V];
  load_scores<T, V, VEC>(static_cast<const T*>(p.logits) + t * p.row_stride, p.experts, lane, z);
  int64_t id = -1;
  if (lane < p.topk) id = p.idx[static_cast<int64_t>(t) * p.topk + lane];
  const bool live = __any_sync(kAll, id >= 0 && id < p.experts);
  T* out = static_cast<T*>(p.grad) + t * p.grad_stride;
  if (live) {
    const int tg = p.tokens_in[g], total = p.tokens_in[p.sequences];
    // sum p = 1, so any constant may be taken from the counts; their mean leaves the most bits
    const int mean = static_cast<int>(static_cast<int64_t>(tg) * p.topk / p.experts);
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = expert_of<VEC, V>(lane, v);
      c[v] = j < p.experts ? static_cast<float>(p.counts_in[static_cast<int64_t>(g) * p.experts + j] - mean) : 0.0f;
    }
    const float lse = probabilities<V, SIGMOID, true>(z, soft, not_s);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) dot = fmaf(c[v], z[v], dot);
    dot = warp_sum(dot);
    const float share = tg > 0 ? p.grad_loss[0] * (static_cast<float>(p.experts) / (static_cast<float>(p.topk) * p.sequences)) / tg / tg : 0.0f;
    const float rise = total > 0 && lse > -INFINITY ? p.grad_loss[1] * 2.0f * lse / total : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float s = SIGMOID ? soft[v] : z[v];
      d[v] = share * z[v] * (c[v] - dot);
      if constexpr (SIGMOID) d[v] *= not_s[v];
      d[v] = s > 0.0f ? fmaf(rise, s, d[v]) : (z[v] > 0.0f ? d[v] : 0.0f);
    }
  } else {
    if (p.accumulate) return;
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = 0.0f;
  }
  if (p.accumulate) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = expert_of<VEC, V>(lane, v);
      if (j < p.experts) d[v] += as_float(out[j]);
    }
  }
  if constexpr (VEC) {
    store_row<T, V>(out, p.experts, lane, true, d);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = 32 * v + lane;
      if (j < p.experts) out[j] = from_float<T>(d[v]);
    }
  }
}

template <class K>
cudaError_t launch_pdl(K kernel, dim3 grid, size_t smem, cudaStream_t s, const BalanceParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  static const bool pdl = PdlEnabled();
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T, int V, bool VEC, bool SIGMOID>
cudaError_t launch_one(const BalanceParams& p, bool backward, cudaStream_t s) {
  if (backward) return launch_pdl(balance_backward_kernel<T, V, VEC, SIGMOID>, dim3((p.n + kWarps - 1) / kWarps), 0, s, p);
  const size_t smem = (kWarps + 1) * static_cast<size_t>(p.experts) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(balance_sums_kernel<T, V, VEC, SIGMOID>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(balance_sums_kernel<T, V, VEC, SIGMOID>, dim3(p.blocks), smem, s, p);
}

template <class T, int V>
cudaError_t launch_v(const BalanceParams& p, bool backward, cudaStream_t s) {
  const int64_t size = static_cast<int64_t>(sizeof(T));
  const bool vec = V * sizeof(T) >= 16 && aligned16(p.logits, p.row_stride * size) &&
                   (!backward || aligned16(p.grad, p.grad_stride * size));
  if (vec) return p.sigmoid ? launch_one<T, V, true, true>(p, backward, s) : launch_one<T, V, true, false>(p, backward, s);
  return p.sigmoid ? launch_one<T, V, false, true>(p, backward, s) : launch_one<T, V, false, false>(p, backward, s);
}

template <class T>
cudaError_t launch(const BalanceParams& p, bool backward, cudaStream_t s) {
  if (p.experts <= 32) return launch_v<T, 1>(p, backward, s);
  if (p.experts <= 64) return launch_v<T, 2>(p, backward, s);
  if (p.experts <= 128) return launch_v<T, 4>(p, backward, s);
  if (p.experts <= 256) return launch_v<T, 8>(p, backward, s);
  if (p.experts <= 512) return launch_v<T, 16>(p, backward, s);
  if (p.experts <= 1024) return launch_v<T, 32>(p, backward, s);
  return launch_v<T, 64>(p, backward, s);
}

}  // namespace

int BalanceBlocks(int n, int num_sms) {
  const int most = 4 * num_sms, some = (n + kWarps - 1) / kWarps;
  return some < 1 ? 1 : some < most ? some : most;
}

cudaError_t LaunchBalance(const BalanceParams& p, cudaStream_t s) {
  if (p.n > 0)
    if (const cudaError_t e = p.bf16 ? launch<__nv_bfloat16>(p, false, s) : launch<float>(p, false, s); e != cudaSuccess)
      return e;
  return launch_pdl(balance_final_kernel, dim3(static_cast<unsigned>(BalancePartWords(p.sequences, p.experts) / 2)), 0, s, p);
}

cudaError_t LaunchBalanceBackward(const BalanceParams& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  return p.bf16 ? launch<__nv_bfloat16>(p, true, s) : launch<float>(p, true, s);
}

}  // namespace epg
