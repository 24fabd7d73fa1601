// ep_balance.cu -- the router's training losses and their gradient
// (include/ep_gb300_balance.h states the formulas).
//
// Bound by reading the scores once, as long as enough rows are under way; a score costs one
// exp (sigmoid: two).
//
// Forward, two launches: each block of the first takes a run of consecutive
// tokens, a warp a few tokens at a time, and keeps a column of sums in every lane; for each
// sequence that its run touches it writes one row of sums (probabilities, counts,
// live tokens, squared lse).  The second adds those rows, 32 experts a block, and the last of its
// blocks adds the losses.  Few tokens of one sequence: one block does both.  The
// pairs (block, sequence) with tokens form a staircase, so block + sequence numbers their
// rows.  Every sum has a fixed order; only whole numbers go through atomics.
//
// Backward: a warp takes up to 16 consecutive tokens, a few at a time, with the counts of their
// sequence in registers.
//
// Measured: 32768 x 256 fp32 scores, 8 sequences, both directions 39.5 us (1.75 TB/s); cold 17 us the sums
// (171 instructions a token, 41% of the issue slots while active), 7 the second launch, 17 the gradient
// (266 instructions a token, 49%).  What bounds them is latency: a block's search, rows, sums and output follow
// each other.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
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

constexpr int kFinalWarps = 16, kBackWarps = 8;
// Warps of a block of sums: registers allow 32 of them up to 256 experts.  Four rows at a time up to 128
// experts, two up to 256, one beyond.
__host__ __device__ constexpr int sum_warps(int v) { return v <= 8 ? 32 : v == 16 ? 16 : 8; }
__host__ __device__ constexpr int at_once(int v) { return v <= 4 ? 4 : v == 8 ? 2 : 1; }

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

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_of(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// U rows: z becomes p; peak and whole (the sum of exp(z - peak), 0 where every score is masked) give
// lse.  SIGMOID and GRAD: soft gets exp(z - lse), not_s 1 - sigmoid(z).  An exponential is one fma and one
// ex2 (off by 2^-22 and by the rounding of peak log2(e), which all of a row share); rows whose peak is
// infinite or next to it are subtracted first.
template <int U, int V, bool SIGMOID, bool GRAD, int SU, int SV>
__device__ __forceinline__ void probabilities(float (&z)[U][V], float (&soft)[SU][SV], float (&not_s)[SU][SV], float (&peak)[U],
                                              float (&whole)[U]) {
  float part[U];
  bool plain = true;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    peak[u] = warp_max(lane_max(z[u]));
    plain = plain && fabsf(peak[u]) < 1e30f;
    whole[u] = part[u] = 0.0f;
  }
  const auto score = [&](int u, int v, float e) {
    whole[u] += e;
    if constexpr (SIGMOID) {
      // scaled by exp(-peak) where every score is below zero, so that ratios survive
      const float x = z[u][v], t = exp2_of(-fabsf(x) * kLog2e), inv = reciprocal(1.0f + t);
      if constexpr (GRAD) soft[u][v] = e, not_s[u][v] = x >= 0.0f ? t * inv : inv;
      z[u][v] = peak[u] < 0.0f ? e * inv : x >= 0.0f ? inv : t * inv;
      part[u] += z[u][v];
    } else {
      z[u][v] = e;
    }
  };
  if (plain) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float c = -peak[u] * kLog2e;
#pragma unroll
      for (int v = 0; v < V; ++v) score(u, v, exp2_of(fmaf(z[u][v], kLog2e, c)));
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = z[u][v];
        score(u, v, x > -INFINITY ? (x == peak[u] ? 1.0f : exp2_of((x - peak[u]) * kLog2e)) : 0.0f);
      }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      whole[u] += __shfl_xor_sync(kAll, whole[u], d);
      if constexpr (SIGMOID) part[u] += __shfl_xor_sync(kAll, part[u], d);
    }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float inv = whole[u] > 0.0f ? reciprocal(whole[u]) : 0.0f;
    const float inv_p = SIGMOID ? (part[u] > 0.0f ? reciprocal(part[u]) : 0.0f) : inv;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[u][v] *= inv_p;
      if constexpr (SIGMOID && GRAD) soft[u][v] *= inv;
    }
  }
}

__device__ __forceinline__ float lse_of(float peak, float whole) { return whole > 0.0f ? peak + logf(whole) : -INFINITY; }

__device__ __forceinline__ int offset_at(const BalanceParams& p, int g) {
  return p.offsets ? min(max(p.offsets[g], 0), p.n) : (g ? p.n : 0);
}

// The first sequence that ends behind token t, and its ends (a whole warp, all lanes the same answer): 128
// places at a time, as each step is a round trip to L2.
__device__ __forceinline__ int sequence_of(const BalanceParams& p, int t, int lane, int& from, int& to) {
  from = 0, to = p.n;
  if (!p.offsets) return t < p.n ? 0 : p.sequences;
  int lo = 0, many = p.sequences;            // the answer is in [lo, lo + many]
  bool known = false;
  while (many > 0) {
    const int step = (many + 127) / 128, end = lo + many;
    int passed = 0, first[4], last[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {            // the last of this lane's stretch, and its ends
      const int g = lo + (32 * i + lane) * step + step - 1;
      const bool there = g < end || (g == end && step == 1 && end < p.sequences);
      first[i] = there && step == 1 ? offset_at(p, g) : 0;
      last[i] = there ? offset_at(p, g + 1) : 0;
      passed += __popc(__ballot_sync(kAll, g < end && last[i] <= t));
    }
    if (step == 1 && passed < 128) {
      known = true;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (passed / 32 == i) from = __shfl_sync(kAll, first[i], passed % 32), to = __shfl_sync(kAll, last[i], passed % 32);
    }
    lo = min(lo + passed * step, end);
    many = step > 1 ? min(step - 1, end - lo) : 0;
  }
  if (!known && lo < p.sequences) from = offset_at(p, lo), to = offset_at(p, lo + 1);
  return lo;
}

// A lane's choice of a token, -1 where it is no expert.
__device__ __forceinline__ int id_of(const BalanceParams& p, const int64_t* at) {
  const uint64_t id = static_cast<uint64_t>(*at);
  return id < static_cast<uint64_t>(p.experts) ? static_cast<int>(id) : -1;
}

__host__ __device__ __forceinline__ int run_of(int n, int blocks) { return (n + blocks - 1) / blocks; }

__device__ __forceinline__ float ld(const float* p) { return ld_coherent(p); }

// A sequence's rows of sums for 32 experts: counts, sums, and the losses' parts.  All WARPS of the
// block.
template <int WARPS>
struct Final {
  float sums[WARPS][32], squares[WARPS];
  int counts[WARPS][32], lives[WARPS];

  __device__ __forceinline__ void columns(const BalanceParams& p, int g, int column, int lane, int warp) {
    const int e = column * kBalanceColumns + lane;
    const int run = run_of(p.n, p.blocks), from = offset_at(p, g), to = offset_at(p, g + 1), words = 2 * p.experts + 2;
    // the blocks that have tokens of this sequence
    const int b0 = to > from ? from / run : 0, b1 = to > from ? (to - 1) / run + 1 : 0;
    float sum = 0.0f, square = 0.0f;
    int count = 0, live = 0;
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += WARPS) {
      const float* row = p.sums + (static_cast<int64_t>(b) + g) * words;
      if (e < p.experts) sum += ld(row + e), count += __float_as_int(ld(row + p.experts + e));
      live += __float_as_int(ld(row + 2 * p.experts));
      square += ld(row + 2 * p.experts + 1);
    }
    sums[warp][lane] = sum, counts[warp][lane] = count;
    if (lane == 0) lives[warp] = live, squares[warp] = square;
    __syncthreads();
    if (warp == 0) {
      sum = square = 0.0f, count = live = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += sums[w][lane], count += counts[w][lane], live += lives[w], square += squares[w];
      if (e < p.experts) {
        p.counts[static_cast<int64_t>(g) * p.experts + e] = count;
        p.prob_sums[static_cast<int64_t>(g) * p.experts + e] = sum;
      }
      const float share = live ? static_cast<float>(p.experts) / (static_cast<float>(p.topk) * p.sequences) / live / live : 0.0f;
      const float dot = warp_sum(e < p.experts ? static_cast<float>(count) * sum : 0.0f) * share;
      if (lane == 0) {
        const int columns = (p.experts + kBalanceColumns - 1) / kBalanceColumns;
        float* part = p.parts + 2 * (static_cast<int64_t>(g) * columns + column);
        part[0] = dot;
        part[1] = column ? 0.0f : square;
        if (column == 0) p.tokens[g] = live;
      }
    }
  }

  // The losses, from the parts of all sequences and columns.
  __device__ __forceinline__ void losses(const BalanceParams& p, int64_t parts, int lane, int warp) {
    float loss = 0.0f, z = 0.0f;
    int total = 0;
    for (int64_t i = threadIdx.x; i < parts; i += WARPS * 32) loss += ld(p.parts + 2 * i), z += ld(p.parts + 2 * i + 1);
    for (int i = threadIdx.x; i < p.sequences; i += WARPS * 32) total += ld_coherent(p.tokens + i);
    loss = warp_sum(loss);
    z = warp_sum(z);
    total = __reduce_add_sync(kAll, total);
    __syncthreads();
    if (lane == 0) sums[warp][0] = loss, squares[warp] = z, lives[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      loss = z = 0.0f, total = 0;
      for (int w = 0; w < WARPS; ++w) loss += sums[w][0], z += squares[w], total += lives[w];
      p.loss[0] = loss;
      p.loss[1] = total ? z / total : 0.0f;
      p.tokens[p.sequences] = total;
    }
  }
};

// ALONE: the only block and the only sequence; it writes the outputs itself.
template <class T, int V, bool VEC, bool SIGMOID, bool ALONE>
__global__ void __launch_bounds__(sum_warps(V) * 32) balance_sums_kernel(BalanceParams p) {
  constexpr int kWarps = sum_warps(V), U = at_once(V);
  extern __shared__ float shared[];                  // [kWarps][E] sums, [E] counts
  __shared__ float zz[kWarps];
  __shared__ int live_of[kWarps];
  allow_dependent_grids();
  int* cnt = reinterpret_cast<int*>(shared + kWarps * p.experts);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = run_of(p.n, p.blocks), start = static_cast<int>(blockIdx.x) * run, end = min(start + run, p.n);
  grid_dependency_wait();
  __shared__ int found[3];
  for (int at = start; at < end;) {
    if (warp == 0) {                         // one warp searches for all
      int from, to;
      const int g = sequence_of(p, at, lane, from, to);
      if (lane == 0) found[0] = g, found[1] = max(at, from), found[2] = min(end, to);
    }
    __syncthreads();
    const int g = found[0], from = found[1], to = found[2];
    if (g >= p.sequences) break;
    at = max(to, at + 1);
    __syncthreads();
    if (from >= to) continue;
    for (int e = threadIdx.x; e < p.experts; e += kWarps * 32) cnt[e] = 0;
    __syncthreads();
    float acc[V], squares = 0.0f;
    int live = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    // lane i has peak and whole of the warp's i-th live token, until 32 of them are there
    float my_peak = 0.0f, my_whole = 0.0f;
    const auto square = [&] {
      const float lse = lse_of(my_peak, my_whole);
      if (lse > -INFINITY) squares = fmaf(lse, lse, squares);
      my_whole = 0.0f;
    };
    const T* row = static_cast<const T*>(p.logits) + (from + warp) * p.row_stride;
    const int64_t* ids = p.idx + static_cast<int64_t>(from + warp) * p.topk + lane;
    const int64_t rows_on = kWarps * p.row_stride, ids_on = static_cast<int64_t>(kWarps) * p.topk;
    const bool chooses = lane < p.topk;
    for (int t = from + warp; t < to; t += U * kWarps) {
      float z[U][V], peak[U], whole[U];
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool there = u == 0 || t + u * kWarps < to;
        load_scores<T, V, VEC>(there ? row : static_cast<const T*>(p.logits), p.experts, lane, z[u]);
        id[u] = chooses && there ? id_of(p, ids) : -1;
        row += rows_on, ids += ids_on;
      }
      probabilities<U, V, SIGMOID, false>(z, z, z, peak, whole);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!__any_sync(kAll, id[u] >= 0)) continue;
        if (id[u] >= 0) atomicAdd(cnt + id[u], 1);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += z[u][v];
        if (lane == (live & 31)) my_peak = peak[u], my_whole = whole[u];
        if ((++live & 31) == 0) square();
      }
    }
    square();
    squares = warp_sum(squares);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = expert_of<VEC, V>(lane, v);
      if (j < p.experts) shared[warp * p.experts + j] = acc[v];
    }
    if (lane == 0) zz[warp] = squares, live_of[warp] = live;
    __syncthreads();
    float s = 0.0f;
    int k = 0;
    if (ALONE || threadIdx.x == 0)
      for (int w = 0; w < kWarps; ++w) s += zz[w], k += live_of[w];
    if constexpr (ALONE) {
      float dot = 0.0f;
      for (int e = threadIdx.x; e < p.experts; e += kWarps * 32) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += shared[w * p.experts + e];
        p.prob_sums[e] = sum;
        p.counts[e] = cnt[e];
        dot = fmaf(static_cast<float>(cnt[e]), sum, dot);
      }
      dot = warp_sum(dot);
      __syncthreads();                       // zz has been read
      if (lane == 0) zz[warp] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        dot = 0.0f;
        for (int w = 0; w < kWarps; ++w) dot += zz[w];
        p.tokens[0] = p.tokens[1] = k;
        p.loss[0] = k ? dot * (static_cast<float>(p.experts) / static_cast<float>(p.topk)) / k / k : 0.0f;
        p.loss[1] = k ? s / k : 0.0f;
      }
      return;
    }
    float* out = p.sums + (static_cast<int64_t>(blockIdx.x) + g) * (2 * p.experts + 2);
    for (int e = threadIdx.x; e < p.experts; e += kWarps * 32) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += shared[w * p.experts + e];
      out[e] = sum;
      out[p.experts + e] = __int_as_float(cnt[e]);
    }
    if (threadIdx.x == 0) out[2 * p.experts] = __int_as_float(k), out[2 * p.experts + 1] = s;
    __syncthreads();
  }
  if constexpr (ALONE) {                     // the sequence has no tokens
    for (int e = threadIdx.x; e < p.experts; e += kWarps * 32) p.prob_sums[e] = 0.0f, p.counts[e] = 0;
    if (threadIdx.x < 2) p.tokens[threadIdx.x] = 0, p.loss[threadIdx.x] = 0.0f;
  }
}

// grid: the column blocks of each sequence in turn
__global__ void __launch_bounds__(kFinalWarps * 32) balance_final_kernel(BalanceParams p) {
  __shared__ Final<kFinalWarps> f;
  __shared__ bool last;
  allow_dependent_grids();
  const int columns = (p.experts + kBalanceColumns - 1) / kBalanceColumns;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  f.columns(p, static_cast<int>(blockIdx.x) / columns, static_cast<int>(blockIdx.x) % columns, lane, warp);
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  f.losses(p, gridDim.x, lane, warp);
  if (threadIdx.x == 0) *p.ticket = 0;
}

template <class T, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kBackWarps * 32, V > 8 ? 1 : SIGMOID ? 4 : 6) balance_backward_kernel(BalanceParams p, int tokens) {
  constexpr int U = V <= 4 ? 2 : 1;          // more registers cost more than they bring (256 experts, two rows: 24 us, one: 20)
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int start = (blockIdx.x * kBackWarps + static_cast<int>(threadIdx.x >> 5)) * tokens;
  grid_dependency_wait();
  const int end = min(start + tokens, p.n);
  if (start >= end) return;
  const int total = p.tokens_in[p.sequences];
  const float gb = p.grad_loss[0], gz = total > 0 ? p.grad_loss[1] * 2.0f / total : 0.0f;
  for (int at = start, g, from, to; at < end && (g = sequence_of(p, at, lane, from, to)) < p.sequences;) {
    from = max(at, from), to = min(end, to);
    at = max(to, at + 1);
    if (from >= to) continue;
    const int tg = p.tokens_in[g];
    // sum p = 1, so any constant may be taken from the counts; their mean leaves the most bits
    const int mean = static_cast<int>(static_cast<int64_t>(tg) * p.topk / p.experts);
    const float share = tg > 0 ? gb * (static_cast<float>(p.experts) / (static_cast<float>(p.topk) * p.sequences)) / tg / tg : 0.0f;
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = expert_of<VEC, V>(lane, v);
      c[v] = j < p.experts ? static_cast<float>(p.counts_in[static_cast<int64_t>(g) * p.experts + j] - mean) : 0.0f;
    }
#pragma unroll 1
    for (int t = from; t < to; t += U) {
      float z[U][V], soft[SIGMOID ? U : 1][SIGMOID ? V : 1], not_s[SIGMOID ? U : 1][SIGMOID ? V : 1], peak[U], whole[U], dot[U];
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int mine = min(t + u, to - 1);
        load_scores<T, V, VEC>(static_cast<const T*>(p.logits) + mine * p.row_stride, p.experts, lane, z[u]);
        id[u] = lane < p.topk ? id_of(p, p.idx + static_cast<int64_t>(mine) * p.topk + lane) : -1;
      }
      probabilities<U, V, SIGMOID, true>(z, soft, not_s, peak, whole);
      // one logarithm for all of them: lane u's is the u-th's
      float my_lse = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (lane == u || U == 1) my_lse = whole[u];
      const float my_log = logf(my_lse);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) dot[u] = fmaf(c[v], z[u][v], dot[u]);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) dot[u] += __shfl_xor_sync(kAll, dot[u], d);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= to) break;
        const bool live = __any_sync(kAll, id[u] >= 0);
        if (!live && p.accumulate) continue;
        T* out = static_cast<T*>(p.grad) + (t + u) * p.grad_stride;
        // finite, as an infinite one would make the other scores' 0 a NaN
        const float lse = fminf(peak[u] + __shfl_sync(kAll, my_log, U == 1 ? 0 : u), 3e38f);
        const float rise = live && whole[u] > 0.0f ? gz * lse : 0.0f, part = live ? share : 0.0f;
        float d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float apart = c[v] - dot[u];
          if constexpr (SIGMOID)
            d[v] = fmaf(part * apart, z[u][v] * not_s[u][v], rise * soft[u][v]);
          else
            d[v] = z[u][v] * fmaf(part, apart, rise);
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
    }
  }
}

template <class... A, class... B>
cudaError_t launch_pdl(void (*kernel)(A...), unsigned grid, int warps, size_t smem, cudaStream_t s, const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  static const bool pdl = PdlEnabled();
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A>(args)...);
}

template <class T, int V, bool VEC, bool SIGMOID, bool ALONE>
cudaError_t launch_sums(const BalanceParams& p, cudaStream_t s) {
  const size_t smem = (sum_warps(V) + 1) * static_cast<size_t>(p.experts) * 4;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(balance_sums_kernel<T, V, VEC, SIGMOID, ALONE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(balance_sums_kernel<T, V, VEC, SIGMOID, ALONE>, p.blocks, sum_warps(V), smem, s, p);
}

template <class T, int V, bool VEC, bool SIGMOID>
cudaError_t launch_one(const BalanceParams& p, bool backward, cudaStream_t s) {
  if (backward) {
    // 32 warps an SM, and no more than 16 tokens each
    const int tokens = std::min(std::max(p.n / (32 * p.num_sms), 1), 16), per = kBackWarps * tokens;
    return launch_pdl(balance_backward_kernel<T, V, VEC, SIGMOID>, (p.n + per - 1) / per, kBackWarps, 0, s, p, tokens);
  }
  return BalanceAlone(p) ? launch_sums<T, V, VEC, SIGMOID, true>(p, s) : launch_sums<T, V, VEC, SIGMOID, false>(p, s);
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

// One block of the first kernel an SM up to 256 experts, and as many warps beyond; two rounds of
// its warps at least, unless that leaves a single block.
int BalanceBlocks(int n, int experts, int num_sms) {
  const int warps = experts <= 256 ? 32 : experts <= 512 ? 16 : 8;
  const int most = num_sms * (32 / warps), some = (n + 2 * warps - 1) / (2 * warps);
  return some < 1 ? 1 : some < most ? some : most;
}

cudaError_t LaunchBalance(const BalanceParams& p, cudaStream_t s) {
  if (p.n > 0)
    if (const cudaError_t e = p.bf16 ? launch<__nv_bfloat16>(p, false, s) : launch<float>(p, false, s);
        e != cudaSuccess || BalanceAlone(p))
      return e;
  return launch_pdl(balance_final_kernel, static_cast<unsigned>(BalancePartWords(p.sequences, p.experts) / 2), kFinalWarps, 0, s, p);
}

cudaError_t LaunchBalanceBackward(const BalanceParams& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  return p.bf16 ? launch<__nv_bfloat16>(p, true, s) : launch<float>(p, true, s);
}

}  // namespace epg
