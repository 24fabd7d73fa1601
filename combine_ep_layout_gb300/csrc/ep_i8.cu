// ep_i8.cu -- rows to int8 with one scale each, in place of their tokens or to the
// receive rows of a layout (include/ep_gb300_i8.h states the formulas).
//
// Bound by reading the rows once and writing what comes of them.  A group of
// threads holds a row in registers, 16 values each (32 where rows have more than 8192), between the search
// of its largest magnitude and the rounding, so that x is read once; rows of more than 16384 columns are read a second time, out
// of L2.  The magnitude is searched as an unsigned integer, where infinities and NaNs
// are above every number.
//
// Measured: 4096 x 7168 bf16 to 8 receive rows each 47.1 us (6.2 TB/s, 92% of a copy's rate); 1001 x 14336
// fp32 in place 15.7 us (4.6 TB/s: two rows an SM at a time, each load, search, barrier, store).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ep_i8_kernels.hpp"
#include "ep_kernels.hpp"
#include "ep_rows.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kVec = 16;      // columns of one vector: 16 bytes of int8

// 16 values of a row as floats.
template <class T, bool ALIGNED>
__device__ __forceinline__ void load16(const T* at, float (&v)[kVec]) {
  if constexpr (ALIGNED) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kVec; i += kPer) {
      const uint4 q = *reinterpret_cast<const uint4*>(at + i);
      const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[i + j] = rows::as_float(e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = rows::as_float(at[i]);
  }
}

__device__ __forceinline__ unsigned magnitude(const float (&v)[kVec]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// x / s rounded to the nearest integer, ties to even, four to a word.  x inv is off the
// quotient (as fp32 rounds it) by less than 127 (2^-23 + 2^-24) < 2.3e-5, so where it is
// further than 3e-5 from the middle of two integers both round alike; the others are
// divided.  inv is no use where s is (nearly) subnormal.
__device__ __forceinline__ uint4 round16(const float (&v)[kVec], float s, float inv) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer in the low bits
  float r[kVec], off = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const float t = v[i] * inv;
    r[i] = t + kMagic;
    off = fmaxf(off, fabsf(t - (r[i] - kMagic)));
  }
  if (!(off < 0.5f - 3e-5f) || !(s > 1e-30f)) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) r[i] = s > 0.0f ? fminf(fmaxf(__fdiv_rn(v[i], s), -127.0f), 127.0f) + kMagic : kMagic;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __byte_perm(__float_as_uint(r[4 * i]), __float_as_uint(r[4 * i + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(r[4 * i + 2]), __float_as_uint(r[4 * i + 3]), 0x0040);
    w[i] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// How the columns lie among a row's threads.  kTogether: 16 consecutive ones a thread, whose int8 are one store;
// kSpread (in place): four times 4 fp32 or twice 8 bf16, G threads side by side, so that a load's 32 lanes read
// 512 bytes in a row (1001 x 14336: 15.6 us, together 21.4).  kSingle: as kTogether, value by value (not 16-byte aligned).
enum Lie { kTogether, kSpread, kSingle };

// G threads a row, 128 / G rows a block where G is below 128.
template <class T, int G, int MINE, Lie LIE>
__global__ void __launch_bounds__(G < 128 ? 128 : G, (MINE == 1 ? 1536 : 1024) / (G < 128 ? 128 : G)) i8_rows_kernel(I8RowsParams p) {
  constexpr int kThreads = G < 128 ? 128 : G, kRows = kThreads / G, kPer = 16 / sizeof(T);
  constexpr bool kMore = MINE == 2;           // rows may have more vectors than the threads hold
  __shared__ unsigned most[2][kThreads / 32];
  allow_dependent_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = threadIdx.x / G, at = threadIdx.x % G;
  const int vectors = p.cols / kVec;
  grid_dependency_wait();
  const int64_t rows = p.num_recv ? ld_coherent(p.num_recv) : p.rows;
  int turn = 0;
  // uniform trip counts: a block's threads meet at the barrier of every turn
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
    const int64_t row = r0 + group;
    const bool ok = row < rows && (!p.meta || ld_coherent(p.meta + row * p.meta_stride) >= 0);
    const T* x = static_cast<const T*>(p.x) + row * p.row_stride;
    // lane k: the k-th row that this one goes to
    int slot = -1;
    if (p.slots && ok && lane < p.topk) slot = ld_coherent(p.slots + row * p.topk + lane);
    // this thread's part of the row's c-th G vectors
    auto load = [&](int c, float(&a)[kVec]) {
      if constexpr (LIE == kSpread) {
#pragma unroll
        for (int i = 0; i < kVec / kPer; ++i) {
          const int col = 16 * G * c + kPer * G * i + kPer * at;
          uint4 f = make_uint4(0, 0, 0, 0);
          if (ok && col < p.cols) f = *reinterpret_cast<const uint4*>(x + col);
          const T* e = reinterpret_cast<const T*>(&f);
#pragma unroll
          for (int j = 0; j < kPer; ++j) a[kPer * i + j] = rows::as_float(e[j]);
        }
      } else if (ok && c * G + at < vectors) {
        load16<T, LIE == kTogether>(x + static_cast<int64_t>(c * G + at) * kVec, a);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) a[i] = 0.0f;
      }
    };
    float v[MINE][kVec];
    unsigned m = 0;
#pragma unroll
    for (int u = 0; u < MINE; ++u) load(u, v[u]);
#pragma unroll
    for (int u = 0; u < MINE; ++u) m = max(m, magnitude(v[u]));
    if constexpr (kMore)
      for (int c = MINE; c * G < vectors; ++c) {
        float more[kVec];
        load(c, more);
        m = max(m, magnitude(more));
      }
    m = __reduce_max_sync(kAll, m);
    if constexpr (G > 32) {
      if (lane == 0) most[turn][warp] = m;
      __syncthreads();
      m = __reduce_max_sync(kAll, lane < G / 32 ? most[turn][group * (G / 32) + lane] : 0u);
    }
    if (!ok) continue;                         // the same for a whole warp
    const bool fine = m < 0x7f800000u;
    const float s = fine ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(0x7fc00000u);
    const float inv = fine ? 1.0f / s : 0.0f;
    auto store = [&](int c, const float(&a)[kVec]) {
      const int vector = c * G + at;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (fine) q = round16(a, s, inv);
      int8_t* to = p.q + static_cast<int64_t>(vector) * kVec;
      if constexpr (LIE == kSpread) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < kVec / kPer; ++i) {
          const int col = 16 * G * c + kPer * G * i + kPer * at;
          if (col >= p.cols) continue;
          if constexpr (kPer == 4)
            *reinterpret_cast<uint32_t*>(p.q + row * p.cols + col) = w[i];
          else
            *reinterpret_cast<uint2*>(p.q + row * p.cols + col) = make_uint2(w[2 * i], w[2 * i + 1]);
        }
      } else if (!p.slots) {
        if (vector < vectors) *reinterpret_cast<uint4*>(to + row * p.cols) = q;
      } else {
        for (int k = 0; k < p.topk; ++k) {
          const int d = __shfl_sync(kAll, slot, k);
          if (d >= 0 && vector < vectors) *reinterpret_cast<uint4*>(to + static_cast<int64_t>(d) * p.cols) = q;
        }
      }
    };
#pragma unroll
    for (int u = 0; u < MINE; ++u) store(u, v[u]);
    if constexpr (kMore)
      for (int c = MINE; c * G < vectors; ++c) {
        float more[kVec];
        load(c, more);
        store(c, more);
      }
    if (!p.slots) {
      if (at == 0) p.scales[row] = s;
    } else if (at < 32 && slot >= 0) {
      p.scales[slot] = s;
    }
  }
}

template <class T, int G, int MINE = 1>
cudaError_t launch_g(const I8RowsParams& p, cudaStream_t s) {
  constexpr int kThreads = G < 128 ? 128 : G, kRows = kThreads / G;
  const bool vec = rows::aligned16(p.x, p.row_stride * static_cast<int64_t>(sizeof(T)));
  const int64_t blocks = std::min<int64_t>((p.rows + kRows - 1) / kRows, p.num_recv ? 4096 : 1 << 24);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  static const bool pdl = PdlEnabled();
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (!vec) return cudaLaunchKernelEx(&cfg, i8_rows_kernel<T, G, MINE, kSingle>, p);
  if (!p.slots) return cudaLaunchKernelEx(&cfg, i8_rows_kernel<T, G, MINE, kSpread>, p);
  return cudaLaunchKernelEx(&cfg, i8_rows_kernel<T, G, MINE, kTogether>, p);
}

template <class T>
cudaError_t launch(const I8RowsParams& p, cudaStream_t s) {
  const int vectors = p.cols / kVec;
  if (vectors <= 32) return launch_g<T, 32>(p, s);
  if (vectors <= 64) return launch_g<T, 64>(p, s);
  if (vectors <= 128) return launch_g<T, 128>(p, s);
  if (vectors <= 256) return launch_g<T, 256>(p, s);
  if (vectors <= 512) return launch_g<T, 512>(p, s);
  return launch_g<T, 512, 2>(p, s);
}

}  // namespace

cudaError_t LaunchI8Rows(const I8RowsParams& p, cudaStream_t s) {
  if (p.rows == 0) return cudaSuccess;
  return p.bf16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace epg
