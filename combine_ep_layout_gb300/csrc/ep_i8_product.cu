// ep_i8_product.cu -- products of int8 rows with int8 weights, dense and grouped by
// expert (include/ep_gb300_i8.h states the formulas).
//
// The simple form: a block of 256 threads takes 64 weight rows (gated: 32 gate rows and
// their 32 up rows) and 64 rows of x, both staged in shared memory 64 columns at a
// time, and adds four products an instruction (dp4a), exactly.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_gb300_i8.h"
#include "ep_i8_kernels.hpp"
#include "ep_kernels.hpp"
#include "ep_types.cuh"

namespace epg {
namespace {

__device__ int32_t g_error;

constexpr int kTile = 64, kStep = 64, kPitch = kStep / 4 + 1;

__device__ __forceinline__ float activate(int act, float v) {
  if (act == EP_ACT_SILU) return v / (1.0f + expf(-v));
  return 0.5f * v * (1.0f + tanhf(0.7978845608028654f * (v + 0.044715f * v * v * v)));
}

__global__ void __launch_bounds__(256) i8_simple_kernel(I8ProductParams p) {
  __shared__ int ws[kTile][kPitch], xs[kTile][kPitch];
  const int e = blockIdx.z, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const bool gated = p.act != EP_ACT_NONE;
  const int half = p.rows / 2, out_rows = gated ? half : p.rows;
  const int64_t first = p.first ? p.first[e] : 0, n = p.first ? p.count[e] : p.n;
  // tile row i of this block's weights
  auto weight_row = [&](int i) {
    if (!gated) return static_cast<int>(blockIdx.x) * kTile + i;
    const int r = static_cast<int>(blockIdx.x) * (kTile / 2) + i / 2;
    return r < half ? (i & 1 ? half + r : r) : p.rows;
  };
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * kTile; t0 < n; t0 += static_cast<int64_t>(gridDim.y) * kTile) {
    int acc[4][4] = {};
    for (int c0 = 0; c0 < p.cols; c0 += kStep) {
      __syncthreads();
      const int i = threadIdx.x / 4, c = c0 + threadIdx.x % 4 * 16, wr = weight_row(i);
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (wr < p.rows && c < p.cols) a = *reinterpret_cast<const uint4*>(p.w + (static_cast<int64_t>(e) * p.rows + wr) * p.cols + c);
      if (t0 + i < n && c < p.cols) b = *reinterpret_cast<const uint4*>(p.x + (first + t0 + i) * p.cols + c);
      int* w = &ws[i][threadIdx.x % 4 * 4];
      int* x = &xs[i][threadIdx.x % 4 * 4];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      x[0] = b.x, x[1] = b.y, x[2] = b.z, x[3] = b.w;
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kStep / 4; ++k) {
        int u[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = ws[4 * tx + j][k], v[j] = xs[4 * ty + j][k];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int l = 0; l < 4; ++l) acc[j][l] = __dp4a(u[l], v[j], acc[j][l]);
      }
    }
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + 4 * ty + j;
      if (t >= n) continue;
      const float s = p.x_scales[first + t];
      auto value = [&](int l) {
        const int r = weight_row(4 * tx + l);
        return r < p.rows ? static_cast<float>(acc[j][l]) * p.w_scales[static_cast<int64_t>(e) * p.rows + r] * s : 0.0f;
      };
      auto store = [&](int r, float y) {
        const int64_t at = (first + t) * out_rows + r;
        if (p.out_f32)
          static_cast<float*>(p.out)[at] = y;
        else
          static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
      };
      for (int l = 0; l < 4; ++l) {
        const int r = weight_row(4 * tx + l);
        if (!gated && r < p.rows) store(r, value(l));
        if (gated && !(l & 1) && r < half) store(r, activate(p.act, value(l)) * value(l + 1));
      }
    }
  }
}

}  // namespace

cudaError_t LaunchI8Product(const I8ProductParams& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  const int out_rows = p.act == EP_ACT_NONE ? p.rows : p.rows / 2, per = p.act == EP_ACT_NONE ? kTile : kTile / 2;
  const int64_t tiles = (p.n + kTile - 1) / kTile;
  const dim3 grid((out_rows + per - 1) / per, static_cast<unsigned>(p.first ? 4 : tiles < 4096 ? tiles : 4096), p.experts);
  i8_simple_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t ReadI8Error(int32_t* value, cudaStream_t s) {
  int32_t zero = 0;
  if (const cudaError_t e = cudaMemcpyFromSymbolAsync(value, g_error, sizeof zero, 0, cudaMemcpyDeviceToHost, s); e != cudaSuccess) return e;
  if (const cudaError_t e = cudaMemcpyToSymbolAsync(g_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s); e != cudaSuccess) return e;
  return cudaStreamSynchronize(s);
}

}  // namespace epg
