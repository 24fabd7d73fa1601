// ep_moe.cu -- the experts of a few tokens (include/ep_gb300_moe.h: ep_moe_forward).
//
// Two kernels: a warp per (token, choice, intermediate channel) for the gated
// product, then a warp per (token, output channel) that folds the K choices.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_moe_kernels.hpp"
#include "ep_types.cuh"
#include "ep_w4.cuh"

namespace epg {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float activate(float g, int act) {
  if (act == 0) return g / (1.0f + expf(-g));
  const float u = 0.7978845608028654f * (g + 0.044715f * g * g * g);
  return 0.5f * g * (1.0f + tanhf(u));
}

__device__ __forceinline__ float row_dot(const void* w, const float* scales, int64_t row, int cols, int group,
                                         const __nv_bfloat16* x, int lane) {
  return group ? w4_row_dot(static_cast<const uint8_t*>(w), scales, row, cols, group, x, lane)
               : bf16_row_dot(static_cast<const __nv_bfloat16*>(w), row, cols, x, lane);
}

__global__ void __launch_bounds__(kWarps * 32) gate_up_kernel(MoeParams p) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int entry = blockIdx.y;
  const int64_t e = p.topk_idx[entry];
  if (e < 0 || e >= p.experts) {
    if (e != -1 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrBadExpert);
    return;
  }
  if (i >= p.inter) return;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + static_cast<int64_t>(entry / p.topk) * p.hidden;
  const float g = row_dot(p.w13, p.w13_scales, e * 2 * p.inter + i, p.hidden, p.group, x, lane);
  const float u = row_dot(p.w13, p.w13_scales, (e * 2 + 1) * p.inter + i, p.hidden, p.group, x, lane);
  if (lane == 0)
    static_cast<__nv_bfloat16*>(p.h)[static_cast<int64_t>(entry) * p.inter + i] =
        __float2bfloat16_rn(activate(g, p.act) * u);
}

__global__ void __launch_bounds__(kWarps * 32) down_kernel(MoeParams p) {
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = blockIdx.y;
  if (c >= p.hidden) return;
  float acc = 0.0f;
  for (int k = 0; k < p.topk; ++k) {
    const int entry = t * p.topk + k;
    const int64_t e = p.topk_idx[entry];
    if (e < 0 || e >= p.experts) continue;
    const float v = row_dot(p.w2, p.w2_scales, e * p.hidden + c, p.inter, p.group,
                            static_cast<const __nv_bfloat16*>(p.h) + static_cast<int64_t>(entry) * p.inter, lane);
    acc = fmaf(p.topk_weights[entry], v, acc);
  }
  if (lane == 0) {
    const int64_t o = static_cast<int64_t>(t) * p.hidden + c;
    if (p.bias) acc += __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[o]);
    if (p.out_f32)
      static_cast<float*>(p.out)[o] = acc;
    else
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(acc);
  }
}

}  // namespace

cudaError_t LaunchMoe(const MoeParams& p, int, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  gate_up_kernel<<<dim3(static_cast<unsigned>((p.inter + kWarps - 1) / kWarps), static_cast<unsigned>(p.n * p.topk)),
                   kWarps * 32, 0, s>>>(p);
  down_kernel<<<dim3(static_cast<unsigned>((p.hidden + kWarps - 1) / kWarps), static_cast<unsigned>(p.n)),
                kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace epg
