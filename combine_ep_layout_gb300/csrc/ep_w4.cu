// ep_w4.cu -- products of a few activation rows with a 4-bit weight matrix
// (include/ep_gb300_moe.h: the form of the weights and the formula).
//
// One warp per output row and token: each lane takes 32 columns (16 bytes) at
// a time, whole inside one group, and the lanes' sums are added at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_moe_kernels.hpp"
#include "ep_w4.cuh"

namespace epg {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) w4_kernel(W4Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = blockIdx.y;
  if (row >= p.rows) return;
  const float acc = w4_row_dot(p.q, p.scales, row, p.cols, p.group,
                               static_cast<const __nv_bfloat16*>(p.x) + static_cast<int64_t>(t) * p.cols, lane);
  if (lane == 0) {
    const int64_t o = static_cast<int64_t>(t) * p.rows + row;
    if (p.out_f32)
      static_cast<float*>(p.out)[o] = acc;
    else
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(acc);
  }
}

}  // namespace

cudaError_t LaunchW4(const W4Params& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  w4_kernel<<<dim3(static_cast<unsigned>((p.rows + kWarps - 1) / kWarps), static_cast<unsigned>(p.n)),
              kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace epg
