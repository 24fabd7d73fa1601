// ep_w4.cuh -- row products of the weight forms of the decode-side MoE operators.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace epg {

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// sum over the columns of row `row` of a 4-bit matrix times x, in every lane.
__device__ __forceinline__ float w4_row_dot(const uint8_t* q, const float* scales, int64_t row, int cols,
                                            int group, const __nv_bfloat16* x, int lane) {
  float acc = 0.0f;
  const uint8_t* qr = q + row * (cols / 2);
  const float* sr = scales + row * (cols / group);
  for (int c = lane * 32; c < cols; c += 32 * 32) {
    const uint4 v = *reinterpret_cast<const uint4*>(qr + c / 2);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float f = static_cast<float>(static_cast<int>((w[i / 8] >> (4 * (i % 8))) & 15u) - 8);
      sum = fmaf(f, __bfloat162float(x[c + i]), sum);
    }
    acc = fmaf(sum, sr[c / group], acc);
  }
  return warp_total(acc);
}

// the same for a bf16 matrix
__device__ __forceinline__ float bf16_row_dot(const __nv_bfloat16* w, int64_t row, int cols,
                                              const __nv_bfloat16* x, int lane) {
  float acc = 0.0f;
  const __nv_bfloat16* wr = w + row * cols;
  for (int c = lane * 8; c < cols; c += 32 * 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(wr + c);
    const uint4 b = *reinterpret_cast<const uint4*>(x + c);
    const __nv_bfloat16* ae = reinterpret_cast<const __nv_bfloat16*>(&a);
    const __nv_bfloat16* be = reinterpret_cast<const __nv_bfloat16*>(&b);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(__bfloat162float(ae[i]), __bfloat162float(be[i]), acc);
  }
  return warp_total(acc);
}

}  // namespace epg
