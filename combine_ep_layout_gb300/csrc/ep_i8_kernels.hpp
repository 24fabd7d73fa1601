// ep_i8_kernels.hpp -- host-side interface between the C ABI of the int8 path
// (ep_i8_api.cpp, include/ep_gb300_i8.h) and its kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace epg {

struct I8RowsParams {
  const void* x;             // [rows, cols], rows row_stride elements apart
  int64_t row_stride;
  int64_t rows;              // (dispatch: tokens)
  int cols;
  bool bf16;
  int8_t* q;                 // [rows or rcap, cols]
  float* scales;
  // dispatch: the receive rows of each token, topk entries, -1 for none; else null
  const int32_t* slots;
  int topk;
  // quantising receive rows: how many there are and which receive something
  // (meta[row * meta_stride] >= 0); else null
  const int32_t* num_recv;
  const int32_t* meta;
  int meta_stride;
};

cudaError_t LaunchI8Rows(const I8RowsParams& p, cudaStream_t s);

struct I8ProductParams {
  const int8_t* x;           // [n, cols] (grouped: [rcap, cols])
  const float* x_scales;
  const int8_t* w;           // [E, rows, cols]
  const float* w_scales;     // [E, rows]
  void* out;                 // [n or rcap, rows], gated: [., rows / 2]
  int64_t n;                 // rows of x
  int rows, cols;
  int act;                   // EP_ACT_NONE: plain
  bool out_f32;
  // grouped: expert e's rows of x are [first[e], first[e] + count[e]); else null and E = 1
  const int32_t* first;
  const int32_t* count;
  int experts;
  int64_t entries;           // grouped: most rows that the experts can have together
  uint64_t wait_ns;          // bound of one wait on a barrier
};

cudaError_t LaunchI8Product(const I8ProductParams& p, cudaStream_t s);
// Dense products of up to kI8FewTokens tokens, where LaunchI8Product finds that cheaper.
constexpr int kI8FewTokens = 24;
cudaError_t LaunchI8Few(const I8ProductParams& p, int device, int sms, cudaStream_t s);
// Read and clear the current device's error word of the products, in order on s.
cudaError_t ReadI8Error(int32_t* value, cudaStream_t s);

}  // namespace epg
