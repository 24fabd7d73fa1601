// ep_w4.cu -- products of a few activation rows with a 4-bit weight matrix
// (include/ep_gb300_moe.h: the form of the weights and the formula).
//
// Bound by reading the weights once.  A block of 8 warps takes a tile of 16 RT
// rows; its warps split the columns chunk by chunk, each through its own
// cp.async ring (ep_stream.cuh), and add their sums through shared memory.
// Where the rows give too few blocks, a cluster of blocks shares a tile: each
// takes its part of the columns, and the blocks' sums are added in rank order
// through distributed shared memory.  No order is left to chance.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_moe_kernels.hpp"
#include "ep_stream.cuh"

namespace epg {
namespace {

using stream::Form;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

template <int G, int RT, int NT>
struct Shape {
  using F = Form<G, RT>;
  static constexpr int kSlot = F::stage_bytes(NT);
  static constexpr int kStages = 3;
  static constexpr int kRing = kWarps * kStages * kSlot;
  static constexpr int kRedRow = 8 * NT + 2;                     // floats of a row of one warp's sums
  static constexpr int kRed = kWarps * F::kRows * kRedRow * 4;
  static constexpr int kBytes = kRing > kRed ? kRing : kRed;     // the sums come after the ring's last use
};

template <int G, int RT, int NT>
__global__ void __launch_bounds__(kThreads) w4_kernel(const W4Params p, int splits) {
  using F = Form<G, RT>;
  using S = Shape<G, RT, NT>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x / splits, part = blockIdx.x % splits;   // part: the rank in the cluster
  const int t0 = blockIdx.y * 8 * NT, cols = min(8 * NT, p.n - t0);
  const int pieces = p.cols / 32, chunks = (p.cols + F::kCols - 1) / F::kCols;
  const int step = kWarps * splits, c0 = part * kWarps + warp;
  const bool wide = p.cols % 128 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15) == 0;
  const uint32_t ring = stream::smem_addr(smem) + warp * kStages * S::kSlot;
  auto row_of = [&](int r) { return min(tile * F::kRows + r, p.rows - 1); };
  const int lane_row = lane / F::kPieces, lane_piece = lane % F::kPieces;
  const uint8_t* row_ptr[F::kCopies];
#pragma unroll
  for (int i = 0; i < F::kCopies; ++i)
    row_ptr[i] = p.q + static_cast<int64_t>(row_of(lane_row + i * (32 / F::kPieces))) * (p.cols / 2);
  const uint32_t a_dst = F::a_offset(lane_row, lane_piece);
  constexpr int kScaleCopies = (F::kRows + 31) / 32, kXCopies = 8 * NT * F::kXPieces / 32;
  const float* s_src[kScaleCopies];
#pragma unroll
  for (int i = 0; i < kScaleCopies; ++i)
    s_src[i] = p.scales + static_cast<int64_t>(row_of(lane + 32 * i)) * (p.cols / G);
  const int lane_col = lane / F::kXPieces, lane_xpiece = lane % F::kXPieces;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + static_cast<int64_t>(t0 + lane_col) * p.cols;
  auto issue = [&](int c, uint32_t slot) {
    if (c < chunks) {
      const int piece = c * F::kPieces + lane_piece;
      const bool ok = piece < pieces;
      const int w_at = ok ? piece * 16 : 0;
#pragma unroll
      for (int i = 0; i < F::kCopies; ++i)
        stream::copy16(slot + a_dst + i * (32 / F::kPieces) * F::kRowBytes, row_ptr[i] + w_at, ok);
      if (wide) {
#pragma unroll
        for (int i = 0; i < kScaleCopies; ++i)
          if (F::kRows >= 32 || lane < F::kRows)
            stream::copy_wide<4 * F::kScales>(slot + F::kABytes + 4 * F::kScales * (lane + 32 * i), s_src[i] + c * F::kScales);
      } else {
        stream::copy_scales<G, RT>(slot, lane, p.scales, p.cols, c, row_of);
      }
      const int at = c * F::kCols + 8 * lane_xpiece;
      const int x_at = at < p.cols ? at : 0;
#pragma unroll
      for (int i = 0; i < kXCopies; ++i) {
        const int col = lane_col + i * (32 / F::kXPieces);
        if (col < cols)
          stream::copy16(slot + F::x_offset(col, lane_xpiece),
                         x + static_cast<int64_t>(i * (32 / F::kXPieces)) * p.cols + x_at, at < p.cols);
      }
    }
    stream::commit();
  };
  float acc[RT][NT][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[rt][nt][i] = 0.0f;
  for (int s = 0; s < kStages - 1; ++s) issue(c0 + s * step, ring + s * S::kSlot);
  int in = kStages - 1, out = 0;
  for (int c = c0; c < chunks; c += step) {
    stream::wait<kStages - 2>();
    __syncwarp();          // every lane's copies of this stage, and every lane done with the slot refilled next
    issue(c + (kStages - 1) * step, ring + in * S::kSlot);
    in = in + 1 == kStages ? 0 : in + 1;
    stream::consume<G, RT, NT, NT>(ring + out * S::kSlot, lane, acc);
    out = out + 1 == kStages ? 0 : out + 1;
  }
  stream::wait<0>();
  __syncthreads();         // the rings' memory now holds the sums
  float* red = reinterpret_cast<float*>(smem);
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float* r0 = red + (warp * F::kRows + 16 * rt + g) * S::kRedRow + 8 * nt + 2 * t;
      *reinterpret_cast<float2*>(r0) = make_float2(acc[rt][nt][0], acc[rt][nt][1]);
      *reinterpret_cast<float2*>(r0 + 8 * S::kRedRow) = make_float2(acc[rt][nt][2], acc[rt][nt][3]);
    }
  __syncthreads();
  // each thread adds the 8 warps' sums of its values and keeps them in the first
  // warp's place, which nothing else reads
  for (int v = tid; v < F::kRows * cols; v += kThreads) {
    float* at = red + (v / cols) * S::kRedRow + v % cols;
    float sum = *at;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += at[w * F::kRows * S::kRedRow];
    *at = sum;
  }
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  if (splits > 1)
    cl.sync();
  else
    __syncthreads();
  // each block of the cluster finishes its share of the tile's values
  for (int v = part * kThreads + tid; v < F::kRows * cols; v += splits * kThreads) {
    const int r = v % F::kRows, col = v / F::kRows;
    const int row = tile * F::kRows + r;
    if (row >= p.rows) continue;
    float sum = red[r * S::kRedRow + col];
    if (splits > 1) {
      sum = 0.0f;
      for (int b = 0; b < splits; ++b) sum += cl.map_shared_rank(red, b)[r * S::kRedRow + col];
    }
    const int64_t o = static_cast<int64_t>(t0 + col) * p.rows + row;
    if (p.out_f32)
      static_cast<float*>(p.out)[o] = sum;
    else
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(sum);
  }
  if (splits > 1) cl.sync();   // no block leaves while another reads its sums
}

template <int G, int RT, int NT>
cudaError_t launch(const W4Params& p, int splits, cudaStream_t s) {
  using S = Shape<G, RT, NT>;
  auto kernel = w4_kernel<G, RT, NT>;
  if (const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
      e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  const int tiles = (p.rows + 16 * RT - 1) / (16 * RT);
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), static_cast<unsigned>((p.n + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, splits);
}

template <int G>
cudaError_t launch_g(const W4Params& p, cudaStream_t s) {
  const int rt = p.n <= 2 ? 1 : p.n <= 4 ? 2 : 4;
  const int tiles = (p.rows + 16 * rt - 1) / (16 * rt);
  const int chunks = (p.cols + 127) / 128;
  int splits = 1;
  while (splits < 8 && tiles * splits < 2 * 152 && chunks >= 2 * 8 * splits) splits *= 2;
  if (rt == 1) return launch<G, 1, 1>(p, splits, s);
  if (rt == 2) return launch<G, 2, 1>(p, splits, s);
  if (p.n <= 8) return launch<G, 4, 1>(p, splits, s);
  return launch<G, 4, 2>(p, splits, s);
}

}  // namespace

cudaError_t LaunchW4(const W4Params& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  switch (p.group) {
    case 32: return launch_g<32>(p, s);
    case 64: return launch_g<64>(p, s);
    default: return launch_g<128>(p, s);
  }
}

}  // namespace epg
