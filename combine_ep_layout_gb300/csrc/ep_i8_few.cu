// ep_i8_few.cu -- the dense int8 product of a few tokens (include/ep_gb300_i8.h states
// the formulas).
//
// Bound by reading the weights once.  A block of 8 warps takes 32 weight rows (gated: 16 gate rows and
// their 16 up rows); its warps split the columns 128 at a time, each through its own
// cp.async ring, from a warp to itself: no barrier before the sums, no wait that
// could hang.  Integer mma.sync needs no conversion and its sums are exact, so their
// order does not matter; it does 261 multiply-adds a cycle and SM (a 16th of what fp16 tcgen05
// does), half of which is reached here.  The widening kernel (ep_i8_product.cu) takes over where that costs
// more than its own ends.  Where the rows give too few
// blocks, a cluster of blocks shares a tile's columns.  A block goes on to its next tile with its
// rings full.
//
// Measured, us, this kernel and the widening one: 7168 x 7168, 1 token 12.7 and 17.9, 8 tokens 13.9 and
// 18.8, 16 tokens 23.3 and 18.8; 2048 x 7168, 16 tokens 10.6 and 19.0; 20011 x 4096, 1 token
// 16.7 and 25.4, 16 tokens 34.6 and 25.4.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "ep_gb300_i8.h"
#include "ep_i8_act.cuh"
#include "ep_i8_kernels.hpp"
#include "ep_kernels.hpp"
#include "ep_stream.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kStages = 3;
constexpr int kTileRows = 32, kCols = 128, kWeightBytes = kTileRows * kCols;
constexpr int kPitch = kTileRows + 4;           // of a column of sums

constexpr int slot_bytes(int columns) { return kWeightBytes + columns * kCols; }
constexpr int sum_bytes(int nc) { return kWarps * 8 * nc * kPitch * 4; }
// What a product reads of columns that are not there lies in the next slot, or past the last one in the sums.
constexpr int smem_bytes(int nc, int n) { return kWarps * kStages * slot_bytes(n) + std::max(sum_bytes(nc), 8 * nc * kCols); }

// Where 16-byte piece c of row r lies: the rows that a quarter of the reading lanes touch fall on different banks.
__device__ __forceinline__ uint32_t place(int r, int c) { return static_cast<uint32_t>(r * kCols + 16 * (c ^ ((r & 1) << 2))); }

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NC: column tiles of 8 tokens.
template <bool GATED, int NC>
__global__ void __launch_bounds__(kThreads, 2) i8_few_kernel(const I8ProductParams p, int splits) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(128) uint8_t smem[];
  allow_dependent_grids();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = static_cast<int>(p.n);
  const int part = blockIdx.x % splits;         // the rank in the cluster
  const int channels = GATED ? p.rows / 2 : p.rows, per = GATED ? kTileRows / 2 : kTileRows;
  const int tiles = (channels + per - 1) / per, at_once = gridDim.x / splits;
  const int chunks = (p.cols + kCols - 1) / kCols, step = kWarps * splits, c0 = part * kWarps + warp;
  const uint32_t slot = slot_bytes(n), ring_bytes = kStages * slot;
  const uint8_t* ring = smem + warp * ring_bytes;
  const uint32_t ring_at = stream::smem_addr(ring);
  // where the copies stand: chunk c of tile `ahead`; a lane copies piece lane % 8 of every fourth row
  int ahead = blockIdx.x / splits, c = c0 < chunks ? c0 : chunks;
  const int piece = lane % 8, row0 = lane / 8;
  const int8_t* from[kTileRows / 4];
  auto enter_tile = [&] {
#pragma unroll
    for (int i = 0; i < kTileRows / 4; ++i) {
      const int r = row0 + 4 * i;
      const int channel = min(ahead * per + (GATED ? r % per : r), channels - 1);
      from[i] = p.w + static_cast<int64_t>(GATED && r >= per ? channels + channel : channel) * p.cols;
    }
  };
  enter_tile();
  auto issue = [&](uint32_t to) {
    if (c < chunks && ahead < tiles) {
      const int at = c * kCols + 16 * piece;
      const bool ok = at < p.cols;
      const int in = ok ? at : 0;
#pragma unroll
      for (int i = 0; i < kTileRows / 4; ++i) stream::copy16(to + place(row0 + 4 * i, piece), from[i] + in, ok);
#pragma unroll
      for (int i = 0; i < 2 * NC; ++i) {
        const int t = row0 + 4 * i;
        if (t < n) stream::copy16(to + kWeightBytes + place(t, piece), p.x + static_cast<int64_t>(t) * p.cols + in, ok);
      }
      c += step;
      if (c >= chunks) {
        c = c0;
        ahead += at_once;
        if (ahead < tiles) enter_tile();
      }
    }
    stream::commit();
  };
  grid_dependency_wait();                       // nothing of memory has been touched before this
  for (int s = 0; s < kStages - 1; ++s) issue(ring_at + s * slot);
  uint32_t in = (kStages - 1) * slot, out = 0;
  int* sums = reinterpret_cast<int*>(smem + kWarps * ring_bytes);       // [warp][column][row]
  const int g = lane >> 2, t = lane & 3;
  for (int tile = blockIdx.x / splits; tile < tiles; tile += at_once) {
    int acc[2][NC][4] = {};
    for (int k = c0; k < chunks; k += step) {
      stream::wait<kStages - 2>();
      __syncwarp();                             // every lane's copies of this stage, and every lane done with the slot refilled next
      issue(ring_at + in);
      in = in + slot == ring_bytes ? 0 : in + slot;
      const uint8_t* w = ring + out;
      const uint8_t* x = w + kWeightBytes;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint4 b[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) b[j] = stream::load16(x + place(8 * j + g, 4 * kk + t));
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          // a lane's 16 columns of two rows: a product over k may take k in any order that both operands share
          const uint4 lo = stream::load16(w + place(16 * rt + g, 4 * kk + t)), hi = stream::load16(w + place(16 * rt + g + 8, 4 * kk + t));
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            mma_s8(acc[rt][j], lo.x, hi.x, lo.y, hi.y, b[j].x, b[j].y);
            mma_s8(acc[rt][j], lo.z, hi.z, lo.w, hi.w, b[j].z, b[j].w);
          }
        }
      }
      out = out + slot == ring_bytes ? 0 : out + slot;
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sums[(warp * 8 * NC + 8 * j + 2 * t + (i & 1)) * kPitch + 16 * rt + g + 8 * (i >> 1)] = acc[rt][j][i];
    __syncthreads();
    // each thread adds the 8 warps' sums of its values and keeps them in the first warp's place, which nothing else reads
    for (int v = tid; v < kTileRows * n; v += kThreads) {
      int* at = sums + v / kTileRows * kPitch + v % kTileRows;
      int sum = *at;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) sum += at[w * 8 * NC * kPitch];
      *at = sum;
    }
    if (splits > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
    // each block of the cluster finishes its share
    for (int v = part * kThreads + tid; v < per * n; v += splits * kThreads) {
      const int r = v % per, token = v / per, channel = tile * per + r;
      if (channel >= channels) continue;
      int own = 0, up = 0;
      for (int b = 0; b < splits; ++b) {
        const int* s = (splits > 1 ? cg::this_cluster().map_shared_rank(sums, b) : sums) + token * kPitch + r;
        own += s[0];
        if (GATED) up += s[per];
      }
      const float xs = ld_coherent(p.x_scales + token);
      float y = static_cast<float>(own) * ld_coherent(p.w_scales + channel) * xs;
      if (GATED) y = i8_activate(p.act, y) * (static_cast<float>(up) * ld_coherent(p.w_scales + channels + channel) * xs);
      const int64_t at = static_cast<int64_t>(token) * channels + channel;
      if (p.out_f32)
        static_cast<float*>(p.out)[at] = y;
      else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    }
    // the next tile's sums take the same place, and no block leaves while another reads its sums
    if (splits > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  }
  stream::wait<0>();
}

template <bool GATED, int NC>
cudaError_t launch(const I8ProductParams& p, int device, int sms, cudaStream_t s) {
  // the kernel's shared-memory limit is raised once on each device
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (device & 63);
  if (device >= 64 || !(ready.load(std::memory_order_relaxed) & bit)) {
    if (const cudaError_t e = cudaFuncSetAttribute(i8_few_kernel<GATED, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(NC, 8 * NC));
        e != cudaSuccess)
      return e;
    if (device < 64) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int bytes = smem_bytes(NC, static_cast<int>(p.n));
  const int fit = std::min(2, 232448 / (bytes + 1024)), per = GATED ? kTileRows / 2 : kTileRows;
  const int channels = GATED ? p.rows / 2 : p.rows, tiles = (channels + per - 1) / per;
  const int stages = (p.cols + kCols * kWarps - 1) / (kCols * kWarps);
  // a tile's columns are shared as long as that fills SMs and leaves each warp two stages
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= sms * fit && stages >= 4 * splits) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(tiles, std::max(1, sms * fit / splits)) * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  static const bool pdl = PdlEnabled();
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (splits > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, i8_few_kernel<GATED, NC>, p, splits);
}

}  // namespace

cudaError_t LaunchI8Few(const I8ProductParams& p, int device, int sms, cudaStream_t s) {
  const int nc = static_cast<int>(p.n + 7) / 8;
  if (p.act != EP_ACT_NONE)
    return nc == 1 ? launch<true, 1>(p, device, sms, s) : nc == 2 ? launch<true, 2>(p, device, sms, s) : launch<true, 3>(p, device, sms, s);
  return nc == 1 ? launch<false, 1>(p, device, sms, s) : nc == 2 ? launch<false, 2>(p, device, sms, s) : launch<false, 3>(p, device, sms, s);
}

}  // namespace epg
