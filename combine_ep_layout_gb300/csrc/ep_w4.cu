// ep_w4.cu -- products of a few activation rows with a 4-bit weight matrix
// (include/ep_gb300_moe.h: the form of the weights and the formula).
//
// Bound by reading the weights once, as long as turning nibbles into operands
// keeps up.  Two kernels, by the number of tokens:
//
//   narrow (up to 8 tokens)  a block of 8 warps takes 32 rows; its warps split
//       the columns chunk by chunk, each through its own cp.async ring
//       (ep_stream.cuh), and add their sums through shared memory.  Small tiles,
//       as a few MB of weights have to reach every SM at once; where there are more
//       than fit, a block goes on to the next tile with its rings full.
//   wide (9 to 64 tokens)    each of a block's 4 warps takes its own 16 rows and all
//       share a stage's activations, which would outweigh the weights if every
//       warp had its own.  Bound by the latency of making operands of nibbles and
//       of a stage's barrier, so the blocks are small and many.
//
// Where the rows give too few blocks, a cluster of blocks shares a tile: each
// takes its part of the columns, and the blocks' sums are added in rank order
// through distributed shared memory.  No order is left to chance.
//
// Measured one after the other in a graph, with weights that L2 does not hold, groups of
// 128 (bytes of the weights, of a copy's 6.8 TB/s): 7168 x 7168, 1 token 10.1 us (2.7 TB/s);
// 20011 x 4096, 1 and 8 tokens 14.4 and 14.8 us (3.0 TB/s); 4096 x 14336, 8, 16, 32 and 64
// tokens 11.3, 17.2, 22.9 and 33.1 us.  No unit is saturated (7168 x 7168: 50% of the issue
// slots while active, ALU 45%; 4096 x 14336, 32 tokens: 38%, 33%, tensor 30%): what is left is
// latency, the first 2.6 us of each that of the first loads.  mma.sync alone would take
// 4096 x 14336 6.2 us for 32 and 12.4 for 64 tokens.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ep_kernels.hpp"
#include "ep_moe_kernels.hpp"
#include "ep_stream.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

using stream::Form;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void store(const W4Params& p, int token, int row, float v) {
  const int64_t o = static_cast<int64_t>(token) * p.rows + row;
  if (p.out_f32)
    static_cast<float*>(p.out)[o] = v;
  else
    static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
}

// A tile's sums in shared memory: [column][row], 4 floats of padding a column, so
// that writing fragments and reading rows both miss each other's banks, and what
// another block of the cluster reads comes in whole 16 bytes (read 4 bytes at a
// time at strides, the remote reads took 30 us of a 70 us product).
template <int ROWS>
__device__ __forceinline__ int sum_at(int row, int col) { return col * (ROWS + 4) + row; }

// The sums of every block of the cluster, added in rank order and stored: each
// block finishes its share, four rows of a column at a time.
template <int ROWS, int THREADS>
__device__ __forceinline__ void finish(const W4Params& p, float* red, int cols, int row0, int part, int splits) {
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  if (splits > 1)
    cl.sync();
  else
    __syncthreads();
  for (int v = part * THREADS + threadIdx.x; v < ROWS / 4 * cols; v += splits * THREADS) {
    const int r = v % (ROWS / 4) * 4, col = v / (ROWS / 4), at = sum_at<ROWS>(r, col);
    if (row0 + r >= p.rows) continue;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b = 0; b < splits; ++b) {
      const float4 s = *reinterpret_cast<const float4*>((splits > 1 ? cl.map_shared_rank(red, b) : red) + at);
      sum.x += s.x, sum.y += s.y, sum.z += s.z, sum.w += s.w;
    }
    const float each[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row0 + r + i < p.rows) store(p, col, row0 + r + i, each[i]);
  }
  if (splits > 1) cl.sync();   // no block leaves while another reads its sums
}

// A warp's fragments into such a tile.
template <int ROWS, int RT, int NT>
__device__ __forceinline__ void put_sums(float* red, int row0, int lane, const float (&acc)[RT][NT][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[sum_at<ROWS>(row0 + 16 * rt + g + 8 * (i >> 1), 8 * nt + 2 * t + (i & 1))] = acc[rt][nt][i];
}

// ------------------------------------------------------------------ narrow

template <int G>
struct Narrow {
  static constexpr int kRowTiles = 2;
  using F = Form<G, kRowTiles>;
  static constexpr int kStages = 3;
  static constexpr int kFit = 2;                                 // blocks that fit together
  static constexpr int kWarpRed = 8 * (F::kRows + 4);            // floats of one warp's sums
  static constexpr int kRed = kWarps * kWarpRed * 4;
  // a slot holds n columns; what a product reads of the others past the last slot (and does
  // not use) are the sums
  static constexpr int slot(int n) { return F::kABytes + F::kSBytes + n * F::kXBytes; }
  static constexpr int bytes(int n) { return kWarps * kStages * slot(n) + kRed; }
  static_assert(kRed >= 8 * F::kXBytes);
};

template <int G>
__global__ void __launch_bounds__(kThreads, Narrow<G>::kFit) w4_narrow_kernel(const W4Params p, int splits) {
  using S = Narrow<G>;
  using F = typename S::F;
  constexpr int kStages = S::kStages, RT = S::kRowTiles, NT = 1;
  extern __shared__ __align__(128) uint8_t smem[];
  allow_dependent_grids();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x % splits;                               // the rank in the cluster
  const int tiles = (p.rows + F::kRows - 1) / F::kRows, at_once = gridDim.x / splits;
  const int pieces = p.cols / 32, chunks = (p.cols + F::kCols - 1) / F::kCols;
  const int step = kWarps * splits, c0 = part * kWarps + warp;
  const bool whole = p.cols % 128 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15) == 0;
  const uint32_t slot_bytes = F::kABytes + F::kSBytes + p.n * F::kXBytes;
  const uint32_t ring = stream::smem_addr(smem) + warp * kStages * slot_bytes;
  // where the copies stand: chunk c of tile `ahead`
  int ahead = blockIdx.x / splits, c = c0 < chunks ? c0 : chunks;
  auto row_of = [&](int r) { return min(ahead * F::kRows + r, p.rows - 1); };
  const int lane_row = lane / F::kPieces, lane_piece = lane % F::kPieces;
  const uint32_t a_dst = F::a_offset(lane_row, lane_piece);
  constexpr int kScaleCopies = (F::kRows + 31) / 32, kXCopies = 8 * NT * F::kXPieces / 32;
  const uint8_t* row_ptr[F::kCopies];
  const float* s_src[kScaleCopies];
  auto enter_tile = [&]() {
#pragma unroll
    for (int i = 0; i < F::kCopies; ++i)
      row_ptr[i] = p.q + static_cast<int64_t>(row_of(lane_row + i * (32 / F::kPieces))) * (p.cols / 2);
#pragma unroll
    for (int i = 0; i < kScaleCopies; ++i)
      s_src[i] = p.scales + static_cast<int64_t>(row_of(lane + 32 * i)) * (p.cols / G);
  };
  enter_tile();
  const int lane_col = lane / F::kXPieces, lane_xpiece = lane % F::kXPieces;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + static_cast<int64_t>(lane_col) * p.cols;
  auto issue = [&](uint32_t slot) {
    if (c < chunks && ahead < tiles) {
      const int piece = c * F::kPieces + lane_piece;
      const bool ok = piece < pieces;
      const int w_at = ok ? piece * 16 : 0;
#pragma unroll
      for (int i = 0; i < F::kCopies; ++i)
        stream::copy16(slot + a_dst + i * (32 / F::kPieces) * F::kRowBytes, row_ptr[i] + w_at, ok);
      if (whole) {
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
        if (col < p.n)
          stream::copy16(slot + F::x_offset(col, lane_xpiece),
                         x + static_cast<int64_t>(i * (32 / F::kXPieces)) * p.cols + x_at, at < p.cols);
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
  grid_dependency_wait();   // nothing of memory has been touched before this
  const uint32_t ring_bytes = kStages * slot_bytes;
  for (int s = 0; s < kStages - 1; ++s) issue(ring + s * slot_bytes);
  uint32_t in = (kStages - 1) * slot_bytes, out = 0;
  float* red = reinterpret_cast<float*>(smem + kWarps * ring_bytes);
  for (int tile = blockIdx.x / splits; tile < tiles; tile += at_once) {
    float acc[RT][NT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[rt][nt][i] = 0.0f;
    for (int k = c0; k < chunks; k += step) {
      stream::wait<kStages - 2>();
      __syncwarp();        // every lane's copies of this stage, and every lane done with the slot refilled next
      issue(ring + in);
      in = in + slot_bytes == ring_bytes ? 0 : in + slot_bytes;
      stream::consume<G, RT, NT, NT>(smem + warp * ring_bytes + out, lane, acc);
      out = out + slot_bytes == ring_bytes ? 0 : out + slot_bytes;
    }
    put_sums<F::kRows>(red + warp * S::kWarpRed, 0, lane, acc);
    __syncthreads();
    // each thread adds the 8 warps' sums of its values and keeps them in the first
    // warp's place, which nothing else reads
    for (int v = tid; v < F::kRows * p.n; v += kThreads) {
      float* at = red + sum_at<F::kRows>(v % F::kRows, v / F::kRows);
      float sum = *at;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) sum += at[w * S::kWarpRed];
      *at = sum;
    }
    finish<F::kRows, kThreads>(p, red, p.n, tile * F::kRows, part, splits);
    if (splits == 1) __syncthreads();   // the next tile's sums take the same place
  }
  stream::wait<0>();
}

// -------------------------------------------------------------------- wide

template <int G, int NT>
struct Wide {
  using F = Form<G, 1>;
  static constexpr int kWarps = 4, kThreads = 32 * kWarps;
  static constexpr int kWarpBytes = F::kABytes + F::kSBytes;     // a warp's own part of a stage
  static constexpr int kXAt = kWarps * kWarpBytes;
  static constexpr int kSlot = kXAt + 8 * NT * F::kXBytes;
  static constexpr int kStages = 4;
  // Blocks that fit together.  With 5 up to 16 tokens registers get scarce: of eleven
  // matrices, 13 tokens, groups of 64, six took 6 to 18% longer (7168 x 2048: 7.4 us, with 4
  // 6.4; 4096 x 14336: 17.8 and 15.1; 16384 x 2048: 11.4 and 9.9), four were up to 5% faster
  // (20011 x 4096: 20.1 and 21.1), with groups of 128 none differs by more than 2%.  Up to 32 tokens
  // 4096 x 14336 takes 23 us with 4 and 26 with 5 and a stage less.  64 tokens leave room for 2.
  static constexpr int kPerSm = NT == 8 ? 2 : 4;
  static constexpr int kRows = kWarps * F::kRows;
  static constexpr int kRed = 8 * NT * (kRows + 4) * 4;
  static constexpr int kBytes = kStages * kSlot > kRed ? kStages * kSlot : kRed;
};

template <int G, int NT>
__global__ void __launch_bounds__(Wide<G, NT>::kThreads, Wide<G, NT>::kPerSm) w4_wide_kernel(const W4Params p, int splits) {
  using S = Wide<G, NT>;
  using F = typename S::F;
  constexpr int kStages = S::kStages, kThreads = S::kThreads, RT = 1;
  extern __shared__ __align__(128) uint8_t smem[];
  allow_dependent_grids();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x / splits, part = blockIdx.x % splits;
  const int pieces = p.cols / 32, chunks = (p.cols + F::kCols - 1) / F::kCols;
  const bool whole = p.cols % 128 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15) == 0;
  const uint32_t base = stream::smem_addr(smem);
  auto row_of = [&](int r) { return min(tile * S::kRows + warp * F::kRows + r, p.rows - 1); };
  const int lane_row = lane / F::kPieces, lane_piece = lane % F::kPieces;
  const uint8_t* row_ptr[F::kCopies];
#pragma unroll
  for (int i = 0; i < F::kCopies; ++i)
    row_ptr[i] = p.q + static_cast<int64_t>(row_of(lane_row + i * (32 / F::kPieces))) * (p.cols / 2);
  const uint32_t a_dst = F::a_offset(lane_row, lane_piece);
  const float* s_src = p.scales + static_cast<int64_t>(row_of(lane)) * (p.cols / G);
  static_assert(F::kRows <= 32);
  constexpr int kXCopies = 8 * NT * F::kXPieces / kThreads;      // of each thread
  const int x_col = tid / F::kXPieces, x_piece = tid % F::kXPieces;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + static_cast<int64_t>(x_col) * p.cols;
  auto issue = [&](int c, uint32_t slot) {
    if (c < chunks) {
      const int piece = c * F::kPieces + lane_piece;
      const bool ok = piece < pieces;
      const int w_at = ok ? piece * 16 : 0;
      const uint32_t own = slot + warp * S::kWarpBytes;
#pragma unroll
      for (int i = 0; i < F::kCopies; ++i)
        stream::copy16(own + a_dst + i * (32 / F::kPieces) * F::kRowBytes, row_ptr[i] + w_at, ok);
      if (whole) {
        if (F::kRows >= 32 || lane < F::kRows)
          stream::copy_wide<4 * F::kScales>(own + F::kABytes + 4 * F::kScales * lane, s_src + c * F::kScales);
      } else {
        stream::copy_scales<G, RT>(own, lane, p.scales, p.cols, c, row_of);
      }
      const int at = c * F::kCols + 8 * x_piece;
      const int x_at = at < p.cols ? at : 0;
#pragma unroll
      for (int i = 0; i < kXCopies; ++i) {
        const int col = x_col + i * (kThreads / F::kXPieces);
        if (col < p.n)
          stream::copy16(slot + S::kXAt + F::x_at(col, x_piece),
                         x + static_cast<int64_t>(i * (kThreads / F::kXPieces)) * p.cols + x_at, at < p.cols);
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
  grid_dependency_wait();   // nothing of memory has been touched before this
  for (int s = 0; s < kStages - 1; ++s) issue(part + s * splits, base + s * S::kSlot);
  int in = kStages - 1, out = 0;
  for (int c = part; c < chunks; c += splits) {
    stream::wait<kStages - 2>();
    __syncthreads();       // every thread's copies of this stage, and every warp done with the slot refilled next
    issue(c + (kStages - 1) * splits, base + in * S::kSlot);
    in = in + 1 == kStages ? 0 : in + 1;
    const uint8_t* slot = smem + out * S::kSlot;
    stream::consume_at<G, RT, NT, NT>(slot + warp * S::kWarpBytes, slot + S::kXAt, lane, acc);
    out = out + 1 == kStages ? 0 : out + 1;
  }
  stream::wait<0>();
  __syncthreads();         // the ring's memory now holds the sums
  float* red = reinterpret_cast<float*>(smem);
  put_sums<S::kRows>(red, warp * F::kRows, lane, acc);
  finish<S::kRows, S::kThreads>(p, red, p.n, tile * S::kRows, part, splits);
}

// ------------------------------------------------------------------ launch

// How many blocks of a cluster share a tile: the cheapest by the time of its stages,
// one block's alone (`alone`, its latency) or all of an SM's blocks together
// (`together` each), in units of 10 ns.  A block's beginning and end cost as much as
// `ends` stages, a cluster 1 us more.  At most the 8 blocks that a cluster may always
// have.  Held against every number of blocks (1, 2, 4, 8) on eleven matrices from 512 x 1024
// to 20011 x 4096 with 1 to 64 tokens, groups of 128: the choice is the fastest or within 9%
// of it, but for 4096 x 4096 with up to 8 tokens (6.5 us, with two blocks 5.2), 1024 x 1024
// with 12 to 32 (3.6 and 3.0 with four) and 7168 x 2048 with 64 (14.3 and 11.8 with two); one
// block always takes up to 4.6 times as long (512 x 14336, 64 tokens).
int choose_splits(int sms, int tiles, int stages, int alone, int together, int ends) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= 8 && s <= stages; s *= 2) {
    const int64_t each = (stages + s - 1) / s + ends, per_sm = (static_cast<int64_t>(tiles) * s + sms - 1) / sms;
    int64_t cost = per_sm * together > alone ? per_sm * each * together : each * alone;
    if (s > 1) cost += 100;
    if (cost < least) least = cost, best = s;
  }
  return best;
}

// What the shape of a launch goes by, asked once for each device.
struct Gpu {
  int device, sms, smem_per_sm;
};
cudaError_t current_gpu(Gpu* g) {
  static std::atomic<uint64_t> known[64];   // by device: SMs and bytes of an SM, 0: not asked yet
  if (const cudaError_t e = cudaGetDevice(&g->device); e != cudaSuccess) return e;
  if (g->device < 64) {
    if (const uint64_t v = known[g->device].load(std::memory_order_relaxed); v != 0) {
      g->sms = static_cast<int>(v >> 32), g->smem_per_sm = static_cast<int>(v & 0xffffffffu);
      return cudaSuccess;
    }
  }
  if (const cudaError_t e = cudaDeviceGetAttribute(&g->sms, cudaDevAttrMultiProcessorCount, g->device); e != cudaSuccess) return e;
  if (const cudaError_t e = cudaDeviceGetAttribute(&g->smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, g->device);
      e != cudaSuccess)
    return e;
  if (g->device < 64)
    known[g->device].store(static_cast<uint64_t>(g->sms) << 32 | static_cast<uint32_t>(g->smem_per_sm), std::memory_order_relaxed);
  return cudaSuccess;
}

template <class K>
cudaError_t launch(K kernel, std::atomic<uint64_t>& ready, int dev, const W4Params& p, int tiles, int splits, int threads,
                   int most_bytes, int bytes, cudaStream_t s) {
  // the kernel's shared-memory limit is raised once on each device
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) & bit)) {
    if (const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_bytes);
        e != cudaSuccess)
      return e;
    if (dev < 64) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * static_cast<unsigned>(splits));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
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
  return cudaLaunchKernelEx(&cfg, kernel, p, splits);
}

template <int G>
cudaError_t launch_narrow(const W4Params& p, cudaStream_t s) {
  using S = Narrow<G>;
  static std::atomic<uint64_t> ready{0};
  const int tiles = (p.rows + S::F::kRows - 1) / S::F::kRows, chunks = (p.cols + 127) / 128;
  Gpu gpu;
  if (const cudaError_t e = current_gpu(&gpu); e != cudaSuccess) return e;
  const int splits = choose_splits(gpu.sms, tiles, (chunks + kWarps - 1) / kWarps, 60, 40, 3);
  // as many tiles at once as the blocks that fit together can take
  const int by_bytes = gpu.smem_per_sm / (S::bytes(p.n) + 1024);
  const int blocks = gpu.sms * (by_bytes < S::kFit ? by_bytes : S::kFit), most = blocks > splits ? blocks / splits : 1;
  return launch(w4_narrow_kernel<G>, ready, gpu.device, p, tiles < most ? tiles : most, splits, kThreads, S::bytes(8), S::bytes(p.n), s);
}

template <int G, int NT>
cudaError_t launch_wide(const W4Params& p, cudaStream_t s) {
  using S = Wide<G, NT>;
  static std::atomic<uint64_t> ready{0};
  const int tiles = (p.rows + S::kRows - 1) / S::kRows, chunks = (p.cols + 127) / 128;
  Gpu gpu;
  if (const cudaError_t e = current_gpu(&gpu); e != cudaSuccess) return e;
  return launch(w4_wide_kernel<G, NT>, ready, gpu.device, p, tiles, choose_splits(gpu.sms, tiles, chunks, 90, 12 + 4 * NT, 4),
                S::kThreads, S::kBytes, S::kBytes, s);
}

// Where narrow and wide meet: with 8 tokens narrow is the faster one on all of eleven
// matrices (4096 x 14336: 11.3 us, wide 16.9; 20011 x 4096: 14.8 and 19.4).  A narrow kernel
// with two column tiles, which is not built, won with 13 tokens on nine (4096 x 14336: 13.5
// and 17.1; 20011 x 4096: 18.3 and 19.6), with 16 it lost on the large ones (20011 x 4096:
// 23.2 and 19.6).
template <int G>
cudaError_t launch_g(const W4Params& p, cudaStream_t s) {
  if (p.n <= 8) return launch_narrow<G>(p, s);
  if (p.n <= 16) return launch_wide<G, 2>(p, s);
  if (p.n <= 32) return launch_wide<G, 4>(p, s);
  return launch_wide<G, 8>(p, s);
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
