// ep_i8_product.cu -- products of int8 rows with int8 weights, dense and grouped by
// expert (include/ep_gb300_i8.h states the formulas).
//
// sm_103a has no integer tcgen05, and dp4a and integer mma.sync do 76 T multiply-adds a
// second.  fp16 holds every int8 exactly and the 16-bit tensor cores do twelve times as
// many, with products that are exact and fp32 sums that are exact below 2^24.  So both operands are
// widened on the way: int8 travels from HBM and through L2 by TMA, and warps of the
// multiplying SM turn it into fp16.
//
// A pair of CTAs takes 256 weight rows (128 each) and up to NT rows of x.  The weights
// are the operand in tensor memory, where their fp16 form costs shared memory neither a write
// nor a read; x is the operand in shared memory, each CTA widening half of it.  With the
// weights along the 256 rows of the instruction, the number of tokens of a tile is free (a multiple of
// 32), which experts with few tokens need.  Roles of a CTA's 28 warps:
//   0       TMA loads of both operands, a ring of 128 columns a stage
//   1       (first CTA) issues the products
//   2       tensor memory
//   4-19    widen, in groups that take the stages in turn, as a stage's latency (reads, fence,
//           tensor memory, barriers) is a multiple of its work: 32 weight rows a warp, and a share of x
//   20-27   sums times scales, activation, output; up to 128 tokens the sums are double
//           buffered, so that this runs beside the next tile
// A CTA's rows are two half tiles of up to 64, in the lanes from 0 and from 64 on: gated, the
// second half is the up rows of the first, and the warps that hold them swap halves through
// shared memory.  Where rows are few, half tiles are smaller, so that every SM has some.
//
// Measured: 8192 x 7168 x 7168 451 us (1.87 PFLOP/s, 97% of the library's bf16 rate; the tensor cores 87% of
// their cycles at 2048 tokens), where the products of a stage, 8 x 137 cycles, are what bounds it; 64 tokens over 64
// experts of 7168 x 4096, gated, top-8, 270 us (7.0 TB/s of weights); 8192 tokens over 128 experts of 4096 x 2816,
// gated, top-6, 823 us (1.38 PFLOP/s: tiles of 192 tokens, whose stages shared memory bounds, and their ends); 45 x
// 20011 x 4096 27.4 us (a stage's latency, 650 cycles for 330 of products).  A fetch of the next tile's
// rows hides behind the rings; the ends of a tile do not where its sums are not double buffered.
//
// Every wait is bounded.  A warp that gives up records it, marks its CTA and leaves; the
// others of the pair give up by the mark or by their own limit, and all meet before the
// tensor memory is freed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>

#include "ep_gb300_i8.h"
#include "ep_i8_act.cuh"
#include "ep_i8_kernels.hpp"
#include "ep_i8_mma.cuh"
#include "ep_kernels.hpp"
#include "ep_types.cuh"

namespace epg {
namespace {

__device__ int32_t g_error;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWideners = 16, kOfQuad = 2, kWriters = 4 * kOfQuad;   // warps; writing ones of 32 lanes of tensor memory
constexpr int kFirstWriter = 4 + kWideners, kThreads = 32 * (kFirstWriter + kWriters);
constexpr int kRows = 128;                 // weight rows of a CTA
constexpr int kStep = 128;                 // columns of a stage
constexpr int kColumnsA = kStep / 2;       // tensor memory columns of a stage's weights
constexpr uint32_t kTmem = 512;
constexpr int kMaxShared = 232448 - 1024 - 64;   // less what aligning the buffers may take, and static data

// Groups of widening warps that take the stages in turn, and widened stages: as many as tensor memory
// holds beside the sums, and shared memory, up to 6.  Up to 128 tokens a stage's latency counts for more than
// its work: 4 groups (gated 333 x 11008 x 4096: 32 us, with 2 groups 35; 45 x 20011 x 4096: 28.6 and 31.6).
__host__ __device__ constexpr int groups(int nt) { return nt <= 128 ? 4 : 2; }
__host__ __device__ constexpr int stages_out(int nt) { return nt == 256 ? 3 : nt == 128 ? 4 : 6; }
__host__ __device__ constexpr int sums(int nt) { return nt == 256 ? 1 : 2; }         // sum buffers
__host__ __device__ constexpr int bytes_in(int nt) { return kRows * kStep + nt / 2 * kStep; }
__host__ __device__ constexpr int bytes_out(int nt) { return nt / 2 * kStep * 2; }
// Rows of x come in boxes of 32, as many as the tile has.  Widening 256 tokens' rows for 192 took as long as 256
// tokens do: shared memory moves 128 bytes a cycle and a stage needs 112 KB of it (copies, reads, widened writes,
// and what the products read), 1000 cycles where the products of 192 tokens take 840.
__host__ __device__ constexpr int x_box(int nt) { return nt / 2 < 32 ? nt / 2 : 32; }
constexpr int kSwap = 16 * 32 * 4;         // what a writing warp hands over, or 32 tokens of its output
constexpr int kBarBytes = 592;             // and 16 words: a stage's rows of x
constexpr int kScaleBytes = (8 + kOfQuad - 1) / kOfQuad * 32 * 4;    // a writing warp's scales of x
constexpr int kFixed = kWriters * kSwap + kWriters * kScaleBytes + kBarBytes;

struct Args {
  I8ProductParams p;
  int steps;         // stages of a tile
  int part;          // weight rows of a CTA's half tile: a multiple of 8 up to 64
  int row_tiles;     // pair tiles along the weight rows
  int stages_in;
  CUtensorMap w, x;
};

struct Tile {
  int expert, row_tile;
  int first;         // row of x
  int tokens;        // rows of x that count
  int width;         // columns of the product: a multiple of 32
};

// Expert e's rows go to the fewest tiles, of (nearly) one size each.
__host__ __device__ __forceinline__ int token_tiles(int64_t count, int nt) { return static_cast<int>((count + nt - 1) / nt); }

// A role's way through its pair's tiles, in ascending order.
template <int NT>
struct Tiles {
  const Args& a;
  const int* starts;
  int expert = 0;

  __device__ __forceinline__ Tile operator()(int tile) {
    Tile t;
    int first = 0, count = static_cast<int>(a.p.n);
    if (a.p.first) {
      while (starts[expert + 1] <= tile) ++expert;
      tile -= starts[expert];
      first = ld_coherent(a.p.first + expert);
      count = ld_coherent(a.p.count + expert);
    }
    const unsigned tiles = token_tiles(count, NT), at = static_cast<unsigned>(tile) / static_cast<unsigned>(a.row_tiles);
    const int per = static_cast<int>((count + tiles - 1) / tiles + 31) / 32 * 32;
    t.expert = expert;
    t.row_tile = tile - static_cast<int>(at) * a.row_tiles;
    t.first = first + static_cast<int>(at) * per;
    t.tokens = min(per, count - static_cast<int>(at) * per);
    t.width = (t.tokens + 31) / 32 * 32;
    return t;
  }
};

// Waits of one CTA: false, and the CTA marked, when the limit has passed or the mark is there.
struct Waits {
  volatile int* dead;
  uint64_t limit;

  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (limit == 0 ? tma::mbar_test(bar, parity) : pair::try_wait(bar, parity)) return true;
    if (limit != 0) {
      const uint64_t t0 = tma::global_ns();
      do {
        if (*dead) return false;
        if (pair::try_wait(bar, parity)) return true;
      } while (tma::global_ns() - t0 <= limit);
    }
    *dead = 1;
    atomicOr(&g_error, kErrTimeout);
    return false;
  }
};

// Four int8 as fp16: offset by 128 a byte is the low byte of 1024 + it, less 1152.
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi) {
  v ^= 0x80808080u;
  const __half2 base = __half2half2(__ushort_as_half(0x6480));
  const uint32_t l = __byte_perm(v, 0x64646464u, 0x4140), h = __byte_perm(v, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), base), b = __hsub2(*reinterpret_cast<const __half2*>(&h), base);
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 read16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void write16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A warp's 8 N tokens of 32 channels, as fragments: y[h][i][e] is channel 16 h + lane / 4 + 8 (e / 2) of
// token 8 i + 2 (lane % 4) + e % 2.  `many` tokens and `channels` channels count.  bf16: turned by
// stmatrix through 64 bytes a token at `stage`, and written as 16-byte pieces where the output's rows allow them.
template <int N>
__device__ __forceinline__ void store_tile(const I8ProductParams& p, bool wide, uint32_t stage, int lane, int64_t at, int pitch, int many,
                                           int channels, const float (&y)[2][N][4]) {
  if (p.out_f32) {
    float* out = static_cast<float*>(p.out) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int token = 8 * i + 2 * (lane & 3) + e;
        float* row = out + static_cast<int64_t>(token) * pitch + (lane >> 2);
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (token < many && 8 * g + (lane >> 2) < channels) row[8 * g] = y[g >> 1][i][2 * (g & 1) + e];
      }
    return;
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + at;
  // piece (8 channels) g of a token lies at place g ^ (token / 2 % 4): no two of a store on the same banks
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t v[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(y[g >> 1][i][2 * (g & 1)], y[g >> 1][i][2 * (g & 1) + 1]);
      v[g] = *reinterpret_cast<const uint32_t*>(&two);
    }
    pair::store_transposed(stage + 64 * (8 * i + (lane & 7)) + 16 * ((lane >> 3) ^ ((lane >> 1) & 3)), v[0], v[1], v[2], v[3]);
  }
  __syncwarp();
  if (wide) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int token = 8 * i + lane / 4, piece = lane % 4;
      const uint4 v = read16(stage + 64 * token + 16 * (piece ^ ((token >> 1) & 3)));
      if (token < many && 8 * piece < channels) *reinterpret_cast<uint4*>(out + static_cast<int64_t>(token) * pitch + 8 * piece) = v;
    }
  } else if (lane < channels) {
    for (int j = 0; j < 8 * N && j < many; ++j, out += pitch) {
      uint16_t v;
      asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(stage + 64 * j + 16 * ((lane >> 3) ^ ((j >> 1) & 3)) + 2 * (lane & 7)) : "memory");
      out[lane] = __ushort_as_bfloat16(v);
    }
  }
  __syncwarp();
}

template <int NT, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) i8_mma_kernel(const __grid_constant__ Args a) {
  constexpr int kTok = NT / 2, kIn = bytes_in(NT), kOut = bytes_out(NT), kS2 = stages_out(NT), kD = sums(NT);
  constexpr int kGroups = groups(NT), kOfStage = kWideners / kGroups;      // warps of a stage
  static_assert(kS2 >= kGroups && kD * NT + kS2 * kColumnsA <= static_cast<int>(kTmem));
  constexpr uint32_t kSumColumns = kD * NT;
  constexpr int kBox = x_box(NT);
  extern __shared__ uint8_t raw[];
  __shared__ int dead;
  __shared__ uint32_t tmem_at;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kAll, static_cast<int>(threadIdx.x >> 5), 0), s1 = a.stages_in;
  const uint32_t cta = pair::rank();
  const uint32_t base = (tma::smem_u32(raw) + 1023) & ~1023u;
  const uint32_t out0 = base + s1 * kIn, swap0 = out0 + kS2 * kOut, xs0 = swap0 + kWriters * kSwap, bars = xs0 + kWriters * kScaleBytes;
  int* starts = reinterpret_cast<int*>(raw + (bars + kBarBytes - tma::smem_u32(raw)));
  // barriers: s1 (at most 16) full, empty of the int8 ring; kS2 full, empty of the widened one; sums
  // full, empty; swaps ready, done; end
  const auto full_in = [&](int s) { return bars + 8 * s; };
  const auto empty_in = [&](int s) { return bars + 128 + 8 * s; };
  const auto full_out = [&](int s) { return bars + 256 + 8 * s; };
  const auto empty_out = [&](int s) { return bars + 304 + 8 * s; };
  const auto full_sum = [&](int s) { return bars + 352 + 8 * s; };
  const auto empty_sum = [&](int s) { return bars + 368 + 8 * s; };
  const auto swap_ready = [&](int s) { return bars + 384 + 8 * s; };
  const auto swap_done = [&](int s) { return bars + 448 + 8 * s; };
  const uint32_t end_bar = bars + 512;
  const auto x_rows = [&](int s) { return bars + 528 + 4 * s; };   // rows of x in a stage of the int8 ring

  if (threadIdx.x == 0) {
    dead = 0;
    for (int s = 0; s < s1; ++s) tma::mbar_init(full_in(s), 1), tma::mbar_init(empty_in(s), kOfStage);
    for (int s = 0; s < kS2; ++s) tma::mbar_init(full_out(s), 2 * kOfStage), tma::mbar_init(empty_out(s), 1);
    for (int s = 0; s < kD; ++s) tma::mbar_init(full_sum(s), 1), tma::mbar_init(empty_sum(s), 2 * kWriters);
    for (int s = 0; s < kWriters; ++s) tma::mbar_init(swap_ready(s), 1), tma::mbar_init(swap_done(s), 1);
    tma::mbar_init(end_bar, 1);
    tma::mbar_init_fence();
    pair::prefetch_map(&a.w);
    pair::prefetch_map(&a.x);
  }
  if (warp == 2) {
    pair::alloc(tma::smem_u32(&tmem_at), kTmem);
    pair::relinquish();
  }
  allow_dependent_grids();
  grid_dependency_wait();
  int total;
  if (a.p.first) {
    // each expert's first tile, by a scan of warp 3's
    if (warp == 3) {
      int sum = 0;
      for (int e0 = 0; e0 < a.p.experts; e0 += 32) {
        const int e = e0 + lane;
        const int mine = e < a.p.experts ? token_tiles(ld_coherent(a.p.count + e), NT) * a.row_tiles : 0;
        int up = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(kAll, up, d);
          if (lane >= d) up += v;
        }
        if (e < a.p.experts) starts[e] = sum + up - mine;
        sum += __shfl_sync(kAll, up, 31);
      }
      if (lane == 0) starts[a.p.experts] = sum;
    }
  }
  pair::fence_before();
  __syncthreads();
  pair::cluster_sync();
  pair::fence_after();
  total = a.p.first ? starts[a.p.experts] : token_tiles(a.p.n, NT) * a.row_tiles;
  const uint32_t tmem = *const_cast<volatile uint32_t*>(&tmem_at);
  const Waits wait{&dead, a.p.wait_ns};
  const int pairs = static_cast<int>(gridDim.x) / 2, first_tile = static_cast<int>(blockIdx.x) / 2;
  const int half = a.p.rows / 2;
  Tiles<NT> tile_of{a, starts};

  if (warp == 0) {
    // as for the products, the whole warp goes along and one elected lane issues
    const bool one = pair::elect();
    int in = 0;
    uint32_t turn = 0, copies = 0;
    bool ok = true;
    for (int tile = first_tile; ok && tile < total; tile += pairs) {
      const Tile t = tile_of(tile);
      const int lead = (2 * t.row_tile + static_cast<int>(cta)) * (GATED ? a.part : 2 * a.part);
      const int y0 = t.expert * a.p.rows + lead, y1 = y0 + (GATED ? half : a.part);
      const int yx = t.first + static_cast<int>(cta) * (t.width / 2), boxes = (t.width / 2 + kBox - 1) / kBox;
      const uint32_t bytes = (2 * a.part + boxes * kBox) * kStep;
      for (int k = 0; k < a.steps; ++k) {
        if (!(ok = __all_sync(kAll, wait(empty_in(in), turn ^ 1)))) break;
        if (one) {
          const uint32_t at = base + in * kIn, bar = full_in(in);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(x_rows(in)), "r"(boxes * kBox) : "memory");
          tma::mbar_expect_tx(bar, bytes);
          pair::load_box(at, &a.w, k * kStep, y0, bar);
          pair::load_box(at + kRows / 2 * kStep, &a.w, k * kStep, y1, bar);
#pragma unroll
          for (int i = 0; i < kTok / kBox; ++i)
            if (i < boxes) pair::load_box(at + (kRows + i * kBox) * kStep, &a.x, k * kStep, yx + i * kBox, bar);
        }
        __syncwarp();
        copies = min(copies + 1, static_cast<uint32_t>(s1));
        if (++in == s1) in = 0, turn ^= 1;
      }
    }
    // the copies in flight land before the block ends
    for (; copies != 0; --copies) {
      if (--in < 0) in = s1 - 1, turn ^= 1;
      tma::mbar_wait_bounded(full_in(in), turn, tma::kDrainNs);
    }
  } else if (warp == 1) {
    if (cta == 0) {
      // the whole warp goes along, and one lane that the compiler knows to be one issues: the operands
      // stay in uniform registers (27 cycles a product of 32 tokens, 136 of 256; by `lane == 0` 94 at least)
      const bool one = pair::elect();
      int stage = 0, buf = 0;
      uint32_t stage_turn = 0, buf_turn = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < total; tile += pairs) {
        const Tile t = tile_of(tile);
        const uint32_t d = tmem + buf * NT, shape = pair::shape_f16(t.width);
        if (!(ok = __all_sync(kAll, wait(empty_sum(buf), buf_turn ^ 1)))) break;
        pair::fence_after();
        for (int k = 0; k < a.steps; ++k) {
          if (!(ok = __all_sync(kAll, wait(full_out(stage), stage_turn)))) break;
          pair::fence_after();
          const int parts = min(kStep, a.p.cols - k * kStep) / 16;
          const uint32_t at = tmem + kSumColumns + stage * kColumnsA;
          const uint64_t b = pair::operand(out0 + stage * kOut);
          if (one) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < parts) pair::mma(d, at + 8 * i, b + (((i >> 2) * (kTok * 128) + (i & 3) * 32) >> 4), shape, k + i != 0);
            pair::commit(empty_out(stage));
          }
          __syncwarp();
          if (++stage == kS2) stage = 0, stage_turn ^= 1;
        }
        if (ok && one) pair::commit(full_sum(buf));
        __syncwarp();
        if (++buf == kD) buf = 0, buf_turn ^= 1;
      }
      if (one) pair::commit(end_bar);
      __syncwarp();
    }
  } else if (warp >= 4 && warp < kFirstWriter) {
    const int w = (warp - 4) % kOfStage, group = (warp - 4) / kOfStage, quad = w & 3, part = w >> 2, row = 32 * quad + lane;
    constexpr int kMineA = 32 / kOfStage;      // 16-column chunks of a row of w that a thread widens
    constexpr int kRowParts = 32 * kOfStage / kTok, kMine = kRowParts < 8 ? 8 / kRowParts : 1;   // threads of a row of x, its chunks of a thread
    const int thread = 32 * w + lane, xrow = thread % kTok, xpart = thread / kTok;
    const bool has_rows = a.part > 32 * (quad & 1);
    const uint32_t to = tmem + (static_cast<uint32_t>(32 * quad) << 16) + kSumColumns + part * 8 * kMineA;
    const uint32_t from_a = base + row * kStep, from_x = base + kRows * kStep + xrow * kStep;
    const uint32_t to_x = out0 + xrow * 128;
    // the group's stage of either ring, and the parity of its turn there
    int in = group, out = group;
    uint32_t in_turn = 0, out_turn = 0;
    const int64_t all = first_tile < total ? static_cast<int64_t>((total - first_tile + pairs - 1) / pairs) * a.steps : 0;
    bool ok = true;
    for (int64_t it = group; it < all; it += kGroups) {
      // Where the int8 ring has a number of stages that the groups do not divide, they take turns on
      // each of them, and a parity alone cannot tell the copy meant from the one before: so the one before
      // has to have been read.
      ok = __all_sync(kAll, wait(empty_in(in), in_turn ^ 1) && wait(full_in(in), in_turn));
      if (!ok) break;
      uint32_t there;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(there) : "r"(x_rows(in)) : "memory");
      const bool has_x = xpart < 8 && xrow < static_cast<int>(there);
      uint4 va[kMineA], vx[kMine];
      if (has_rows)
#pragma unroll
      for (int c = 0; c < kMineA; ++c) va[c] = read16(from_a + in * kIn + (((kMineA * part + c) ^ (row & 7)) << 4));
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (has_x) vx[i] = read16(from_x + in * kIn + (((xpart + i * kRowParts) ^ (xrow & 7)) << 4));
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(empty_in(in));
      ok = __all_sync(kAll, wait(empty_out(out), out_turn ^ 1));
      if (!ok) break;
      pair::fence_after();
      if (has_rows)
#pragma unroll
      for (int c = 0; c < kMineA; c += 2) {
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          widen(va[c + i].x, r[8 * i], r[8 * i + 1]);
          widen(va[c + i].y, r[8 * i + 2], r[8 * i + 3]);
          widen(va[c + i].z, r[8 * i + 4], r[8 * i + 5]);
          widen(va[c + i].w, r[8 * i + 6], r[8 * i + 7]);
        }
        pair::st16(to + out * kColumnsA + 8 * c, r);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (has_x) {
          const int c = xpart + i * kRowParts, c2 = 2 * (c & 3);
          uint32_t q[8];
          widen(vx[i].x, q[0], q[1]);
          widen(vx[i].y, q[2], q[3]);
          widen(vx[i].z, q[4], q[5]);
          widen(vx[i].w, q[6], q[7]);
          const uint32_t at = to_x + out * kOut + (c >> 2) * (kTok * 128);
          write16(at + ((c2 ^ (xrow & 7)) << 4), q[0], q[1], q[2], q[3]);
          write16(at + (((c2 + 1) ^ (xrow & 7)) << 4), q[4], q[5], q[6], q[7]);
        }
      pair::fence_async();
      pair::wait_st();
      pair::fence_before();
      __syncwarp();
      if (lane == 0) pair::arrive_remote(pair::in_cta(full_out(out), 0));
      if ((in += kGroups) >= s1) in -= s1, in_turn ^= 1;
      if ((out += kGroups) >= kS2) out -= kS2, out_turn ^= 1;
    }
  } else if (warp >= kFirstWriter) {
    const int w = warp - kFirstWriter, quad = w & 3, which = w >> 2, other = w ^ 2;   // other: of the same tokens
    const int out_rows = GATED ? half : a.p.rows;
    const bool gate = quad < 2;                // (not gated: the first half tile)
    // this warp's scales of x, and what it hands over and is handed
    float* xs = reinterpret_cast<float*>(raw + (xs0 + w * kScaleBytes - tma::smem_u32(raw)));
    float* mine = reinterpret_cast<float*>(raw + (swap0 + w * kSwap - tma::smem_u32(raw)));
    const uint32_t stage = swap0 + w * kSwap;
    const bool wide = out_rows % 8 == 0 && (reinterpret_cast<uintptr_t>(a.p.out) & 15) == 0;
    const float* theirs = reinterpret_cast<const float*>(raw + (swap0 + other * kSwap - tma::smem_u32(raw)));
    int buf = 0;
    uint32_t buf_turn = 0, swap_turn = 0;
    bool ok = true;
    for (int tile = first_tile; ok && tile < total; tile += pairs) {
      const Tile t = tile_of(tile);
      // the warp's 32 output channels, their rows of w, and the scales of the four that a lane has
      const int lead = (2 * t.row_tile + static_cast<int>(cta)) * (GATED ? a.part : 2 * a.part) + (GATED || gate ? 0 : a.part);
      const int channel = lead + 32 * (quad & 1), row = GATED && !gate ? half + channel : channel;
      const int channels = min(out_rows - channel, a.part - 32 * (quad & 1));
      float ws[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int at = 8 * g + (lane >> 2);
        ws[g] = at < channels ? ld_coherent(a.p.w_scales + static_cast<int64_t>(t.expert) * a.p.rows + row + at) : 0.0f;
      }
      __syncwarp();
      for (int i = 0, c = 32 * which + lane; c < t.width; ++i, c += 32 * kOfQuad)
        xs[32 * i + lane] = c < t.tokens ? ld_coherent(a.p.x_scales + t.first + c) : 0.0f;
      __syncwarp();
      ok = __all_sync(kAll, wait(full_sum(buf), buf_turn));
      if (!ok) break;
      pair::fence_after();
      if (32 * which >= t.width && lane == 0) pair::arrive_remote(pair::in_cta(empty_sum(buf), 0));   // nothing here for it
      for (int i = 0, c = 32 * which; c < t.width; ++i, c += 32 * kOfQuad) {
        uint32_t r[2][16];
        const uint32_t from = tmem + (static_cast<uint32_t>(32 * quad) << 16) + buf * NT + c;
        pair::ld16x32(from, r[0]);
        pair::ld16x32(from + (16u << 16), r[1]);
        pair::wait_ld();
        if (c + 32 * kOfQuad >= t.width) {               // the sums may be overwritten
          pair::fence_before();
          __syncwarp();
          if (lane == 0) pair::arrive_remote(pair::in_cta(empty_sum(buf), 0));
        }
        float y[2][4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(xs + 32 * i + 8 * j + 2 * (lane & 3));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[h][j][e] = __uint_as_float(r[h][4 * j + e]) * ws[2 * h + e / 2] * (e & 1 ? f.y : f.x);
        }
        const int many = t.tokens - c;
        const int64_t at = static_cast<int64_t>(t.first + c) * out_rows + channel;
        if constexpr (GATED) {
          // gate warps finish the first 16 tokens, up warps the last 16
#pragma unroll
          for (int j = 0; j < 16; ++j) mine[32 * j + lane] = gate ? y[j >> 3][2 + (j >> 2 & 1)][j & 3] : y[j >> 3][j >> 2 & 1][j & 3];
          __syncwarp();
          if (lane == 0) tma::mbar_arrive(swap_ready(w));
          ok = __all_sync(kAll, wait(swap_ready(other), swap_turn));
          if (!ok) break;
          float h[2][2][4];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float v = theirs[32 * j + lane], own = gate ? y[j >> 3][j >> 2 & 1][j & 3] : y[j >> 3][2 + (j >> 2 & 1)][j & 3];
            h[j >> 3][j >> 2 & 1][j & 3] = i8_activate(a.p.act, gate ? own : v) * (gate ? v : own);
          }
          __syncwarp();
          if (lane == 0) tma::mbar_arrive(swap_done(other));
          // what was handed over has been read: its place takes the output on its way
          ok = __all_sync(kAll, wait(swap_done(w), swap_turn));
          if (!ok) break;
          swap_turn ^= 1;
          store_tile<2>(a.p, wide, stage, lane, at + (gate ? 0 : 16 * static_cast<int64_t>(out_rows)), out_rows,
                         gate ? many : many - 16, channels, h);
        } else {
          store_tile<4>(a.p, wide, stage, lane, at, out_rows, many, channels, y);
        }
      }
      if (++buf == kD) buf = 0, buf_turn ^= 1;
    }
  }
  __syncwarp();
  pair::fence_before();
  __syncthreads();
  // in both CTAs: the products in flight, and their arrivals here, are over before this block's memory goes
  if (warp == 1) tma::mbar_wait_bounded(end_bar, 0, tma::kDrainNs);
  __syncwarp();
  pair::cluster_sync();
  pair::fence_after();
  if (warp == 2) pair::dealloc(tmem, kTmem);
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

// Boxes of 128 columns by `box` rows of an int8 matrix; zeros outside it.
cudaError_t map_of(CUtensorMap* map, const void* at, int64_t rows, int cols, int box) {
  const Encode f = encoder();
  if (!f) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)}, pitch[1] = {dims[0]};
  const cuuint32_t boxes[2] = {kStep, static_cast<cuuint32_t>(box)}, steps[2] = {1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(at), dims, pitch, boxes, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

struct Gpu {
  int device, sms;
};
cudaError_t current_gpu(Gpu* g) {
  static std::atomic<int> known[64];   // SMs by device, 0: not asked yet
  if (const cudaError_t e = cudaGetDevice(&g->device); e != cudaSuccess) return e;
  g->sms = g->device < 64 ? known[g->device].load(std::memory_order_relaxed) : 0;
  if (g->sms == 0) {
    if (const cudaError_t e = cudaDeviceGetAttribute(&g->sms, cudaDevAttrMultiProcessorCount, g->device); e != cudaSuccess) return e;
    if (g->device < 64) known[g->device].store(g->sms, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

template <int NT, bool GATED>
cudaError_t launch(Args& a, const Gpu& gpu, int64_t most_tiles, cudaStream_t s) {
  const int starts = a.p.first ? 4 * (a.p.experts + 1) : 0;
  const int room = kMaxShared - kFixed - stages_out(NT) * bytes_out(NT) - starts;
  a.stages_in = std::min(16, room / bytes_in(NT));
  static_assert((kMaxShared - kFixed - stages_out(NT) * bytes_out(NT) - 4 * 2049) / bytes_in(NT) >= 2);
  const int smem = 1024 + a.stages_in * bytes_in(NT) + stages_out(NT) * bytes_out(NT) + kFixed + starts;
  if (const cudaError_t e = map_of(&a.x, a.p.x, a.p.n, a.p.cols, x_box(NT)); e != cudaSuccess) return e;
  if (const cudaError_t e = map_of(&a.w, a.p.w, static_cast<int64_t>(a.p.experts) * a.p.rows, a.p.cols, a.part); e != cudaSuccess) return e;
  // the kernel's shared-memory limit is raised once on each device
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (gpu.device & 63);
  if (gpu.device >= 64 || !(ready.load(std::memory_order_relaxed) & bit)) {
    if (const cudaError_t e = cudaFuncSetAttribute(i8_mma_kernel<NT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared + 1024);
        e != cudaSuccess)
      return e;
    if (gpu.device < 64) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(gpu.sms / 2, most_tiles)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  static const bool pdl = PdlEnabled();
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, i8_mma_kernel<NT, GATED>, a);
}

// Cycles of a tile: a stage takes the longest of its products (measured, 8 instructions), widening
// and its share of the memory's rate; the ends are set-up and output, which up to
// 128 tokens run beside the next tile.
int64_t tile_cost(int width, int part, int steps) {
  const int products = 8 * (9 + width / 2), widen = 390 + 3 * width / 2, bytes = 2 * part * kStep / 22;
  return static_cast<int64_t>(steps) * std::max(products, std::max(widen, bytes)) + (width > 128 ? 6000 : 4000);
}

// Tokens of a tile and weight rows of a half tile of a dense product: what takes the fewest cycles
// when each pair of SMs takes its share of the tiles in turn.
int64_t choose(int64_t n, int channels, bool gated, int steps, int pairs, int* nt, int* part) {
  int64_t least = INT64_MAX;
  const int per = gated ? 2 : 4;             // channels of a pair tile for each row of a half tile
  for (int t = 32; t <= 256; t *= 2) {
    const int64_t token_tiles = (n + t - 1) / t;
    const int width = static_cast<int>(((n + token_tiles - 1) / token_tiles + 31) / 32) * 32;
    for (int m = 8; m <= 64; m += 8) {
      const int64_t tiles = token_tiles * ((channels + per * m - 1) / (per * m));
      const int64_t cost = (tiles + pairs - 1) / pairs * tile_cost(width, m, steps);
      if (cost < least) least = cost, *nt = t, *part = m;
    }
  }
  return least;
}

}  // namespace

cudaError_t LaunchI8Product(const I8ProductParams& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  Gpu gpu;
  if (const cudaError_t e = current_gpu(&gpu); e != cudaSuccess) return e;
  const bool gated = p.act != EP_ACT_NONE;
  const int channels = gated ? p.rows / 2 : p.rows;
  Args a{};
  a.p = p;
  a.steps = (p.cols + kStep - 1) / kStep;
  int nt = 256;
  a.part = kRows / 2;
  if (!p.first) {
    // beginning and end take this kernel some 8000 cycles, the other one half of that; that one reaches
    // half of the integer rate, for whole column tiles of 8 tokens
    const int64_t few = 2 * static_cast<int64_t>(p.rows) * p.cols * ((p.n + 7) / 8 * 8) / (261 * gpu.sms) + 4000;
    const bool can = p.n <= kI8FewTokens;
    if (can && few < tile_cost(32, 8, a.steps) + 8000) return LaunchI8Few(p, gpu.device, gpu.sms, s);   // no tile takes less
    const int64_t cost = choose(p.n, channels, gated, a.steps, gpu.sms / 2, &nt, &a.part);
    if (can && few < cost + 8000) return LaunchI8Few(p, gpu.device, gpu.sms, s);
  } else {
    // the average expert's rows, and some more, in one tile
    const int64_t mean = p.entries / p.experts + 1;
    nt = mean <= 24 ? 32 : mean <= 48 ? 64 : mean <= 96 ? 128 : 256;
  }
  const int per = gated ? 2 * a.part : 4 * a.part;
  a.row_tiles = (channels + per - 1) / per;
  const int64_t most = static_cast<int64_t>(a.row_tiles) * (p.first ? std::min<int64_t>(p.entries, p.experts + p.entries / nt)
                                                                    : (p.n + nt - 1) / nt);
  if (gated) {
    if (nt == 32) return launch<32, true>(a, gpu, most, s);
    if (nt == 64) return launch<64, true>(a, gpu, most, s);
    if (nt == 128) return launch<128, true>(a, gpu, most, s);
    return launch<256, true>(a, gpu, most, s);
  }
  if (nt == 32) return launch<32, false>(a, gpu, most, s);
  if (nt == 64) return launch<64, false>(a, gpu, most, s);
  if (nt == 128) return launch<128, false>(a, gpu, most, s);
  return launch<256, false>(a, gpu, most, s);
}

cudaError_t ReadI8Error(int32_t* value, cudaStream_t s) {
  int32_t zero = 0;
  if (const cudaError_t e = cudaMemcpyFromSymbolAsync(value, g_error, sizeof zero, 0, cudaMemcpyDeviceToHost, s); e != cudaSuccess) return e;
  if (const cudaError_t e = cudaMemcpyToSymbolAsync(g_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s); e != cudaSuccess) return e;
  return cudaStreamSynchronize(s);
}

}  // namespace epg
