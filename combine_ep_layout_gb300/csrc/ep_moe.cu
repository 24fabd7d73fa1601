// ep_moe.cu -- the experts of a few tokens in one launch (include/ep_gb300_moe.h:
// ep_moe_forward).
//
// What bounds it: every active expert's 3 H I weights are read once (a token's
// own rows are a few KB), so the work is to keep HBM busy from the first byte to
// the last.  A persistent grid, one block per SM, walks one list of
// items: first the gate/up items (expert, 16 or more channels: the gate's and the up
// projection's rows together, so that the product act(gate) up is formed where
// the sums are), then the down items (expert, 32 or more output channels).  Eight
// (4-bit: twelve) warps split an item's k range chunk by chunk; each streams its own chunks through
// its own cp.async ring (ep_stream.cuh) across items and phases, so the ring never
// drains.  For each column tile of an item (a round) they leave their sums in one
// of two buffers and go on; two more warps, one for each buffer, add up the
// sums and write the round's results; one last warp tells the other blocks, with
// one memory fence for all the rounds written since its last one.  So neither the
// sums nor the microseconds of a fence and an atomic stop the streams.
//
// Up to 8 tokens are routed here as well, every block for itself, a warp a token (one
// launch instead of two: one token over 64 experts of 7168 x 2048 takes 1.2 us less than
// with the router's own launch).
//
// A down item needs its expert's whole h: a counter per active expert, raised by
// each finished gate/up item, is waited for (bounded) just before the item's
// activations are copied; its weights are under way by then.  Experts come in one
// order in both phases, so the wait is short unless few experts are active.
//
// h is kept as several bf16 that add up to it, in as many columns of the down product,
// whose sums are added: two (16 significant bits) for a bf16 output, whose error would
// double with one (columns cost nothing until 4 tokens meet on an expert); three (24 bits,
// all of fp32's) for an fp32 output (2048 x 1024: off by 6e-7 of its norm, 2.4e-6 with two).
// The three take four columns, so that a tile of 8 holds two tokens: 64 experts of 7168 x
// 2048 take 1, 8 and 64 tokens 115, 542 and 1304 us, with a bf16 output 113, 527 and 921.
//
// The down items write fp32 expert rows.  A block that is through with its items
// waits for the rounds of its share of the channel tiles and folds the K rows of
// each token there in order (fmaf over k, as the combine does); every block has the
// same share, whichever was late (folded by the block that finished a tile last, 64
// tokens' rows took the latest block 120 us).  No sum depends on the order of blocks:
// equal inputs, equal bits.
//
// Measured with the routing, of a copy's 6.8 TB/s: bf16, 64 experts of 7168 x
// 2048, top-8: 1 token 113 us (6.2 TB/s), 8 tokens 527 us (7.0 TB/s), 64 tokens 0.92 ms
// (6.1 TB/s: half the experts have more than the 8 tokens of a down job, so part of
// w2 passes the SMs twice, at what L2 gives them).  4-bit, group 128, 128 experts of
// 4096 x 1408, top-6: 8 tokens 104 us (3.6 TB/s) at 54% of the issue slots while active and
// no unit above 44%: latency of 15 warps an SM.  A layer of 32 experts of 1024 x 512 takes 4
// tokens 24 us: set-up 3.7, first weights 4.2, gate/up 3.5, their fences 3.4, down 1.3,
// theirs and the fold 5.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ep_moe_kernels.hpp"
#include "ep_route.cuh"
#include "ep_stream.cuh"
#include "ep_tma.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

using stream::Form;

constexpr int kFinishers = 2;             // warps that finish rounds, one buffer each
constexpr int kMaxEntries = kFewTokens * 16;
using route::kAll;
constexpr int kSmemLimit = 232448 - 3072;  // dynamic shared memory of one block (its static part aside)

__device__ __forceinline__ float activate(float g, int act) {
  if (act == 0) return g / (1.0f + expf(-g));
  const float u = 0.7978845608028654f * (g + 0.044715f * g * g * g);
  return 0.5f * g * (1.0f + tanhf(u));
}

__device__ __forceinline__ int32_t load_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Rounds written whose word to the other blocks may be outstanding; a power of two.
constexpr int kQueue = 64;

// Where the sum of a row and a column (8 of them) or a token (4) lies: both the
// writing lanes (fragments) and the reading ones (rows in sequence) miss each
// other's banks.
__device__ __forceinline__ int red_8(int row, int col) { return row * 8 + (col ^ (row >> 1 & 6)); }
__device__ __forceinline__ int red_4(int row, int tok) { return row * 4 + (tok ^ (row >> 3 & 3)); }

// Every wait is bounded.  Where one gives up, the block is lost: the launch's output is
// not valid (the error word says so), the block's other waits give up as well, and each
// warp stays away from what it waited for and leaves its phase.  No buffer is written
// that may still be read, no word is told of a round that may not be written.
__device__ __forceinline__ void lose(int* lost, int32_t* err) {
  *static_cast<volatile int*>(lost) = 1;
  atomicOr(err, kErrTimeout);
}

// Until the counter that other blocks raise is at `want`, for at most wait_ns.  The
// caller goes on, in bounds.
__device__ __forceinline__ void await_global(const int32_t* counter, int want, uint64_t wait_ns, int* lost, int32_t* err) {
  if (load_acquire(counter) >= want || *static_cast<volatile int*>(lost)) return;
  const uint64_t t0 = now_ns();
  while (load_acquire(counter) < want) {
    if (now_ns() - t0 > wait_ns) {
      lose(lost, err);
      return;
    }
  }
}

// Waits of a whole warp on other warps of its block until test() holds, for at most limit_ns.
// False, for every lane, where the block is lost.
template <class Test>
__device__ __forceinline__ bool await_block(Test test, uint64_t limit_ns, int* lost, int32_t* err) {
  bool ok = test();
  if (__all_sync(kAll, ok)) return true;
  const uint64_t t0 = now_ns();
  while (!ok && !*static_cast<volatile int*>(lost) && now_ns() - t0 < limit_ns) ok = test();
  if (__all_sync(kAll, ok)) return true;
  if ((threadIdx.x & 31) == 0) lose(lost, err);
  return false;
}
// until the phase of a barrier with the given parity is over (the test may rest until it is,
// but not with a limit of 0)
__device__ __forceinline__ bool await_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns, int* lost, int32_t* err) {
  return await_block([&]() { return limit_ns ? tma::mbar_try_wait(bar, parity) : tma::mbar_test(bar, parity); }, limit_ns,
                     lost, err);
}
// until *count >= want, a count in shared memory
__device__ __forceinline__ bool await_count(const int* count, int want, uint64_t limit_ns, int* lost, int32_t* err) {
  auto there = [&]() { return *static_cast<const volatile int*>(count) >= want; };
  return __all_sync(kAll, there()) || await_block([&]() { __nanosleep(64); return there(); }, limit_ns, lost, err);
}

// A job: some tokens (at most the phase's cap, 16) of one active expert, in one
// word: the expert, the first of its entries in the grouped list, how many, and
// the column tiles of 8 tokens that the whole expert has.
struct Job {
  int expert, start, count, parts;
};
__device__ __forceinline__ uint32_t pack_job(int expert, int start, int count, int parts) {
  return static_cast<uint32_t>(expert) | static_cast<uint32_t>(start) << 11 | static_cast<uint32_t>(count - 1) << 21 |
         static_cast<uint32_t>(parts - 1) << 25;
}
__device__ __forceinline__ Job unpack_job(uint32_t j) {
  return {static_cast<int>(j & 2047), static_cast<int>(j >> 11 & 1023), static_cast<int>(j >> 21 & 15) + 1,
          static_cast<int>(j >> 25) + 1};
}

// Shared memory behind the rings, sized by the number of entries n K.
struct Lists {
  uint32_t *jobs_0, *jobs_1;
  uint16_t* entry;     // entries grouped by expert, ascending within one
  uint32_t* valid;     // by entry, one bit each
};

constexpr int lists_bytes(int entries) { return (entries * (4 + 4 + 2) + entries / 8 + 4 + 15) & ~15; }

// How a block is cut for weights of form G and up to NT column tiles a job.  The
// ring takes what shared memory is left; 64 KB of weights under way per SM carry
// HBM's full rate.
template <int G, int NT>
struct Shape {
  // 4 row tiles spare 4-bit weights half the work on the activations (105 us, with 2
  // 116 us: 8 tokens, 128 experts of 4096 x 1408, groups of 128; with groups of 32 121 and
  // 133); with 16 columns they would leave the ring too short
  static constexpr int kRowTiles = G != 0 && NT == 1 ? 4 : 2;
  // columns of one job: gate/up a token each, down as many for a token as it has parts
  static constexpr int kLogCap = NT == 1 ? 3 : 4, kCap = 1 << kLogCap;
  static constexpr int kEnough = 8, kItems = 4;              // stages of a warp in an item, items of a block (see widen)
  using F = Form<G, kRowTiles>;
  // 4-bit weights take more instructions a byte: 12 warps (105 and 391 us for 8 and 64
  // tokens of those experts, with 8 warps 114 and 451 us; groups of 32 and 64 the same to 1%)
  static constexpr int kWarps = G != 0 ? 12 : 8;
  static constexpr int kAllWarps = kWarps + kFinishers + 1;
  static constexpr int kThreads = 32 * kAllWarps;
  static constexpr int kTokens = NT == 1 ? 8 : kFewTokens;   // most tokens of a call
  static constexpr int kRed = kWarps * F::kRows * 8 * 4;     // one round's partial sums, one of two buffers
  static constexpr int kSlot = F::stage_bytes(NT);
  static constexpr int kFit = (kSmemLimit - 2 * kRed - lists_bytes(kTokens * 16)) / (kWarps * kSlot);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kRing = kWarps * kStages * kSlot;
  static_assert(kStages >= 2);
  // the set-up's counts (of 2048 experts, 32 bytes and a word each) and ranks use the ring
  static_assert(kRing >= 2048 * 36 + 4 * kMaxEntries + 2 * kOwnTokens * kOwnTopk + 4 * 32 * kOwnTokens);
};

// F32: fp32 output.
template <int G, int NT, bool F32>
__global__ void __launch_bounds__(Shape<G, NT>::kThreads, 1) moe_kernel(const MoeParams p) {
  using S = Shape<G, NT>;
  using F = typename S::F;
  constexpr int RT = F::kRowTiles, kStages = S::kStages, kWarps = S::kWarps, kAllWarps = S::kAllWarps;
  constexpr int kThreads = S::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t scan_warp[kAllWarps];
  __shared__ float own_weight[kOwnTokens * kOwnTopk];   // by entry, of tokens routed here
  __shared__ int s_flag, s_lost, s_rounds;
  __shared__ __align__(8) uint64_t s_full[2], s_free[2];   // by buffer: its sums are written, are read
  __shared__ int s_written[2], s_told;       // rounds written by each finisher, rounds told
  __shared__ uint16_t queue[kQueue];         // by round: the expert (gate/up) or the tile (down)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int entries = p.n * p.topk;
  constexpr int h_rows = F32 ? 3 : 2;        // bf16 parts of h, rows of I next to one another
  constexpr int log_part = F32 ? 2 : 1;      // columns of a token in the down product: 4 or 2
  constexpr int log_toks = 3 - log_part;     // tokens of a column tile there: 2 or 4
  float* red_all = reinterpret_cast<float*>(smem + S::kRing);
  Lists L;
  {
    uint8_t* b = smem + S::kRing + 2 * S::kRed;
    L.jobs_0 = reinterpret_cast<uint32_t*>(b);
    L.jobs_1 = L.jobs_0 + entries;
    L.valid = L.jobs_1 + entries;
    L.entry = reinterpret_cast<uint16_t*>(L.valid + (entries + 31) / 32);
  }

  // ---- which experts, with which tokens: every block works it out for itself
  // Entries go by chunks of 32, a warp each, in any order: what an entry's place
  // among its expert's needs is how many of the expert's entries earlier chunks have,
  // one byte for each expert and chunk.
  uint32_t* by_chunk = reinterpret_cast<uint32_t*>(smem);                 // [E][32 bytes]
  int* first_of = reinterpret_cast<int*>(smem + 2048 * 32);               // by expert
  uint16_t* expert_of = reinterpret_cast<uint16_t*>(smem + 2048 * 36);    // by entry
  uint16_t* rank_of = expert_of + kMaxEntries;                            // within its chunk
  int16_t* routed = reinterpret_cast<int16_t*>(rank_of + kMaxEntries);    // by entry: the expert, -1 for none
  int* slots = reinterpret_cast<int*>(routed + kOwnTokens * kOwnTopk);    // 32 of each token
  const int chunk_words = (entries + 127) / 128;                          // of 4 bytes
  auto entries_before = [&](int e, int chunk) {
    int sum = 0;
    for (int w = 0; 4 * w < chunk; ++w) {
      const int bytes = chunk - 4 * w;
      const uint32_t mask = bytes >= 4 ? ~0u : (1u << 8 * bytes) - 1u;
      sum = static_cast<int>(__dp4a(by_chunk[8 * e + w] & mask, 0x01010101u, static_cast<unsigned>(sum)));
    }
    return sum;
  };
  if (tid == 0) {
    s_lost = s_rounds = s_written[0] = s_written[1] = s_told = 0;
    for (int b = 0; b < 2; ++b) {
      tma::mbar_init(stream::smem_addr(&s_full[b]), kWarps);
      tma::mbar_init(stream::smem_addr(&s_free[b]), 1);
    }
  }
  const uint32_t full_bar = stream::smem_addr(s_full), free_bar = stream::smem_addr(s_free);
  for (int i = tid; i < p.experts * chunk_words; i += kThreads) by_chunk[i / chunk_words * 8 + i % chunk_words] = 0;
  // a few tokens' routing, a warp each: every block for itself, the first one writes it down
  if (p.logits && warp < p.n) {
    const float* row = static_cast<const float*>(p.logits) + warp * p.logits_stride;
    const __nv_bfloat16* row16 = static_cast<const __nv_bfloat16*>(p.logits) + warp * p.logits_stride;
    auto score = [&](int j) { return fmaxf(p.logits_bf16 ? __bfloat162float(row16[j]) : row[j], -INFINITY); };
    float key[kOwnExperts / 32];
#pragma unroll
    for (int v = 0; v < kOwnExperts / 32; ++v) key[v] = 32 * v + lane < p.experts ? score(32 * v + lane) : -INFINITY;
    float zk = -INFINITY;
    const int chosen = route::choose<kOwnExperts / 32, kOwnTopk, true>(key, p.topk, lane, slots + 32 * warp, score, zk);
    const float f = route::chosen_weight(zk, p.sigmoid, p.renorm);
    if (lane < p.topk) {
      const int i = warp * p.topk + lane;
      const float w = chosen >= 0 ? f * p.route_scale : 0.0f;
      routed[i] = static_cast<int16_t>(chosen);
      own_weight[i] = w;
      if (blockIdx.x == 0) p.idx_out[i] = chosen, p.weights_out[i] = w;
    }
  }
  __syncthreads();
  for (int i0 = 32 * warp; i0 < entries; i0 += kThreads) {
    const int i = i0 + lane;
    int64_t id = -1;
    if (i < entries) id = p.logits ? routed[i] : p.topk_idx[i];
    const bool ok = id >= 0 && id < p.experts;
    if (i < entries && !ok && id != -1 && blockIdx.x == 0) atomicOr(p.err, kErrBadExpert);
    const int e = ok ? static_cast<int>(id) : -1 - lane;
    const unsigned same = __match_any_sync(kAll, e), before = same & ((1u << lane) - 1u);
    const unsigned oks = __ballot_sync(kAll, ok);
    if (ok && before == 0) reinterpret_cast<uint8_t*>(by_chunk)[32 * e + i0 / 32] = static_cast<uint8_t>(__popc(same));
    if (lane == 0) L.valid[i0 / 32] = oks;
    if (i < entries) {
      expert_of[i] = ok ? static_cast<uint16_t>(e) : 0xffff;
      rank_of[i] = static_cast<uint16_t>(__popc(before));
    }
  }
  __syncthreads();
  int jobs_0, jobs_1;
  {
    // three 16-bit sums in one word: entries, gate/up jobs, down jobs
    const int per = (p.experts + kThreads - 1) / kThreads, e0 = tid * per;
    const int e1 = min(e0 + per, p.experts);
    auto word = [&](int c) -> uint64_t {
      return c == 0 ? 0
                    : static_cast<uint64_t>(c) | static_cast<uint64_t>((c - 1 >> S::kLogCap) + 1) << 16 |
                          static_cast<uint64_t>((c - 1 >> (S::kLogCap - log_part)) + 1) << 32;
    };
    uint64_t mine = 0;
    int rounds = 0;        // down rounds of one channel tile
    for (int e = e0; e < e1; ++e) {
      const int c = entries_before(e, 4 * chunk_words);
      first_of[e] = c;
      mine += word(c), rounds += (c - 1 >> log_toks) + 1;   // (0 for c = 0)
    }
    if (rounds) atomicAdd(&s_rounds, rounds);
    uint64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t v = __shfl_up_sync(kAll, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31) scan_warp[warp] = upto;
    __syncthreads();
    uint64_t base = upto - mine, all = 0;
    for (int w = 0; w < kAllWarps; ++w) {
      if (w < warp) base += scan_warp[w];
      all += scan_warp[w];
    }
    jobs_0 = static_cast<int>(all >> 16 & 0xffff);
    jobs_1 = static_cast<int>(all >> 32 & 0xffff);
    for (int e = e0; e < e1; ++e) {
      const int c = first_of[e];
      if (c == 0) continue;
      const int start = static_cast<int>(base & 0xffff);
      for (int ph = 0; ph < 2; ++ph) {
        const int cap = ph == 0 ? S::kCap : S::kCap >> log_part;
        int j = static_cast<int>(base >> (16 + 16 * ph) & 0xffff);
        for (int o = 0; o < c; o += cap, ++j)
          (ph == 0 ? L.jobs_0 : L.jobs_1)[j] = pack_job(e, start + o, min(cap, c - o), (c + 7) >> 3);
      }
      base += word(c);
      first_of[e] = start;
    }
  }
  __syncthreads();
  for (int i = tid; i < entries; i += kThreads) {
    const int e = expert_of[i];
    if (e != 0xffff) {
      L.entry[first_of[e] + entries_before(e, i / 32) + rank_of[i]] = static_cast<uint16_t>(i);
    }
  }
  __syncthreads();   // the ring's memory is free from here on

  // ---- the list of items and this warp's walk through it
  // (pick: by phase, without arrays that would have to live in memory)
  auto pick = [](int ph, auto a, auto b) { return ph == 0 ? a : b; };
  auto dim_k = [&](int ph) { return pick(ph, p.hidden, p.inter); };       // columns of the weight rows
  constexpr int kHalf = F::kRows / 2;       // gate rows, and up rows, of a gate/up tile
  const int grid = gridDim.x;
  const int chunks_0 = (p.hidden + F::kCols - 1) / F::kCols, chunks_1 = (p.inter + F::kCols - 1) / F::kCols;
  auto chunks = [&](int ph) { return pick(ph, chunks_0, chunks_1); };
  // An item is `wide` row tiles side by side, 1, 2 or 4, each with its share of the
  // warps: where the columns are few, one tile would give a warp so few stages that
  // setting them up costs more than they do (8 tokens, 128 4-bit experts of 4096 x
  // 1408: 105 us, with one tile always 114, 64 tokens 391 and 509; 64 tokens, 64 experts of
  // 7168 x 2048: 0.91 and 0.98 ms).  As long as every block keeps enough items for all to end together, and
  // not for bf16 weights with an fp32 output: a warp's sums are then up to four times as
  // long, and the matrix instruction's additions round worse than fp32's (2048 x 1024, 64
  // tokens: off by 1.5e-6 of the output's norm, with one tile always 6.1e-7; 4-bit groups
  // have sums of their own, 1.5e-7).
  auto widen = [&](int subtiles, int jobs, int n_chunks) {   // the logarithm of the tiles
    int r = 0;
    while (r < 2 && !(F32 && G == 0) && (n_chunks << r) < S::kEnough * kWarps && jobs * (((subtiles - 1) >> (r + 1)) + 1) >= S::kItems * grid) ++r;
    return r;
  };
  const int sub_0 = (p.inter + kHalf - 1) / kHalf, sub_1 = (p.hidden + F::kRows - 1) / F::kRows;
  const int side_0 = widen(sub_0, jobs_0, chunks_0), side_1 = widen(sub_1, jobs_1, chunks_1);
  const int tiles_0 = ((sub_0 - 1) >> side_0) + 1, tiles_1 = ((sub_1 - 1) >> side_1) + 1;
  auto tiles = [&](int ph) { return pick(ph, tiles_0, tiles_1); };
  auto jobs_of = [&](int ph) { return pick(ph, jobs_0, jobs_1); };
  auto job_at = [&](int ph, int j) { return unpack_job(pick(ph, L.jobs_0, L.jobs_1)[j]); };
  const uint32_t by_topk = 65536u / static_cast<uint32_t>(p.topk) + 1;    // entry / topk, exact below 2^14
  // This block's items, phase by phase: every grid-th of the list, but where the
  // gate/up items do not go round evenly, the blocks with one fewer (`late` on) take
  // the first `extra` rounds of down items among themselves, as many as weigh what a
  // gate/up item does.
  const int late = jobs_0 * tiles_0 % grid, lates = grid - late;
  const int extra = late == 0 ? 0
                              : min((2 * (p.hidden << side_0) / (p.inter << side_1) + 1) / 2, jobs_1 * tiles_1 / lates);
  const int block = static_cast<int>(blockIdx.x), my_extra = block >= late ? extra : 0;
  struct Items {
    int ph, job, tile, n;   // the n-th of this block in phase ph
  };
  auto settle_tile = [&](Items& i) {
    while (i.tile >= tiles(i.ph)) i.tile -= tiles(i.ph), ++i.job;
  };
  auto begin_items = [&](Items& i, int ph) {
    i = {ph, 0, block, 0};
    if (ph == 1) i.tile = my_extra > 0 ? block - late : extra * lates + block;
    if (ph < 2) settle_tile(i);
  };
  auto next_item = [&](Items& i) {
    ++i.n;
    i.tile += i.ph == 0 || i.n > my_extra ? grid : i.n < my_extra ? lates : lates + late;
    settle_tile(i);
  };
  auto there = [&](const Items& i) { return i.job < jobs_of(i.ph); };

  if (warp < kWarps) {   // ---- the streaming warps
  const uint32_t ring = stream::smem_addr(smem) + warp * kStages * S::kSlot;
  const bool whole_0 = F::kInt4 && p.hidden % 128 == 0 && (reinterpret_cast<uintptr_t>(p.w13_scales) & 15) == 0;
  const bool whole_1 = F::kInt4 && p.inter % 128 == 0 && (reinterpret_cast<uintptr_t>(p.w2_scales) & 15) == 0;

  // This warp's place in an item: row tile `sub` of it, and chunk c = lead, lead +
  // step, ... of the columns; an item's last chunk is followed by the next item's
  // first, so that no warp has more chunks than another in the long run.
  const int step_0 = kWarps >> side_0, step_1 = kWarps >> side_1;
  const int at_0 = warp / step_0, at_1 = warp / step_1, lead_0 = warp % step_0, lead_1 = warp % step_1;
  auto step = [&](int ph) { return pick(ph, step_0, step_1); };
  auto lead = [&](int ph) { return pick(ph, lead_0, lead_1); };
  auto sub_tile = [&](int ph, int tile) { return pick(ph, (tile << side_0) + at_0, (tile << side_1) + at_1); };
  struct Walk : Items {
    int c;
  };
  auto begin = [&](Walk& w, int ph) {
    begin_items(w, ph);
    w.c = ph < 2 ? lead(ph) : 0;
  };
  // to an item where this warp has a chunk: over the ends of items and phases
  auto settle = [&](Walk& w) {
    while (w.ph < 2) {
      if (!there(w)) {
        begin(w, w.ph + 1);
      } else if (w.c < chunks(w.ph)) {
        return;
      } else {
        w.c -= chunks(w.ph);
        next_item(w);
      }
    }
  };
  // to the next chunk; true when that is another item
  auto advance = [&](Walk& w) {
    w.c += step(w.ph);
    if (w.c < chunks(w.ph)) return false;
    settle(w);
    return true;
  };

  // What a lane copies of each stage of an item.  Weights: piece `lane_piece` of
  // kCopies rows; activations: piece `lane_xpiece` of kXCopies columns; scales:
  // of tile rows `lane`, `lane` + 32.
  constexpr int kXCopies = 8 * NT * F::kXPieces / 32;
  const int lane_row = lane / F::kPieces, lane_piece = lane % F::kPieces;
  const int lane_col = lane / F::kXPieces, lane_xpiece = lane % F::kXPieces;
  const uint32_t a_dst = F::a_offset(lane_row, lane_piece);
  const uint8_t *w_lo = nullptr, *w_hi = nullptr;   // this lane's first row of either half of the tile
  uint32_t w_step = 0;                      // bytes from one of its rows to the next
  int w_left = 0;                           // rows of a half that exist (gate/up: of either; down: of the tile)
  const float* s_src[F::kRows / 32] = {};   // of tile rows `lane`, `lane` + 32
  auto channel_row = [&](int ph, int tile, int r) {
    const int at = sub_tile(ph, tile);
    if (ph == 1) return min(at * F::kRows + r, p.hidden - 1);
    const int ch = min(at * kHalf + (r < kHalf ? r : r - kHalf), p.inter - 1);
    return r < kHalf ? ch : p.inter + ch;
  };
  auto expert_scales = [&](const Walk& w) {
    return pick(w.ph, p.w13_scales, p.w2_scales) +
           static_cast<int64_t>(job_at(w.ph, w.job).expert) * pick(w.ph, 2 * p.inter, p.hidden) * (dim_k(w.ph) / (F::kInt4 ? G : 1));
  };
  auto enter_weights = [&](const Walk& w) {
    // rows of a tile that do not exist (the last tile's) are zeros
    const int64_t row_bytes = dim_k(w.ph) / F::kPerPiece * 16;
    const int at = sub_tile(w.ph, w.tile), row = at * pick(w.ph, kHalf, F::kRows);
    w_left = pick(w.ph, p.inter, p.hidden) - row;
    w_lo = static_cast<const uint8_t*>(pick(w.ph, p.w13, p.w2)) + lane_piece * 16 +
           (static_cast<int64_t>(job_at(w.ph, w.job).expert) * pick(w.ph, 2 * p.inter, p.hidden) + row + lane_row) * row_bytes;
    w_hi = w_lo + pick(w.ph, p.inter, kHalf) * row_bytes;
    w_step = static_cast<uint32_t>(row_bytes) * (32 / F::kPieces);
    if constexpr (F::kInt4) {
      const float* scales = expert_scales(w);
#pragma unroll
      for (int i = 0; i < F::kRows / 32; ++i)
        s_src[i] = scales + static_cast<int64_t>(channel_row(w.ph, w.tile, lane + 32 * i)) * (dim_k(w.ph) / G);
    }
  };
  auto copy_weights = [&](const Walk& w, uint32_t slot) {
    const bool ok = w.c * F::kPieces + lane_piece < dim_k(w.ph) / F::kPerPiece;
    const int64_t at = ok ? w.c * F::kRowBytes : 0;
    const uint8_t *lo = w_lo + at, *hi = w_hi + at;
    const uint32_t dst = slot + a_dst;
    constexpr int kEach = F::kCopies / 2, kPitch = 32 / F::kPieces * F::kRowBytes;
    if (w_left >= pick(w.ph, kHalf, F::kRows)) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) stream::copy16(dst + i * kPitch, lo + static_cast<uint64_t>(i) * w_step, ok);
#pragma unroll
      for (int i = 0; i < kEach; ++i) stream::copy16(dst + (kEach + i) * kPitch, hi + static_cast<uint64_t>(i) * w_step, ok);
    } else {
      const int left_hi = pick(w.ph, w_left, w_left - kHalf);
      const uint8_t* none = static_cast<const uint8_t*>(pick(w.ph, p.w13, p.w2));   // read by nobody
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = lane_row + i * (32 / F::kPieces);
        const bool ok_lo = ok && r < w_left, ok_hi = ok && r < left_hi;
        stream::copy16(dst + i * kPitch, ok_lo ? lo + static_cast<uint64_t>(i) * w_step : none, ok_lo);
        stream::copy16(dst + (kEach + i) * kPitch, ok_hi ? hi + static_cast<uint64_t>(i) * w_step : none, ok_hi);
      }
    }
    if constexpr (F::kInt4) {
      if (pick(w.ph, whole_0, whole_1)) {
#pragma unroll
        for (int i = 0; i < F::kRows / 32; ++i)
          stream::copy_wide<4 * F::kScales>(slot + F::kABytes + 4 * F::kScales * (lane + 32 * i), s_src[i] + w.c * F::kScales);
      } else {
        stream::copy_scales<G, RT>(slot, lane, expert_scales(w), dim_k(w.ph), w.c,
                                   [&](int r) { return channel_row(w.ph, w.tile, r); });
      }
    }
  };
  // the activations' part: the job's columns (phase 1: the parts of each entry's h; what
  // the fourth column of a token with three parts holds is not used)
  uint32_t x_off[kXCopies];                 // elements, from x or h
  int x_cols = 0;
  auto enter_columns = [&](const Walk& w) {
    const Job job = job_at(w.ph, w.job);
    x_cols = job.count << pick(w.ph, 0, log_part);
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) {
      const int col = lane_col + i * (32 / F::kXPieces);
      if (col < x_cols)
        x_off[i] = (w.ph == 0 ? (L.entry[job.start + col] * by_topk >> 16)
                              : static_cast<uint32_t>(h_rows * L.entry[job.start + (col >> log_part)] +
                                                      min(col & ((1 << log_part) - 1), h_rows - 1))) *
                   static_cast<uint32_t>(dim_k(w.ph));
    }
  };
  auto copy_columns = [&](const Walk& w, uint32_t slot) {
    const int at = w.c * F::kCols + 8 * lane_xpiece;
    const bool ok = at < dim_k(w.ph);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(pick(w.ph, p.x, static_cast<const void*>(p.h))) + (ok ? at : 0);
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) {
      const int col = lane_col + i * (32 / F::kXPieces);
      if (col < x_cols) stream::copy16(slot + F::x_offset(col, lane_xpiece), src + x_off[i], ok);
    }
  };
  // until every gate/up item of the job's expert is done
  auto await_expert = [&](const Walk& w) {
    const Job job = job_at(1, w.job);
    if (lane == 0) await_global(p.ready + job.expert, tiles_0 * job.parts, p.wait_ns, &s_lost, p.err);
    __syncwarp();
  };

  Walk pf;
  begin(pf, 0);
  settle(pf);
  int ahead = 0;           // stages of phase 1 whose weights are under way without their columns
  int phase = 0, awaited = -1;
  bool fresh = true;       // pf stands at an item whose copies are not set up
  auto issue = [&](int slot_index) {
    if (pf.ph < 2) {
      const uint32_t slot = ring + slot_index * S::kSlot;
      if (fresh) enter_weights(pf);
      copy_weights(pf, slot);
      if (pf.ph == phase) {
        if (fresh) {
          if (phase == 1 && pf.job != awaited) await_expert(pf), awaited = pf.job;
          enter_columns(pf);
        }
        copy_columns(pf, slot);
      } else {
        ++ahead;
      }
      fresh = advance(pf);
    }
    stream::commit();
  };
  int round = 0;
  int in = 0, out = 0;     // ring positions of the next stage to fill and to use
  bool whole = true;       // no wait on the block gave up
  for (int s = 0; s < kStages - 1; ++s) issue(in), ++in;

  for (phase = 0; phase < 2 && whole; ++phase) {
    if (phase == 1 && ahead > 0) {
      Walk w;
      begin(w, 1);
      settle(w);
      int slot = out;
      bool enter = true;
      for (int s = 0; s < ahead; ++s) {
        if (enter) {
          if (w.job != awaited) await_expert(w), awaited = w.job;
          enter_columns(w);
        }
        copy_columns(w, ring + slot * S::kSlot);
        slot = slot + 1 == kStages ? 0 : slot + 1;
        enter = advance(w);
      }
      // pf stands where w does; its item's columns are the ones just set up unless it is another item
      stream::commit();
      stream::wait<0>();
      __syncwarp();
    }
    Items item;
    int c = lead(phase);
    for (begin_items(item, phase); whole && there(item); next_item(item)) {
      const Job job = job_at(phase, item.job);
      const int cols = job.count << (phase == 0 ? 0 : log_part);
      const int nts = (cols + 7) >> 3;
      float acc[RT][NT][4];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][nt][i] = 0.0f;
      for (; c < chunks(phase); c += step(phase)) {
        stream::wait<kStages - 2>();
        __syncwarp();      // every lane's copies of this stage, and every lane done with the slot refilled next
        issue(in);
        in = in + 1 == kStages ? 0 : in + 1;
        const uint8_t* slot = smem + (warp * kStages + out) * S::kSlot;
        out = out + 1 == kStages ? 0 : out + 1;
        if (NT == 1 || nts == 1)
          stream::consume<G, RT, 1, NT>(slot, lane, acc);
        else
          stream::consume<G, RT, NT, NT>(slot, lane, acc);
      }
      c -= chunks(phase);
      // one round per column tile: the sums to its buffer
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt >= nts) break;
        const int buf = round & 1;
        float* red = red_all + buf * (S::kRed / 4);
        whole = round < 2 || await_phase(free_bar + 8 * buf, (round >> 1) - 1 & 1, p.block_wait_ns, &s_lost, p.err);
        if (!whole) break;
        if (phase == 0) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float* r0 = red + warp * F::kRows * 8;
            *reinterpret_cast<float2*>(r0 + red_8(16 * rt + g, 2 * t)) = make_float2(acc[rt][nt][0], acc[rt][nt][1]);
            *reinterpret_cast<float2*>(r0 + red_8(16 * rt + g + 8, 2 * t)) = make_float2(acc[rt][nt][2], acc[rt][nt][3]);
          }
        } else {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float* r0 = red + warp * F::kRows * 4;
            float lo = acc[rt][nt][0], hi = acc[rt][nt][2];
            if (log_part == 1 || (t & 1) == 0) lo += acc[rt][nt][1], hi += acc[rt][nt][3];
            if (log_part == 2) lo += __shfl_xor_sync(kAll, lo, 1), hi += __shfl_xor_sync(kAll, hi, 1);
            if (log_part == 1 || (t & 1) == 0) {
              r0[red_4(16 * rt + g, t >> (log_part - 1))] = lo;
              r0[red_4(16 * rt + g + 8, t >> (log_part - 1))] = hi;
            }
          }
        }
        __syncwarp();
        if (lane == 0) tma::mbar_arrive(full_bar + 8 * buf);
        ++round;
      }
    }
  }
  stream::wait<0>();
  } else if (warp < kWarps + kFinishers) {
    // ---- the finishing warps: every other round each
    const int buf = warp - kWarps;
    const float* red = red_all + buf * (S::kRed / 4);
    int round = 0;
    bool whole = true;       // no wait on the block gave up
    // the sums of the warps that share a row tile, in the order of warps
    auto add_up = [](const float* at, int stride, int warps) {
      float sum = 0.0f;
      if (warps == kWarps) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += at[w * stride];
      } else {
        for (int w = 0; w < warps; ++w) sum += at[w * stride];
      }
      return sum;
    };
    for (int phase = 0; phase < 2; ++phase) {
      const int step = kWarps >> pick(phase, side_0, side_1);
      Items item;
      for (begin_items(item, phase); whole && there(item); next_item(item)) {
        const Job job = job_at(phase, item.job);
        const int tile = item.tile;
        const int cols = job.count << pick(phase, 0, log_part);
        for (int nt = 0; 8 * nt < cols; ++nt, ++round) {
          if ((round & 1) != buf) continue;
          whole = await_phase(full_bar + 8 * buf, round >> 1 & 1, p.block_wait_ns, &s_lost, p.err);
          if (!whole) break;
          if (phase == 0) {
            const int n_cols = min(8, cols - 8 * nt);
            for (int v = lane; v < kHalf * n_cols << side_0; v += 32) {
              const int ch = v % kHalf, at = v / kHalf & ((1 << side_0) - 1), col = v / kHalf >> side_0;
              const int i = ((tile << side_0) + at) * kHalf + ch;
              const float* from = red + at * step * F::kRows * 8;
              const float gate = add_up(from + red_8(ch, col), F::kRows * 8, step);
              const float up = add_up(from + red_8(kHalf + ch, col), F::kRows * 8, step);
              if (i < p.inter) {
                const float h = activate(gate, p.act) * up;
                const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                // an infinite or NaN h has nothing below it
                const float rest = fabsf(h - __bfloat162float(hi)) < INFINITY ? h - __bfloat162float(hi) : 0.0f;
                const __nv_bfloat16 mid = __float2bfloat16_rn(rest);
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.h) +
                                     static_cast<int64_t>(h_rows * L.entry[job.start + 8 * nt + col]) * p.inter + i;
                dst[0] = hi;
                dst[p.inter] = mid;
                if (h_rows == 3) dst[2 * p.inter] = __float2bfloat16_rn(rest - __bfloat162float(mid));
              }
            }
          } else {
            const int n_tok = min(1 << log_toks, job.count - (nt << log_toks));
            for (int v = lane; v < F::kRows * n_tok << side_1; v += 32) {
              const int r = v % F::kRows, at = v / F::kRows & ((1 << side_1) - 1), tok = v / F::kRows >> side_1;
              const int c = ((tile << side_1) + at) * F::kRows + r;
              const float sum = add_up(red + at * step * F::kRows * 4 + red_4(r, tok), F::kRows * 4, step);
              if (c < p.hidden) p.part[static_cast<int64_t>(L.entry[job.start + (nt << log_toks) + tok]) * p.hidden + c] = sum;
            }
          }
          __syncwarp();
          if (lane == 0) tma::mbar_arrive(free_bar + 8 * buf);
          whole = await_count(&s_told, round - kQueue + 1, p.block_wait_ns, &s_lost, p.err);
          if (!whole) break;
          if (lane == 0) {
            queue[round % kQueue] = static_cast<uint16_t>(phase == 0 ? job.expert : tile);
            __threadfence_block();
            *static_cast<volatile int*>(&s_written[buf]) = (round >> 1) + 1;
          }
        }
      }
    }
  } else {
    // ---- the warp that tells: rounds [told, upto) are written, one fence for all of them
    int total[2] = {0, 0};
    for (int ph = 0; ph < 2; ++ph) {
      Items item;
      for (begin_items(item, ph); there(item); next_item(item)) {
        const int count = job_at(ph, item.job).count;
        total[ph] += (count - 1 >> pick(ph, 3, log_toks)) + 1;
      }
    }
    const int rounds = total[0] + total[1];
    for (int told = 0; told < rounds;) {
      if (!await_count(&s_written[told & 1], (told >> 1) + 1, p.block_wait_ns, &s_lost, p.err)) break;
      const int w0 = *static_cast<volatile int*>(&s_written[0]), w1 = *static_cast<volatile int*>(&s_written[1]);
      // even rounds below 2 w0 and odd rounds below 2 w1 are written
      const int upto = max(told + 1, min(min(2 * w0, 2 * w1 + 1), told + 32));
      __threadfence();
      __syncwarp();
      const int r = __shfl_sync(kAll, told, 0) + lane;
      if (r < __shfl_sync(kAll, upto, 0)) {
        const int what = *static_cast<volatile uint16_t*>(&queue[r % kQueue]);
        atomicAdd(r < total[0] ? p.ready + what : p.tile_done + what, 1);
      }
      told = __shfl_sync(kAll, upto, 0);
      if (lane == 0) *static_cast<volatile int*>(&s_told) = told;
    }
  }
  // ---- this block's share of the channel tiles: the K rows of each token
  const int my_tiles = blockIdx.x < tiles_1 ? (tiles_1 - 1 - static_cast<int>(blockIdx.x)) / grid + 1 : 0;
  for (int f = tid; f < my_tiles; f += kThreads)
    await_global(p.tile_done + blockIdx.x + f * grid, s_rounds, p.wait_ns, &s_lost, p.err);
  __syncthreads();
  {
    // four channels at a time, two of them in flight a thread and step of k
    const int rows = F::kRows << side_1, quads = rows / 4, per_tile = quads * p.n, total = my_tiles * per_tile;
    for (int v0 = tid; v0 < total; v0 += 2 * kThreads) {
      float4 sum[2];
      int tok[2], c[2];        // c < 0: no value
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int v = min(v0 + i * kThreads, total - 1), f = v / per_tile, w = v - f * per_tile;
        tok[i] = w / quads;
        c[i] = (static_cast<int>(blockIdx.x) + f * grid) * rows + 4 * (w - tok[i] * quads);
        if (v0 + i * kThreads >= total || c[i] >= p.hidden) c[i] = -1;
        sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll 4
      for (int k = 0; k < p.topk; ++k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int en = tok[i] * p.topk + k;
          if (c[i] < 0 || !(L.valid[en / 32] >> (en % 32) & 1)) continue;
          const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(en) * p.hidden + c[i]));
          const float w = p.logits ? own_weight[en] : p.topk_weights[en];
          sum[i].x = fmaf(w, y.x, sum[i].x), sum[i].y = fmaf(w, y.y, sum[i].y);
          sum[i].z = fmaf(w, y.z, sum[i].z), sum[i].w = fmaf(w, y.w, sum[i].w);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (c[i] < 0) continue;
        const int64_t o = static_cast<int64_t>(tok[i]) * p.hidden + c[i];
        if (p.bias) {
          const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.bias) + o);
          sum[i].x += __uint_as_float(b.x << 16), sum[i].y += __uint_as_float(b.x & 0xffff0000u);
          sum[i].z += __uint_as_float(b.y << 16), sum[i].w += __uint_as_float(b.y & 0xffff0000u);
        }
        if constexpr (F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = sum[i];
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(sum[i].x, sum[i].y), hi = __floats2bfloat162_rn(sum[i].z, sum[i].w);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    }
  }
  // the last block to get here clears the counters for the next launch
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_flag = atomicAdd(p.blocks_done, 1) == grid - 1;
    __threadfence();
  }
  __syncthreads();
  if (s_flag) {
    for (int i = tid; i < p.experts; i += kThreads) p.ready[i] = 0;
    for (int i = tid; i < tiles_1; i += kThreads) p.tile_done[i] = 0;
    if (tid == 0) *p.blocks_done = 0;
  }
}

template <int G, int NT, bool F32>
cudaError_t launch(const MoeParams& p, int num_sms, cudaStream_t s) {
  using S = Shape<G, NT>;
  static std::atomic<uint64_t> ready{0};   // devices on which the shared-memory limit is raised
  const int bytes = S::kRing + 2 * S::kRed + lists_bytes(p.n * p.topk);
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) & bit)) {
    if (const cudaError_t e = cudaFuncSetAttribute(moe_kernel<G, NT, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        e != cudaSuccess)
      return e;
    if (dev < 64) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = s;
  // Every block resident: the waits on other blocks end.  (Programmatic launch beside it
  // was measured and changes nothing: the grid needs every SM's shared memory, so it
  // starts when the one before it ends.)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel<G, NT, F32>, p);
}

// One column tile a job for few tokens, which leaves the ring longer: for 4-bit weights
// up to 8 tokens (128 experts of 4096 x 1408, 8 tokens: 105 us, with two tiles 137), for
// bf16 up to the 4 that a down job then holds (64 experts of 7168 x 2048, 1 token: 111
// us, with two tiles 113; 8 tokens: 528 and 519 us).
template <int G>
cudaError_t launch_g(const MoeParams& p, int num_sms, cudaStream_t s) {
  if (p.n <= (G != 0 ? 8 : 4)) return p.out_f32 ? launch<G, 1, true>(p, num_sms, s) : launch<G, 1, false>(p, num_sms, s);
  return p.out_f32 ? launch<G, 2, true>(p, num_sms, s) : launch<G, 2, false>(p, num_sms, s);
}

}  // namespace

cudaError_t LaunchMoe(const MoeParams& p, int num_sms, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  switch (p.group) {
    case 0: return launch_g<0>(p, num_sms, s);
    case 32: return launch_g<32>(p, num_sms, s);
    case 64: return launch_g<64>(p, num_sms, s);
    default: return launch_g<128>(p, num_sms, s);
  }
}

}  // namespace epg
