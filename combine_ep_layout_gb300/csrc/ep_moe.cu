// ep_moe.cu -- the experts of a few tokens in one launch (include/ep_gb300_moe.h:
// ep_moe_forward).
//
// What bounds it: every active expert's 3 H I weights are read once (a token's
// own rows are a few KB), so the work is to keep HBM busy from the first byte to
// the last.  A persistent grid, one block of 8 warps per SM, walks one list of
// items: first the gate/up items (expert, 16 or 32 channels: the gate's and the
// up projection's rows together, so that the product act(gate) up is formed where
// the sums are), then the down items (expert, 32 or 64 output channels).  The 8
// warps split an item's k range chunk by chunk and add their sums through shared
// memory; each warp streams its own chunks through its own cp.async ring
// (ep_stream.cuh) across items and phases, so the ring never drains.
//
// A down item needs its expert's whole h: a counter per active expert, raised by
// each finished gate/up item, is waited for (bounded) just before the item's
// activations are copied; its weights are under way by then.  Experts come in one
// order in both phases, so the wait is short unless few experts are active.
//
// h is kept as two bf16, h = hi + lo (16 significant bits), in two columns of the
// down product whose sums are added: a column costs nothing until 4 tokens meet
// on an expert, and the rounding of h to 8 bits would double the output's error.
//
// The down items write fp32 expert rows; the block that finishes the last item of
// a channel tile folds the K rows of each token in order (fmaf over k, as the
// combine does).  No sum depends on the order of blocks: equal inputs, equal bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ep_moe_kernels.hpp"
#include "ep_stream.cuh"
#include "ep_types.cuh"

namespace epg {
namespace {

using stream::Form;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Row tiles of an item: bf16 32 rows, 4-bit 64.
template <int G>
using MoeForm = Form<G, G == 0 ? 2 : 4>;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSmemLimit = 232448 - 256;  // dynamic shared memory of one block (its static part aside)

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

// A job: some tokens (at most the phase's cap) of one active expert.
struct Job {
  uint16_t expert, active, start, count;
};

// Shared memory behind the rings, sized by the number of entries n K.
struct Lists {
  Job *jobs_0, *jobs_1;
  float* weight;       // by entry
  uint16_t* entry;     // entries grouped by expert, ascending within one
  uint16_t* token;     // entry / K
  uint16_t* parts;     // by active expert: its gate/up jobs
  uint8_t* valid;      // by entry
};

constexpr int lists_bytes(int entries) { return ((entries * (2 * 8 + 4 + 3 * 2 + 1) + 15) & ~15) + 16; }

template <int G, int NT>
struct Shape {
  using F = MoeForm<G>;
  static constexpr int kTokens = NT == 1 ? 8 : kFewTokens;   // most tokens of a call
  static constexpr int kRed = kWarps * F::kRows * 10 * 4;    // partial sums of one column tile
  static constexpr int kSlot = F::stage_bytes(NT);
  static constexpr int kFit = (kSmemLimit - kRed - lists_bytes(kTokens * 16)) / (kWarps * kSlot);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kRing = kWarps * kStages * kSlot;
  static_assert(kStages >= 2);
  // the expert counts of the set-up (2048 x 4 bytes) and the ranks use the ring
  static_assert(kRing >= 4 * 2048 + 2 * 1024 + 2 * 1024);
};

template <int G, int NT>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const MoeParams p) {
  using F = MoeForm<G>;
  using S = Shape<G, NT>;
  constexpr int RT = F::kRowTiles, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t scan_warp[kWarps];
  __shared__ int s_flag, s_lost;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int entries = p.n * p.topk;
  float* red = reinterpret_cast<float*>(smem + S::kRing);
  Lists L;
  {
    uint8_t* b = smem + S::kRing + S::kRed;
    L.jobs_0 = reinterpret_cast<Job*>(b);
    L.jobs_1 = L.jobs_0 + entries;
    L.weight = reinterpret_cast<float*>(L.jobs_1 + entries);
    L.entry = reinterpret_cast<uint16_t*>(L.weight + entries);
    L.token = L.entry + entries;
    L.parts = L.token + entries;
    L.valid = reinterpret_cast<uint8_t*>(L.parts + entries);
  }

  // ---- which experts, with which tokens: every block works it out for itself
  int* count = reinterpret_cast<int*>(smem);                              // by expert
  uint16_t* expert_of = reinterpret_cast<uint16_t*>(smem + 4 * 2048);     // by entry
  uint16_t* rank_of = expert_of + 1024;
  if (tid == 0) s_lost = 0;
  for (int e = tid; e < p.experts; e += kThreads) count[e] = 0;
  __syncthreads();
  if (warp == 0) {   // one warp in entry order: the order within an expert is the same in every block
    for (int i0 = 0; i0 < entries; i0 += 32) {
      const int i = i0 + lane;
      int64_t id = -1;
      if (i < entries) id = p.topk_idx[i];
      const bool ok = id >= 0 && id < p.experts;
      if (i < entries && !ok && id != -1 && blockIdx.x == 0) atomicOr(p.err, kErrBadExpert);
      const int e = ok ? static_cast<int>(id) : -1 - lane;
      const unsigned same = __match_any_sync(kAll, e);
      const int before = ok ? count[e] : 0;
      __syncwarp();
      if (ok && (same >> lane) == 1u) count[e] = before + __popc(same);   // the last of the equal ones
      __syncwarp();
      if (i < entries) {
        expert_of[i] = ok ? static_cast<uint16_t>(e) : 0xffff;
        rank_of[i] = static_cast<uint16_t>(before + __popc(same & ((1u << lane) - 1u)));
        L.valid[i] = ok;
      }
    }
  }
  __syncthreads();
  int jobs_0, jobs_1, actives;
  {
    // four 16-bit sums in one word: entries, active experts, gate/up jobs, down jobs
    const int per = (p.experts + kThreads - 1) / kThreads, e0 = tid * per;
    const int e1 = min(e0 + per, p.experts);
    auto word = [](int c) -> uint64_t {
      return c == 0 ? 0
                    : static_cast<uint64_t>(c) | 1ull << 16 | static_cast<uint64_t>((c + 8 * NT - 1) / (8 * NT)) << 32 |
                          static_cast<uint64_t>((c + 4 * NT - 1) / (4 * NT)) << 48;
    };
    uint64_t mine = 0;
    for (int e = e0; e < e1; ++e) mine += word(count[e]);
    uint64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t v = __shfl_up_sync(kAll, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31) scan_warp[warp] = upto;
    __syncthreads();
    uint64_t base = upto - mine, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += scan_warp[w];
      all += scan_warp[w];
    }
    actives = static_cast<int>(all >> 16 & 0xffff);
    jobs_0 = static_cast<int>(all >> 32 & 0xffff);
    jobs_1 = static_cast<int>(all >> 48);
    for (int e = e0; e < e1; ++e) {
      const int c = count[e];
      if (c == 0) continue;
      const int start = static_cast<int>(base & 0xffff), active = static_cast<int>(base >> 16 & 0xffff);
      for (int ph = 0; ph < 2; ++ph) {
        const int cap = ph == 0 ? 8 * NT : 4 * NT;
        int j = static_cast<int>(base >> (32 + 16 * ph) & 0xffff);
        if (ph == 0) L.parts[active] = static_cast<uint16_t>((c + cap - 1) / cap);
        for (int o = 0; o < c; o += cap, ++j)
          (ph == 0 ? L.jobs_0 : L.jobs_1)[j] = {static_cast<uint16_t>(e), static_cast<uint16_t>(active), static_cast<uint16_t>(start + o),
                           static_cast<uint16_t>(min(cap, c - o))};
      }
      base += word(c);
      count[e] = start;
    }
  }
  __syncthreads();
  for (int i = tid; i < entries; i += kThreads) {
    const int e = expert_of[i];
    if (e != 0xffff) {
      const int at = count[e] + rank_of[i];
      L.entry[at] = static_cast<uint16_t>(i);
      L.token[at] = static_cast<uint16_t>(i / p.topk);
      L.weight[i] = p.topk_weights[i];
    }
  }
  __syncthreads();   // the ring's memory is free from here on

  // ---- the list of items and this warp's walk through it
  // (pick: by phase, without arrays that would have to live in memory)
  auto pick = [](int ph, auto a, auto b) { return ph == 0 ? a : b; };
  auto dim_k = [&](int ph) { return pick(ph, p.hidden, p.inter); };       // columns of the weight rows
  const int tiles_0 = (p.inter + F::kRows / 2 - 1) / (F::kRows / 2), tiles_1 = (p.hidden + F::kRows - 1) / F::kRows;
  auto tiles = [&](int ph) { return pick(ph, tiles_0, tiles_1); };
  auto jobs_of = [&](int ph) { return pick(ph, jobs_0, jobs_1); };
  auto job_at = [&](int ph, int j) { return pick(ph, L.jobs_0, L.jobs_1)[j]; };
  const int grid = gridDim.x;
  // this block's first item of each phase: the down items go on where the gate/up items ended
  const int first_1 = (static_cast<int>(blockIdx.x) - jobs_0 * tiles_0 % grid + grid) % grid;
  auto first = [&](int ph) { return pick(ph, static_cast<int>(blockIdx.x), first_1); };
  const int chunks_0 = (p.hidden + F::kCols - 1) / F::kCols, chunks_1 = (p.inter + F::kCols - 1) / F::kCols;
  auto chunks = [&](int ph) { return pick(ph, chunks_0, chunks_1); };

  const uint32_t ring = stream::smem_addr(smem) + warp * kStages * S::kSlot;
  const bool wide_0 = F::kInt4 && p.hidden % 128 == 0 && (reinterpret_cast<uintptr_t>(p.w13_scales) & 15) == 0;
  const bool wide_1 = F::kInt4 && p.inter % 128 == 0 && (reinterpret_cast<uintptr_t>(p.w2_scales) & 15) == 0;

  // A walk: the chunk c of an item (job, tile) of a phase.
  struct Walk {
    int ph, job, tile, c;
  };
  auto settle = [&](Walk& w) {   // to a chunk that exists: over item ends, and phases without work for this warp
    while (w.ph < 2) {
      while (w.tile >= tiles(w.ph)) w.tile -= tiles(w.ph), ++w.job;
      if (w.job < jobs_of(w.ph) && w.c < chunks(w.ph)) return;
      ++w.ph;
      if (w.ph < 2) w.job = 0, w.tile = first(w.ph), w.c = warp;
    }
  };
  // the weights' part of a stage
  uint32_t row_off[F::kCopies];   // of the rows this lane copies, in 16-byte units from the expert's matrix
  auto channel_row = [&](int ph, int tile, int r) {
    if (ph == 1) return min(tile * F::kRows + r, p.hidden - 1);
    const int half = F::kRows / 2;
    const int ch = min(tile * half + (r < half ? r : r - half), p.inter - 1);
    return r < half ? ch : p.inter + ch;
  };
  auto enter_item = [&](const Walk& w) {
    if (w.ph > 1) return;
    const int pieces = dim_k(w.ph) / F::kPerPiece;
#pragma unroll
    for (int i = 0; i < F::kCopies; ++i) {
      const int r = lane / F::kPieces + i * (32 / F::kPieces);
      row_off[i] = static_cast<uint32_t>(channel_row(w.ph, w.tile, r)) * static_cast<uint32_t>(pieces);
    }
  };
  const uint32_t a_dst = F::a_offset(lane / F::kPieces, lane % F::kPieces);
  auto copy_weights = [&](const Walk& w, uint32_t slot) {
    const int pieces = dim_k(w.ph) / F::kPerPiece;
    const int64_t rows = w.ph == 0 ? 2 * p.inter : p.hidden;
    const int e = job_at(w.ph, w.job).expert;
    const uint8_t* base = static_cast<const uint8_t*>(w.ph == 0 ? p.w13 : p.w2) + e * rows * pieces * 16;
    const int piece = w.c * F::kPieces + lane % F::kPieces;
    const bool ok = piece < pieces;
    const uint8_t* src = base + (ok ? piece * 16 : 0);
#pragma unroll
    for (int i = 0; i < F::kCopies; ++i)
      stream::copy16(slot + a_dst + i * (32 / F::kPieces) * F::kRowBytes, src + static_cast<uint64_t>(row_off[i]) * 16, ok);
    if constexpr (F::kInt4) {
      const float* sc = (w.ph == 0 ? p.w13_scales : p.w2_scales) + e * rows * (dim_k(w.ph) / G);
      stream::copy_scales<G, RT>(slot, lane, sc, dim_k(w.ph), w.c, pick(w.ph, wide_0, wide_1),
                             [&](int r) { return channel_row(w.ph, w.tile, r); });
    }
  };
  // the activations' part: the job's columns (phase 1: the hi and the lo row of each entry)
  auto copy_columns = [&](const Walk& w, uint32_t slot) {
    const Job job = job_at(w.ph, w.job);
    const int k = dim_k(w.ph);
    const int cols = w.ph == 0 ? job.count : 2 * job.count;
    for (int q = lane; q < cols * F::kXPieces; q += 32) {
      const int col = q / F::kXPieces, c = q % F::kXPieces;
      const int at = w.c * F::kCols + 8 * c;
      const __nv_bfloat16* src =
          w.ph == 0 ? static_cast<const __nv_bfloat16*>(p.x) + static_cast<int64_t>(L.token[job.start + col]) * k
                    : static_cast<const __nv_bfloat16*>(p.h) +
                          (2 * static_cast<int64_t>(L.entry[job.start + (col >> 1)]) + (col & 1)) * k;
      stream::copy16(slot + F::x_offset(col, c), src + (at < k ? at : 0), at < k);
    }
  };
  // until every gate/up item of the job's expert is done; gives up after wait_ns
  auto await_expert = [&](const Walk& w) {
    const Job job = job_at(1, w.job);
    const int want = tiles_0 * L.parts[job.active];
    if (lane == 0 && load_acquire(p.ready + job.active) < want && !*static_cast<volatile int*>(&s_lost)) {
      const uint64_t t0 = now_ns();
      while (load_acquire(p.ready + job.active) < want) {
        if (now_ns() - t0 > p.wait_ns) {
          *static_cast<volatile int*>(&s_lost) = 1;
          atomicOr(p.err, kErrTimeout);
          break;
        }
      }
    }
    __syncwarp();
  };

  Walk pf{0, 0, first(0), warp};
  settle(pf);
  enter_item(pf);
  int ahead = 0;           // stages of phase 1 whose weights are under way without their columns
  int phase = 0, awaited = -1;
  auto issue = [&](int slot_index) {
    if (pf.ph < 2) {
      const uint32_t slot = ring + slot_index * S::kSlot;
      copy_weights(pf, slot);
      if (pf.ph == phase) {
        if (phase == 1 && pf.job != awaited) await_expert(pf), awaited = pf.job;
        copy_columns(pf, slot);
      } else {
        ++ahead;
      }
      const int ph = pf.ph, job = pf.job, tile = pf.tile;
      pf.c += kWarps;
      if (pf.c >= chunks(ph)) pf.c = warp, pf.tile += grid;
      settle(pf);
      if (pf.ph != ph || pf.job != job || pf.tile != tile) enter_item(pf);
    }
    stream::commit();
  };
  int in = 0, out = 0;     // ring positions of the next stage to fill and to use
  for (int s = 0; s < kStages - 1; ++s) issue(in), ++in;

  for (phase = 0; phase < 2; ++phase) {
    if (phase == 1 && ahead > 0) {
      Walk w{1, 0, first(1), warp};
      settle(w);
      int slot = out;
      for (int s = 0; s < ahead; ++s) {
        if (w.job != awaited) await_expert(w), awaited = w.job;
        copy_columns(w, ring + slot * S::kSlot);
        slot = slot + 1 == kStages ? 0 : slot + 1;
        w.c += kWarps;
        if (w.c >= chunks_1) w.c = warp, w.tile += grid;
        settle(w);
      }
      stream::commit();
      stream::wait<0>();
      __syncwarp();
    }
    const int mine = warp < chunks(phase) ? (chunks(phase) - warp + kWarps - 1) / kWarps : 0;
    int job_i = 0, tile = first(phase);
    for (;; tile += grid) {
      while (tile >= tiles(phase)) tile -= tiles(phase), ++job_i;
      if (job_i >= jobs_of(phase)) break;
      const Job job = job_at(phase, job_i);
      const int cols = phase == 0 ? job.count : 2 * job.count;
      const int nts = (cols + 7) >> 3;
      float acc[RT][NT][4];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][nt][i] = 0.0f;
      for (int j = 0; j < mine; ++j) {
        stream::wait<kStages - 2>();
        __syncwarp();      // every lane's copies of this stage, and every lane done with the slot refilled next
        issue(in);
        in = in + 1 == kStages ? 0 : in + 1;
        const uint32_t slot = ring + out * S::kSlot;
        out = out + 1 == kStages ? 0 : out + 1;
        if (NT == 1 || nts == 1)
          stream::consume<G, RT, 1, NT>(slot, lane, acc);
        else if (NT == 2 || nts == 2)
          stream::consume<G, RT, NT < 2 ? NT : 2, NT>(slot, lane, acc);
        else
          stream::consume<G, RT, NT, NT>(slot, lane, acc);
      }
      // the warps' sums, one column tile at a time
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt >= nts) break;
        if (phase == 0) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float* r0 = red + (warp * F::kRows + 16 * rt + g) * 10 + 2 * t;
            *reinterpret_cast<float2*>(r0) = make_float2(acc[rt][nt][0], acc[rt][nt][1]);
            *reinterpret_cast<float2*>(r0 + 80) = make_float2(acc[rt][nt][2], acc[rt][nt][3]);
          }
          __syncthreads();
          constexpr int kCh = F::kRows / 2;
          const int ch = tid % kCh, col = tid / kCh;
          const int i = tile * kCh + ch;
          if (col < 8 && 8 * nt + col < cols && i < p.inter) {
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              gate += red[(w * F::kRows + ch) * 10 + col];
              up += red[(w * F::kRows + kCh + ch) * 10 + col];
            }
            const float h = activate(gate, p.act) * up;
            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
            // an infinite or NaN h has nothing below it
            const float rest = h - __bfloat162float(hi);
            const __nv_bfloat16 lo = __float2bfloat16_rn(rest == rest && fabsf(rest) < INFINITY ? rest : 0.0f);
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.h) +
                                 2 * static_cast<int64_t>(L.entry[job.start + 8 * nt + col]) * p.inter + i;
            dst[0] = hi;
            dst[p.inter] = lo;
          }
        } else {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float* r0 = red + (warp * F::kRows + 16 * rt + g) * 4 + t;
            r0[0] = acc[rt][nt][0] + acc[rt][nt][1];
            r0[32] = acc[rt][nt][2] + acc[rt][nt][3];
          }
          __syncthreads();
          const int r = tid % F::kRows, tok = tid / F::kRows;
          const int c = tile * F::kRows + r;
          if (tok < 4 && 4 * nt + tok < job.count && c < p.hidden) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[(w * F::kRows + r) * 4 + tok];
            p.part[static_cast<int64_t>(L.entry[job.start + 4 * nt + tok]) * p.hidden + c] = v;
          }
        }
        __syncthreads();   // the sums' memory is free, the results are written
      }
      if (phase == 0) {
        if (tid == 0) {
          __threadfence();
          atomicAdd(p.ready + job.active, 1);
        }
      } else {
        if (tid == 0) {
          __threadfence();
          s_flag = atomicAdd(p.tile_done + tile, 1) == jobs_1 - 1;
          __threadfence();
        }
        __syncthreads();
        if (s_flag) {      // the tile's last item: fold every token's K rows
          constexpr int kTok = kThreads / F::kRows;
          const int c = tile * F::kRows + tid % F::kRows;
          if (c < p.hidden) {
            for (int tok = tid / F::kRows; tok < p.n; tok += kTok) {
              float sum = 0.0f;
              for (int k = 0; k < p.topk; ++k) {
                const int en = tok * p.topk + k;
                if (L.valid[en])
                  sum = fmaf(L.weight[en], __ldcg(p.part + static_cast<int64_t>(en) * p.hidden + c), sum);
              }
              const int64_t o = static_cast<int64_t>(tok) * p.hidden + c;
              if (p.bias) sum += __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[o]);
              if (p.out_f32)
                static_cast<float*>(p.out)[o] = sum;
              else
                static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(sum);
            }
          }
        }
        __syncthreads();   // s_flag may change again
      }
    }
  }
  stream::wait<0>();
  if (jobs_1 == 0) {   // every entry masked
    const int64_t total = static_cast<int64_t>(p.n) * p.hidden;
    for (int64_t o = static_cast<int64_t>(blockIdx.x) * kThreads + tid; o < total; o += static_cast<int64_t>(grid) * kThreads) {
      const float v = p.bias ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[o]) : 0.0f;
      if (p.out_f32)
        static_cast<float*>(p.out)[o] = v;
      else
        static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
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
    for (int i = tid; i < actives; i += kThreads) p.ready[i] = 0;
    for (int i = tid; i < tiles_1; i += kThreads) p.tile_done[i] = 0;
    if (tid == 0) *p.blocks_done = 0;
  }
}

template <int G, int NT>
cudaError_t launch(const MoeParams& p, int num_sms, cudaStream_t s) {
  using S = Shape<G, NT>;
  const int bytes = S::kRing + S::kRed + lists_bytes(p.n * p.topk);
  if (const cudaError_t e = cudaFuncSetAttribute(moe_kernel<G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
      e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;   // every block resident: the waits on other blocks end
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel<G, NT>, p);
}

template <int G>
cudaError_t launch_g(const MoeParams& p, int num_sms, cudaStream_t s) {
  if (p.n <= 8) return launch<G, 1>(p, num_sms, s);
  if constexpr (G == 0) {
    if (p.n > 16) return launch<G, 4>(p, num_sms, s);
  }
  return launch<G, 2>(p, num_sms, s);
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
