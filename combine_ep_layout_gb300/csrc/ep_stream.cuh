// ep_stream.cuh -- the inner part of the products that stream a weight matrix
// past a few activation columns: one warp multiplies a tile of weight rows with
// up to 8 NT columns, stage by stage, from its own ring in shared memory.
//
// The weights are the wide operand (16 rows of one mma.m16n8k16), the tokens
// the narrow one (8 columns), so a single token costs one eighth-filled column
// tile and no weight is read twice.  A product over k does not care in which
// order k is visited as long as both operands agree, so each lane takes 16
// consecutive bytes of a row where the instruction's fragment would ask for
// scattered pairs.
//
//   form     columns per stage   bytes per row and stage
//   bf16            64                  128
//   4-bit          128                   64
//
// Everything moves by cp.async (16 bytes a lane, zero-filled past the end of a
// row), from a warp to itself: no barrier between warps, no wait that could hang.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace epg {
namespace stream {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes to shared memory past L1; zeros where !ok (src is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(ok ? BYTES : 0)
               : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread have landed.
template <int N>
__device__ __forceinline__ void wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Plain loads of shared memory (pointers into it), which the compiler may move
// ahead of the arithmetic before them but not past the waits above.
__device__ __forceinline__ uint4 load16(const uint8_t* at) { return *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ uint32_t load4(const uint8_t* at) { return *reinterpret_cast<const uint32_t*>(at); }

// d += a b: a 16x16 bf16 (row major fragments), b 16x8 bf16, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Nibbles become bf16 operands by a mask and an fma.  The bf16 codes 0 to 255 are the
// values code * 2^-133 (subnormals, and the first binade goes on at their spacing), so a
// nibble q in bits 0-3 of a half word is q 2^-133 as it stands, and one in bits 4-7 is
// 16 q 2^-133.  Times 2^127, or 2^123, less 2^-3, both are (q - 8) 2^-6, exactly: 9
// instructions for eight weights (masks, one shift, four fma).  The unit goes into the
// group's scale.  Every product with an activation is exact in fp32, subnormal activations
// too, and infinite ones give what they give in fp32.  Or-ing an exponent and subtracting
// 136 takes 11 instructions (7168 x 7168, 1 token: 9.8 us, this 9.3; 20011 x 4096, 13 tokens:
// 20.6 and 20.0; MoE layer, 8 tokens, 128 experts of 4096 x 1408: 107 and 105).  Leaving q
// in place and subtracting 8 times the sum of the activations afterwards takes 5, but the
// two cancel: bits are lost wherever the activations share a sign.
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
constexpr uint32_t kLiftLow = 0x7f007f00u, kLiftHigh = 0x7d007d00u;   // 2^127, 2^123
constexpr float kUnit = 64.0f;

__device__ __forceinline__ uint32_t nibble_pair(uint32_t masked, uint32_t lift) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(masked), "r"(lift), "r"(0xbe00be00u));   // -2^-3
  return r;
}

// G: 0 for bf16 weights, else the group size of the 4-bit form.  RT: row tiles of 16.
template <int G, int RT>
struct Form {
  static constexpr bool kInt4 = G != 0;
  static constexpr int kRowTiles = RT;
  static constexpr int kRows = 16 * kRowTiles;
  static constexpr int kCols = kInt4 ? 128 : 64;          // columns of one stage
  static constexpr int kPerPiece = kInt4 ? 32 : 8;        // columns in 16 bytes of weights
  static constexpr int kPieces = kCols / kPerPiece;       // 16-byte pieces of a weight row in a stage
  static constexpr int kRowBytes = 16 * kPieces;
  static constexpr int kABytes = kRows * kRowBytes;
  static constexpr int kScales = kInt4 ? kCols / (kInt4 ? G : 1) : 0;   // of a row in a stage
  static constexpr int kSBytes = kRows * kScales * 4;
  static constexpr int kXPieces = kCols / 8;              // 16-byte pieces of an activation column
  static constexpr int kXBytes = 2 * kCols;
  static constexpr int kCopies = kRows * kPieces / 32;    // weight pieces each lane copies

  static constexpr int stage_bytes(int nt) { return kABytes + kSBytes + 8 * nt * kXBytes; }

  // Where piece c of weight row r lies in a stage: the 8 rows that a quarter
  // of the reading lanes touch fall on different banks.
  __device__ static __forceinline__ uint32_t a_offset(int r, int c) {
    return static_cast<uint32_t>(r * kRowBytes + 16 * (kInt4 ? c ^ ((r >> 1) & 3) : c ^ ((r & 1) << 2)));
  }
  // Where piece c of activation column col lies, from the columns' start and from
  // the stage's (weights, scales, columns).
  __device__ static __forceinline__ uint32_t x_at(int col, int c) {
    return static_cast<uint32_t>(col * kXBytes + 16 * (c ^ ((col & 1) << 2)));
  }
  __device__ static __forceinline__ uint32_t x_offset(int col, int c) { return kABytes + kSBytes + x_at(col, c); }
};

// acc[rt][nt] += tile rows (16 rt + ...) times columns (8 nt + ...) of a stage: weights
// and scales at `slot`, columns at `cols`.
template <int G, int RT, int NT, int CAP>
__device__ __forceinline__ void consume_at(const uint8_t* slot, const uint8_t* cols, int lane, float (&acc)[RT][CAP][4]) {
  using F = Form<G, RT>;
  const int g = lane >> 2, t = lane & 3;
  if constexpr (!F::kInt4) {
#pragma unroll
    for (int kk = 0; kk < F::kCols / 32; ++kk) {
      uint4 lo[F::kRowTiles], hi[F::kRowTiles];
#pragma unroll
      for (int rt = 0; rt < F::kRowTiles; ++rt) {
        lo[rt] = load16(slot + F::a_offset(16 * rt + g, 4 * kk + t));
        hi[rt] = load16(slot + F::a_offset(16 * rt + g + 8, 4 * kk + t));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 x = load16(cols + F::x_at(8 * nt + g, 4 * kk + t));
#pragma unroll
        for (int rt = 0; rt < F::kRowTiles; ++rt) {
          mma(acc[rt][nt], lo[rt].x, hi[rt].x, lo[rt].y, hi[rt].y, x.x, x.y);
          mma(acc[rt][nt], lo[rt].z, hi[rt].z, lo[rt].w, hi[rt].w, x.z, x.w);
        }
      }
    }
  } else {
    // 8 columns of a lane are one word of nibbles; masking pairs nibble i with
    // nibble i + 4, and the activations are paired the same way.
#pragma unroll
    for (int grp = 0; grp < F::kScales; ++grp) {
      float sum[F::kRowTiles][NT][4];
#pragma unroll
      for (int q = grp * (G / 32); q < (grp + 1) * (G / 32); ++q) {
        const bool first = q == grp * (G / 32);
        uint32_t b[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 x = load16(cols + F::x_at(8 * nt + g, 4 * q + t));
          b[nt][0] = __byte_perm(x.x, x.z, 0x5410);
          b[nt][1] = __byte_perm(x.x, x.z, 0x7632);
          b[nt][2] = __byte_perm(x.y, x.w, 0x5410);
          b[nt][3] = __byte_perm(x.y, x.w, 0x7632);
        }
#pragma unroll
        for (int rt = 0; rt < F::kRowTiles; ++rt) {
          const uint32_t lo = load4(slot + F::a_offset(16 * rt + g, q) + 4 * t);
          const uint32_t hi = load4(slot + F::a_offset(16 * rt + g + 8, q) + 4 * t);
          uint32_t a[8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[4 * i] = nibble_pair(lo >> 8 * i & kLow, kLiftLow), a[4 * i + 1] = nibble_pair(hi >> 8 * i & kLow, kLiftLow);
            a[4 * i + 2] = nibble_pair(lo >> 8 * i & kHigh, kLiftHigh), a[4 * i + 3] = nibble_pair(hi >> 8 * i & kHigh, kLiftHigh);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (first)
              mma_first(sum[rt][nt], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
            else
              mma(sum[rt][nt], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
            mma(sum[rt][nt], a[4], a[5], a[6], a[7], b[nt][2], b[nt][3]);
          }
        }
      }
#pragma unroll
      for (int rt = 0; rt < F::kRowTiles; ++rt) {
        const float s0 = kUnit * __uint_as_float(load4(slot + F::kABytes + 4 * ((16 * rt + g) * F::kScales + grp)));
        const float s1 = kUnit * __uint_as_float(load4(slot + F::kABytes + 4 * ((16 * rt + g + 8) * F::kScales + grp)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[rt][nt][0] = fmaf(s0, sum[rt][nt][0], acc[rt][nt][0]);
          acc[rt][nt][1] = fmaf(s0, sum[rt][nt][1], acc[rt][nt][1]);
          acc[rt][nt][2] = fmaf(s1, sum[rt][nt][2], acc[rt][nt][2]);
          acc[rt][nt][3] = fmaf(s1, sum[rt][nt][3], acc[rt][nt][3]);
        }
      }
    }
  }
}

template <int G, int RT, int NT, int CAP>
__device__ __forceinline__ void consume(const uint8_t* slot, int lane, float (&acc)[RT][CAP][4]) {
  consume_at<G, RT, NT, CAP>(slot, slot + Form<G, RT>::x_offset(0, 0), lane, acc);
}

// Copy the scales of stage c one by one: kScales of each of the tile's rows,
// zeros past the end of a row.  `row_of(r)` gives the matrix row of tile row r.
template <int G, int RT, class RowOf>
__device__ __forceinline__ void copy_scales(uint32_t slot, int lane, const float* scales, int cols, int c,
                                            RowOf row_of) {
  using F = Form<G, RT>;
  const int groups = cols / G;
#pragma unroll 1
  for (int p = lane; p < F::kRows * F::kScales; p += 32) {
    const int r = p / F::kScales, s = c * F::kScales + p % F::kScales;
    const float* src = scales + static_cast<int64_t>(row_of(r)) * groups;
    copy_small<4>(slot + F::kABytes + 4 * p, src + (s < groups ? s : 0), s < groups);
  }
}

// One row's scales of a stage at once (aligned to BYTES).
template <int BYTES>
__device__ __forceinline__ void copy_wide(uint32_t dst, const float* src) {
  if constexpr (BYTES == 16)
    copy16(dst, src, true);
  else
    copy_small<BYTES>(dst, src, true);
}

}  // namespace stream
}  // namespace epg
