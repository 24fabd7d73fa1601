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

// Nibbles become bf16 operands in one of two ways.
//
// Lifted: the bf16 codes 0 to 255 are the values code * 2^-133 (subnormals, and the
// first binade goes on at their spacing), and the matrix instruction takes them as
// such.  So a nibble q in bits 0-3 of a half word is already q * 2^-133, and one in
// bits 4-7 is 16 q * 2^-133: masks and one shift, 5 instructions, make the operands
// of eight weights.  The activations carry the rest: times 2^90, the odd columns (bits
// 4-7) times 2^86, exact in bf16 for magnitudes below 2^38.  (A larger one becomes
// infinite and its offset as well, so the sum is NaN: see plain_dot.)  The sums' last
// bit is then worth 2^-149 2^43 = 2^-106: activations of 2^-80 lose nothing yet.  The
// offset of 8 is a product too: a row of -8 for every column, the same for all rows,
// added to each group's sums before its scale.  That is 4 instructions and a matrix
// instruction for each 8 activations.
//
// Plain: or-ing an exponent makes the bf16 128 + q, subtracting 136 leaves q - 8: 11
// instructions for eight weights, none for the activations.
//
// Lifted wins where few columns meet many rows (one column tile: 5 tokens over 128
// experts of 4096 x 1408, 115 -> 106 us), plain where one row tile meets many
// columns (32 tokens, 4096 x 14336: 30 -> 23 us).
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;
constexpr float kUnit = 8796093022208.0f;   // 2^43: what sums of such products are to be multiplied by

// (L2's value: it may be another block's, written since this one began)
__device__ __forceinline__ float load_bf16(const __nv_bfloat16* at) {
  return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(at))) << 16);
}
// A row of 4-bit weights times x (+ x_lo where given), product by product: what a
// value is that came out NaN above, be it from activations of 2^38 and more, from
// infinite ones, whose products have each its own sign, or from a NaN.
static __device__ __noinline__ float plain_dot(const uint8_t* q, const float* scales, const __nv_bfloat16* x,
                                               const __nv_bfloat16* x_lo, int cols, int group) {
  float sum = 0.0f;
  for (int c0 = 0; c0 < cols && !(sum != sum); c0 += group) {
    float part = 0.0f;
    for (int c = c0; c < c0 + group; ++c) {
      const int nibble = q[c / 2] >> (4 * (c & 1)) & 15;
      const float v = load_bf16(x + c) + (x_lo ? load_bf16(x_lo + c) : 0.0f);
      part = fmaf(static_cast<float>(nibble - 8), v, part);
    }
    sum = fmaf(scales[c0 / group], part, sum);
  }
  return sum;
}

// Two of a word's nibbles (bits 0-3 and 16-19 of v) as bf16 values nibble - 8.
__device__ __forceinline__ uint32_t nibble_pair(uint32_t v) {
  uint32_t u;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(u) : "r"(v));
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                   __nv_bfloat162(__float2bfloat16(136.0f), __float2bfloat16(136.0f)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Two neighbouring activations (even and odd column) as operands.
__device__ __forceinline__ uint32_t lift(uint32_t x) {
  const uint32_t by = 0x6a806c80u;                  // 2^86 (odd), 2^90 (even)
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(by));
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

  static constexpr float kOut = kInt4 ? kUnit : 1.0f;     // what sums are to be multiplied by

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

// acc[rt][nt] += tile rows (16 rt + ...) times columns (8 nt + ...) of a stage (lifted
// 4-bit weights: in units of 1 / kUnit): weights and scales at `slot`, columns at `cols`.
template <int G, int RT, int NT, int CAP, bool LIFT = true>
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
      [[maybe_unused]] float offset[NT][4];
#pragma unroll
      for (int q = grp * (G / 32); q < (grp + 1) * (G / 32); ++q) {
        const bool first = q == grp * (G / 32);
        uint32_t b[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint4 x = load16(cols + F::x_at(8 * nt + g, 4 * q + t));
          if constexpr (LIFT) x.x = lift(x.x), x.y = lift(x.y), x.z = lift(x.z), x.w = lift(x.w);
          b[nt][0] = __byte_perm(x.x, x.z, 0x5410);
          b[nt][1] = __byte_perm(x.x, x.z, 0x7632);
          b[nt][2] = __byte_perm(x.y, x.w, 0x5410);
          b[nt][3] = __byte_perm(x.y, x.w, 0x7632);
          if constexpr (LIFT) {
            if (first)
              mma_first(offset[nt], kMinus8, kMinus8, kMinus128, kMinus128, b[nt][0], b[nt][1]);
            else
              mma(offset[nt], kMinus8, kMinus8, kMinus128, kMinus128, b[nt][0], b[nt][1]);
            mma(offset[nt], kMinus8, kMinus8, kMinus128, kMinus128, b[nt][2], b[nt][3]);
          }
        }
#pragma unroll
        for (int rt = 0; rt < F::kRowTiles; ++rt) {
          const uint32_t lo = load4(slot + F::a_offset(16 * rt + g, q) + 4 * t);
          const uint32_t hi = load4(slot + F::a_offset(16 * rt + g + 8, q) + 4 * t);
          uint32_t a[8];
          if constexpr (LIFT) {
            const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
            a[0] = lo & kLow, a[1] = hi & kLow, a[2] = lo & kHigh, a[3] = hi & kHigh;
            a[4] = lo8 & kLow, a[5] = hi8 & kLow, a[6] = lo8 & kHigh, a[7] = hi8 & kHigh;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[2 * i] = nibble_pair(lo >> 4 * i), a[2 * i + 1] = nibble_pair(hi >> 4 * i);
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
        const float s0 = __uint_as_float(load4(slot + F::kABytes + 4 * ((16 * rt + g) * F::kScales + grp)));
        const float s1 = __uint_as_float(load4(slot + F::kABytes + 4 * ((16 * rt + g + 8) * F::kScales + grp)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[rt][nt][0] = fmaf(s0, LIFT ? sum[rt][nt][0] + offset[nt][0] : sum[rt][nt][0], acc[rt][nt][0]);
          acc[rt][nt][1] = fmaf(s0, LIFT ? sum[rt][nt][1] + offset[nt][1] : sum[rt][nt][1], acc[rt][nt][1]);
          acc[rt][nt][2] = fmaf(s1, LIFT ? sum[rt][nt][2] + offset[nt][2] : sum[rt][nt][2], acc[rt][nt][2]);
          acc[rt][nt][3] = fmaf(s1, LIFT ? sum[rt][nt][3] + offset[nt][3] : sum[rt][nt][3], acc[rt][nt][3]);
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
