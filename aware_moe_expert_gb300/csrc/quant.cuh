// 4-bit weights: how they are packed, and how a packed word becomes bf16.
//
// A matrix [rows, K] is cut into tiles of 128 rows x 128 inputs, tile after tile
// along K, then row tile by row tile.  A tile is one record of 16-byte pieces,
// so that one bulk copy, or 16-byte loads of neighbouring lanes, fetch it:
//   [128 rows][64 bytes of codes]     then     [128 rows][128 / group scales]
// Rows and inputs past the matrix are zero weights.
//
// Codes: the 16-byte piece c of a row holds its inputs 32 c .. 32 c + 31, so that a lane
// with one piece needs one or two scales, and its 32-bit word w eight of them; four
// lanes with a piece each have, word by word, the K of two mma.m16n8k16.  Piece c of
// row r lies at place c ^ ((r / 2) % 4), which spreads eight rows' equal pieces over
// all banks.
//
// Eight codes of a word are four pairs (k, k + 1), one in each half word, that
// become bf16 pairs by a shift, a mask and one packed bf16 operation:
//   integer codes  nibble i of the low half is input 2i, of the high half 2i + 1.  The
//                  low eight bits of a bf16, a subnormal or just above, count 2^-133
//                  each, so pair 0 masked is q * 2^-133 and pair 1 in its place
//                  q * 2^-129 without a shift (pairs 2 and 3 take one together);
//                  fma(q * 2^-133, s * 2^117, -8 s * 2^-16) = (q - 8) s * 2^-16
//   e2m1           sign, exponent and mantissa stand so that pair i, moved to the
//                  bits 15 and 8-6 of a half word by one shift (i 0, 1) or a product, reads
//                  as code * 2^-126 (a subnormal for 0.5); times s * 2^117 that is
//                  code * s * 2^-9
// Both are exact: s has four significant bits, a code at most three, 8 s four.
// The factor 2^16 or 2^9 joins the matrix's own in the epilogue.
//
// Scales are e4m3 without its sign, stored with a fifth exponent bit so that
// subnormals are like the others: s = 2^E (1 + m / 8) is the byte (E + 16) << 3 | m,
// and (byte << 4) + a constant is s * 2^117 in bf16.  A scale of zero is
// stored as any, with zero codes.
#pragma once

#include "moe_common.cuh"

namespace moe {

constexpr int kQRows = 128, kQK = 128;          // a tile
constexpr uint32_t kQCodeBytes = kQRows * kQK / 2;

__host__ __device__ constexpr uint32_t quant_record(int group) {
  return kQCodeBytes + static_cast<uint32_t>(kQRows * (kQK / group));
}

// Tiles of a matrix along rows and inputs, and its bytes.
struct QuantShape {
  int rt, kb;
  size_t bytes;
};
__host__ __device__ inline QuantShape quant_shape(int rows, int K, int group) {
  QuantShape s;
  s.rt = (rows + kQRows - 1) / kQRows;
  s.kb = (K + kQK - 1) / kQK;
  s.bytes = static_cast<size_t>(s.rt) * s.kb * quant_record(group);
  return s;
}

// Place of the 16-byte piece c of row r within the codes of a tile, in bytes, and of
// its word w.
__host__ __device__ constexpr uint32_t quant_piece(int r, int c) {
  return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
__host__ __device__ constexpr uint32_t quant_word(int r, int c, int w) {
  return quant_piece(r, c) + static_cast<uint32_t>(4 * w);
}

// ---------------------------------------------------------------- values
constexpr uint32_t kScaleBase117 = 0x72007200u;  // exponent field of 2^101: s * 2^117
constexpr uint32_t kScaleBase113 = 0x70007000u;

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (a & b) | c in one operation.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// What a word's expansion needs of its group's scale, a byte of `bytes`, as pairs of
// equal bf16: s * 2^117, and for integer codes s * 2^113 and -8 s * 2^-16.
template <int CODE>
struct QuantScale {
  uint32_t s, t, c;
  __device__ __forceinline__ static QuantScale of(uint32_t twice) {   // the byte in both halves
    QuantScale q;
    q.s = twice * 16u + kScaleBase117;
    q.t = twice * 16u + kScaleBase113;
    q.c = CODE == MOE_QUANT_INT ? hmul2_bf16(q.s, 0x80088008u) : 0u;  // -2^-130
    return q;
  }
  template <int I>
  __device__ __forceinline__ static QuantScale at(uint32_t bytes) {
    return of(__byte_perm(bytes, 0u, 0x4040 | I << 8 | I));
  }
};

// The eight weights of a word, k ascending.
template <int CODE>
__device__ __forceinline__ void quant_expand(uint32_t w, const QuantScale<CODE>& q,
                                             uint32_t (&v)[4]) {
  if (CODE == MOE_QUANT_INT) {
    const uint32_t h = w >> 8;
    v[0] = hfma2_bf16(w & 0x000F000Fu, q.s, q.c);
    v[1] = hfma2_bf16(w & 0x00F000F0u, q.t, q.c);
    v[2] = hfma2_bf16(h & 0x000F000Fu, q.s, q.c);
    v[3] = hfma2_bf16(h & 0x00F000F0u, q.t, q.c);
  } else {
    v[0] = hmul2_bf16(w & 0x81C081C0u, q.s);
    v[1] = hmul2_bf16((w << 3) & 0x81C081C0u, q.s);
    v[2] = hmul2_bf16((w & 0x40074007u) * (64u + 2u) & 0x81C081C0u, q.s);
    v[3] = hmul2_bf16((w >> 3 & 0x05C005C0u) * (32u + 1u) & 0x81C081C0u, q.s);
  }
}

// What the sums of expanded weights are multiplied by, beside the matrix's factor.
template <int CODE>
__device__ __forceinline__ constexpr float quant_unit() {
  return CODE == MOE_QUANT_E2M1 ? 512.f : 65536.f;
}

// Where code q of the input pair's half h (0: even input) goes in its word.
__host__ __device__ inline uint32_t quant_place(int code, uint32_t q, int pair, int half) {
  if (code == MOE_QUANT_INT) return q << (4 * pair + 16 * half);
  // bits of sign, exponent high, exponent low, mantissa for each pair
  const uint32_t at[4] = {0x0F080706u, 0x0C050403u, 0x0E020100u, 0x0D0B0A09u};
  uint32_t v = 0;
  for (int b = 0; b < 4; ++b)
    v |= ((q >> b) & 1u) << (((at[pair] >> (8 * b)) & 31u) + 16u * half);
  return v;
}

}  // namespace moe
