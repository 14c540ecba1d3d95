// Format of the packed (4-bit) KV cache, shared by the kernels that write and read it.
//
// A pool holds [num_pages][n_kv] records of 18 * head_dim bytes, one per page of 16 positions
// and kv head:
//
//   bytes [0, 8 hd)         key codes, one row of hd/2 bytes per position
//   bytes [8 hd, 16 hd)     value codes, the same
//   bytes [16 hd, 17 hd)    key scales, one row of hd/16 bytes per position
//   bytes [17 hd, 18 hd)    value scales
//
// 16 consecutive entries of a row share one scale byte c, s(c) = (1 + (c & 7)/8) 2^((c >> 3) - 19):
// the smallest with 7 s >= the block's largest magnitude.  An entry is kept as the whole number
// n = sign(x) min(7, floor(|x|/s + 1/2)), stored as the nibble n + 8, and stands for n s.
// n has three bits and s four significant ones, so n s has seven: exact in bf16, and the
// tensor cores multiply what the cache stands for without a further rounding.
//
// Inside a row the nibbles stand in the order in which the matrix instructions take them,
// as 32-bit words of eight (nibble i in bits 4i..4i+3):
//   keys:   word t*(hd/32) + u (t < 4), nibble i < 4: entry 16(2u + i/2) + 4t + 2(i%2); nibble
//           i + 4: the entry after it.
//   values: word g*(hd/64) + h (g < 8), nibble i: entry 64h + 16(i/2) + g + 8(i%2).
// Two nibbles 16 bits apart become one pair of bf16 with three operations (a shift for three of
// four, a mask-and-or, one fused multiply-add): the nibble in the lowest mantissa bits of 128
// reads 128 + nibble, and (128 + nibble) S - 136 S = (nibble - 8) S, exactly: 136 S = 8 * 17 S has at
// most eight significant bits (17 * 15 = 255).  The scale byte in the exponent and mantissa bits
// below a fixed upper exponent reads S = s 2^-12, so a key or value of the matrix products is
// 2^-12 of what it stands for (kPackedUnit undoes that).
#pragma once

#include <stdint.h>

#include "pe_device.cuh"

namespace pe {

constexpr int kPackedPage = 16;           // positions per record
constexpr int kPackedBlock = 16;          // entries per scale
constexpr float kPackedUnit = 4096.f;     // value of an entry over its bf16 form in the kernels

template <int HD>
struct PackedLayout {
  static constexpr int kRow = HD / 2;     // bytes of one position's codes
  static constexpr int kScaleRow = HD / kPackedBlock;
  static constexpr int kK = 0, kV = 8 * HD, kKs = 16 * HD, kVs = 17 * HD, kRecord = 18 * HD;
};

// n / d for n < 2^31 by a multiplication: mul = ceil(2^shift / d), shift = 31 + ceil(log2 d), is at most
// d 2^-shift above 1/d, which is less than 1/(n d).  (A division by a value that the compiler does not know
// is a chain of about 150 cycles, several of which stood before the first load.)
struct Div {
  uint32_t mul;
  int shift;
};
inline Div make_div(uint32_t d) {
  int l = 0;
  while ((1u << l) < d) ++l;
  return Div{(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}
PE_DEV uint32_t operator/(uint32_t n, const Div& d) { return (uint32_t)(((uint64_t)n * d.mul) >> d.shift); }

// s(c) as fp32.
PE_DEV float packed_scale(uint32_t c) { return __uint_as_float((c << 20) + (108u << 23)); }

// s(c) as a pair of bf16 (exact: four significant bits).
PE_DEV uint32_t packed_scale_pair(uint32_t c) { return ((c << 4) + (108u << 7)) * 0x10001u; }

// Two of a word's eight nibbles as bf16 pairs 128 + nibble: nibble I in the lower half, I + 4 above.
// (A mask and an exponent are two constants, of which one instruction takes one: the compiler makes two
// instructions of it unless the other is in a register that it does not look into.)
struct PairBits {
  uint32_t exponent;
  PE_DEV PairBits() { asm("mov.b32 %0, 0x43004300;" : "=r"(exponent)); }
  template <int I>
  PE_DEV uint32_t pair(uint32_t w) const {
    uint32_t d;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(d) : "r"(I == 0 ? w : w >> (4 * I)), "r"(exponent));
    return d;
  }
};

// Two scale bytes (the first or the second byte of either half of x) as bf16 pairs s 2^-12.
PE_DEV uint32_t packed_scale_lo(uint32_t x) { return ((x << 4) & 0x0FF00FF0u) | 0x30003000u; }
PE_DEV uint32_t packed_scale_hi(uint32_t x) { return ((x >> 4) & 0x0FF00FF0u) | 0x30003000u; }
PE_DEV uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
PE_DEV uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
constexpr uint32_t kMinus136 = 0xC308C308u;  // -136 twice

}  // namespace pe
