// Format of microscaled (MX) 4-bit matrices, shared by the kernels that write, read and multiply them.
//
// 32 consecutive entries of a row share the scale 2^(c - 127), a byte c (254 at most; 255 stands for NaN).  An entry is
// a 4-bit float: sign, two exponent bits, one mantissa bit, the magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 in the order of
// their codes.
//
// Rows and widths are cut into pieces of 128 x 128, one record of 8704 bytes each, the pieces of the same rows after one
// another:
//   bytes [0, 512)      scales: of row r and 32-entry block b of the piece at (r % 32)*16 + (r / 32)*4 + b, which is the
//                       order in which a copy into tensor memory spreads them over its lanes and columns
//   bytes [512, 8704)   codes: 16 groups of 8 rows, each four blocks x 8 rows x 16 bytes (32 entries, the first in the
//                       lower half of the first byte): the 8-row, 16-byte core matrices of a K-major operand
// So a tile of 128 weight rows streams as contiguous copies of whole records, and the first n rows of a piece are one
// contiguous copy of 512 + 64 n bytes (n a multiple of 8).  Entries of a row's last piece beyond the width are zeros
// with scale byte 0; rows beyond the last are never used.
#pragma once

#include <stdint.h>

#include "pe_device.cuh"

namespace pe {

constexpr int kMxBlock = 32;                             // entries per scale
constexpr int kMxPiece = 128;                            // rows and entries of a record
constexpr uint32_t kMxScales = 512;                      // bytes of a record's scales
constexpr uint32_t kMxGroup = 512;                       // bytes of 8 rows' codes
constexpr uint32_t kMxRecord = kMxScales + 16 * kMxGroup;

__host__ __device__ constexpr uint32_t mx_scale_at(int r, int b) { return (uint32_t)((r & 31) * 16 + (r >> 5) * 4 + b); }
__host__ __device__ constexpr uint32_t mx_code_at(int r, int b) {
  return kMxScales + (uint32_t)(r >> 3) * kMxGroup + (uint32_t)b * 128 + (uint32_t)(r & 7) * 16;
}

// Eight floats, rounded to 4 bits (nearest, ties to the even code, saturating at 6), as one word.
PE_DEV uint32_t mx_encode8(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// The values of a word's eight codes as pairs of fp16 (exact), entries 2i and 2i + 1 in the i-th.
PE_DEV void mx_decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 2^(c - 127): the byte in the exponent field, a denormal for c = 0, NaN for 255.
PE_DEV float mx_scale(uint32_t c) {
  return __uint_as_float(c == 0 ? 0x00400000u : c == 255 ? 0x7FC00000u : c << 23);
}

// Eight entries at a 16-byte boundary.
PE_DEV void get8(const float* p, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 t = __ldcs(reinterpret_cast<const float4*>(p) + k);
    x[4 * k] = t.x; x[4 * k + 1] = t.y; x[4 * k + 2] = t.z; x[4 * k + 3] = t.w;
  }
}
PE_DEV void get8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 t = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
// The first n of them, then zeros.  (Loads under a condition wait for each other, so the last one there is read again in the
// place of those that are not.)
template <typename T>
PE_DEV void get8_of(const T* p, int n, float (&x)[8]) {
  if (n >= 8) {
    get8(p, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (n <= 0) return;
    T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[min(e, n - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) x[e] = to_float<T>(v[e]);
  }
}
PE_DEV uint32_t max_over_four(uint32_t v) {
  v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}

// Rounds the eight entries that this lane has of a block (the three lanes beside it have the others): their codes, and
// the block's scale byte.  The scale is 2^(floor(log2 amax) - 2): the exponent field of amax less two.  Returns whether
// one of the block's entries was NaN (kept as 0) or infinite (kept as +-6 of the scale of the finite ones).
PE_DEV bool mx_round8(float (&x)[8], uint32_t& codes, uint32_t& scale) {
  constexpr uint32_t kInf = 0x7F800000u;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  top = max_over_four(top);
  const bool bad = top >= kInf;
  if (__any_sync(0xFFFFFFFFu, bad)) {
    uint32_t finite = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t m = __float_as_uint(x[e]) & 0x7FFFFFFFu;
      if (m < kInf) finite = max(finite, m);
      if (m > kInf) x[e] = 0.f;
    }
    top = max_over_four(finite);
  }
  // fields 0 to 2 (below 2^-124) have the smallest scale, 2^-127
  scale = (uint32_t)max((int)(top >> 23) - 2, 0);
  const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale): 2^127 down to 2^-125, exact products
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  codes = mx_encode8(x);
  return bad;
}

}  // namespace pe
