// Rotary angles of the append kernels (pe_append.cu has the mathematics).
#pragma once

#include "pe_device.cuh"
#include "pe_internal.h"

namespace pe {

// Cosine and sine of pair i's angle at this position.
PE_DEV void rope_angle(const RopeTable& t, int pos, int i, float& c, float& s) {
  const uint64_t turn = (uint64_t)(int64_t)pos * t.turns[i];
  // the fraction's upper 32 bits, -1/2 to 1/2 of a turn: -1 to 1 half turns
  sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);
}

// (x1, x2) turned by that angle; products and sums are rounded as written, so that every kernel gives the same.
PE_DEV void rope_turn(float& x1, float& x2, float c, float s) {
  const float y1 = fmaf(x1, c, -__fmul_rn(x2, s)), y2 = fmaf(x2, c, __fmul_rn(x1, s));
  x1 = y1;
  x2 = y2;
}

}  // namespace pe
