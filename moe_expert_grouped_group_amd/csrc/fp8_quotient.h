// x / scale for the conversion to 8-bit floating point, decided exactly.  Plain C++, so that the host compiles
// the same arithmetic.
#pragma once

#include <cstdint>

#include "both_sides.h"

namespace mx {

// The quotient rounded to fp32 and, where it is even (a border between two codes is) and not exact, one step
// towards the exact one, so that it lies on the exact quotient's side of every border.  The step goes by the
// sign of x: a quotient that is too small for a number is a zero, whose own sign tells nothing, and with the
// sign bit at hand one step up from either zero is the smallest number of that sign.
MX_BOTH_SIDES float exact_quotient(float x, float scale) {
  if (scale < 0x1p-60f) x *= 0x1p100f, scale *= 0x1p100f;   // the remainder below keeps its bits
  const float v = x / scale;
  const float rest = __builtin_fmaf(-v, scale, x);
  uint32_t bits;
  __builtin_memcpy(&bits, &v, 4);
  if (rest != 0.f && (bits & 1) == 0) bits += (rest > 0.f) == (x > 0.f) ? 1u : ~0u;
  float w;
  __builtin_memcpy(&w, &bits, 4);
  return w;
}

}  // namespace mx
