// bl_sample_bounds.h - bounds of a histogram bin's weight, from its tokens' count
// and the sum of their places. Plain C++ as well as device code.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define BL_BOUNDS_FN __host__ __device__ __forceinline__
#else
#define BL_BOUNDS_FN inline
#endif

namespace bl {

// What a bin's sum of places says: a token of place v lies `unit` v + `mid` bins
// past the bin's start, give or take `half`.
struct BinPlaces {
  float unit, mid, half;
};
// By the bits below a histogram word's count: 19 (64ths), 18 (sixteenths), 0 (none).
// A 64th j is a position rounded to the nearest: j / 64 give or take 1 / 128, so
// tokens of place 0 may lie before the bin that counts them. A sixteenth stands
// for four 64ths and a bare count for all 64: half the way between the first and
// the last, and 1 / 128 more to either side. The position itself is off by its two
// roundings, 2047 bins * 2 * 2^-24 < 0.0003 bins; 0.002 are allowed.
BL_BOUNDS_FN BinPlaces bin_places(int packed) {
  BinPlaces p;
  p.unit = packed == 19 ? 1.0f / 64.0f : (packed == 18 ? 1.0f / 16.0f : 0.0f);
  p.mid = packed == 19 ? 0.0f : (packed == 18 ? 1.5f / 64.0f : 31.5f / 64.0f);
  p.half = (packed == 19 ? 0.5f / 64.0f : (packed == 18 ? 2.0f / 64.0f : 32.0f / 64.0f)) + 0.002f;
  return p;
}

struct WeightBounds {
  float lo, hi;
};
// Bins of width delta in the exponent: a token f bins past the bin's start, where
// the weight is e, weighs e^(-delta f) of it: at least its tangent 1 - delta f, and
// at most the chord 1 - shrink f over [0, 1], shrink = 1 - e^-delta (its series to
// the third term is above it by less than delta^4 / 24). Before the start, down to
// f = -0.01, the curve is above the chord by less than delta^2 / 150; the factor
// 1 + delta^2 covers both. count tokens, their places added to off; the sums of f
// are bounded as they come, below zero too.
BL_BOUNDS_FN WeightBounds bin_weight(float e, float delta, const BinPlaces& p, uint32_t count, uint32_t off) {
  const float shrink = delta * (1.0f - delta * (0.5f - delta * (1.0f / 6.0f)));
  const float c = (float)count, f = (float)off * p.unit + c * p.mid;
  const float slack = c * 1e-12f;  // weights are whole multiples of 2^-40: 1.1 of them a token
  WeightBounds w;
  w.lo = c > 0.f ? fmaxf(e * (c - delta * (f + c * p.half)) - slack, 0.f) : 0.f;
  w.hi = c > 0.f ? e * (c - shrink * (f - c * p.half)) * (1.0f + delta * delta) + slack : 0.f;
  return w;
}

}  // namespace bl
