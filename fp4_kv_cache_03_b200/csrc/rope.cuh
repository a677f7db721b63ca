// Rotary positions, shared by the rotation call and the 8-bit append: the checked parameters,
// frequencies in turns per token, and the sine and cosine of a position.
#pragma once

#include "common.cuh"

namespace csa2 {

constexpr int kMaxRot = 256;

struct RopeArgs {
  int rot, offset, interleaved;
  float amplitude;
  double turns[kMaxRot / 2];        // f_i / (2 pi)
};

// Host: fills *a, or returns the status of the first bad parameter.
csa2_status_t rope_args(const csa2_rope_t* r, RopeArgs* a);

// (cos, sin) of position `pos` for pair i.  pos * turns is exact to 2^-53 of
// itself, so what is left of it after the whole turns is good to 2^-32 of a turn at 2^20
// tokens; fp32 would keep 2^-4.
__device__ __forceinline__ float2 rope_unit(const RopeArgs& a, double pos, int i) {
  const double t = pos * a.turns[i];
  const float x = (float)(2.0 * (t - rint(t)));       // half turns, in [-1, 1]
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c, s);
}
// the same times the amplitude
__device__ __forceinline__ float2 rope_turn(const RopeArgs& a, double pos, int i) {
  const float2 t = rope_unit(a, pos, i);
  return make_float2(t.x * a.amplitude, t.y * a.amplitude);
}

}  // namespace csa2
