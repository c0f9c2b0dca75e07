// zpp_step_count.cuh -- the number of an optimiser step and the factors that depend on it, made on
// the device, where it is known whether the step is taken.
#pragma once

#include "zpp_device.cuh"
#include "zpp_launch.h"

namespace zpp {

// A step's number, its power of one beta (lane 0: beta1, lane 1: beta2) and the factor from it.
struct StepFactor {
  int64_t t;
  double before, power;  // beta^(t-1), beta^t
  float made;            // lane 0: lr / (1 - beta1^t), lane 1: 1 / sqrt(1 - beta2^t)
};

// By the first two lanes of a warp. Powers and factors are in 64 bits, rounded to 32 once, as the host
// makes them where it knows the number. 64-bit operations are slow here and pow takes some 5 us,
// so the power is the last one times beta; pow only after beta was changed. (A product adds 2^-53
// of the power each step, and the power falls as fast: 1 - beta^t stays within 2^-44 for beta <= 0.9999.)
__device__ __forceinline__ StepFactor step_factor(const StepCount& c, int lane) {
  StepFactor f;
  const volatile StepRecord* r = c.record;
  const double beta = lane == 0 ? c.beta[0] : c.beta[1];
  if (c.known > 0) {
    f.t = c.known;
    f.power = lane == 0 ? c.power[0] : c.power[1];
    f.before = f.power;  // (unused unless skipped; write_record then marks it)
    f.made = lane == 0 ? c.step_size : c.inv_root_bc2;
    return f;
  }
  f.t = r->step + 1;
  f.before = r->power[lane];
  if (r->beta[lane] != beta) f.before = pow(beta, static_cast<double>(f.t - 1));
  f.power = f.before * beta;
  const double correction = 1.0 - f.power;
  f.made = static_cast<float>(lane == 0 ? c.lr / correction : 1.0 / sqrt(correction));
  return f;
}
// A lane's part of the record of a step by `factor`; lane 0 the rest of it. inv_root_bc2: lane 1's.
__device__ __forceinline__ void write_record(const StepCount& c, const StepFactor& f, int lane,
                                             float factor, float inv_root_bc2) {
  const bool taken = isfinite(factor);
  c.record->power[lane] = taken ? f.power : f.before;
  // (a known step's power before it is not at hand: no beta is equal to NaN)
  c.record->beta[lane] = taken || c.known == 0 ? (lane == 0 ? c.beta[0] : c.beta[1]) : __longlong_as_double(-1LL);
  if (lane == 0) {
    c.record->step = taken ? f.t : f.t - 1;
    c.record->factor = factor;
    c.record->step_size = f.made;
    c.record->inv_root_bc2 = inv_root_bc2;
    c.record->key = (c.seed * 0x9E3779B9u) ^ (static_cast<uint32_t>(f.t) * 0x510E527Fu);
  }
}

}  // namespace zpp
