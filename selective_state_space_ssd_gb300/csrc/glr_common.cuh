// What the files of the gated linear recurrence share: a call's sizes and the gates of a step.
#pragma once

#include <cuda_bf16.h>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.h"
#include "vec_io.cuh"

namespace ssd {
namespace glr {

constexpr int kMark = 32;  // the stash holds the state that enters every 32nd step

struct Args {
  int N, T, D;  // sequences, steps (of each, or of the packed axis), channels
  bool packed, f32;
  long long xs, rs, is;  // elements from a step to the next of x, r, i
  float scale;
};

// Checks a problem's numbers.
ssd_status make_args(const ssd_glr_problem* p, Args* a);

__device__ __forceinline__ float exp_of(float z, float) { return expf(z); }
__device__ __forceinline__ float exp_of(float z, bf16) { return __expf(z); }

// e^-z, at most e^80 (so that 1 + e and e s(z) stay finite); NaN stays NaN.
template <typename T>
__device__ __forceinline__ float exp_neg(float z) {
  return exp_of(z < -80.f ? 80.f : -z, T());
}
__device__ __forceinline__ float inv(float x) { return __fdividef(1.f, x); }
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  return inv(1.f + exp_neg<T>(z));
}

// e^g - 1 for g <= 0: the series to g^7 / 7! where |g| < 0.4 (what is left out is below 4e-8 of the sum), else e^g itself.
template <typename T>
__device__ __forceinline__ float expm1_neg(float g) {
  float s = fmaf(g, 1.f / 7.f, 1.f);
  s = fmaf(g * (1.f / 6.f), s, 1.f);
  s = fmaf(g * (1.f / 5.f), s, 1.f);
  s = fmaf(g * (1.f / 4.f), s, 1.f);
  s = fmaf(g * (1.f / 3.f), s, 1.f);
  s = fmaf(g * (1.f / 2.f), s, 1.f);
  return g > -0.4f ? g * s : exp_of(g, T()) - 1.f;
}

// a = e^g and m = sqrt(1 - a^2) of a step's gate.
template <typename T>
__device__ __forceinline__ void gates(float r, float ksp, float& a, float& m) {
  const float p = expm1_neg<T>(ksp * sigmoid<T>(r));
  a = 1.f + p;
  m = __fsqrt_rn(-p * (1.f + a));
}

}  // namespace glr
}  // namespace ssd
