// The gated linear recurrence's recurrent form, for serving: T >= 1 steps of every sequence of a batch on a cache of fp32
// states that is updated in place (formulas: ssd_glr.cu).  One thread has kW channels of a sequence; the state is read
// once, held in registers over all steps and written once.  Bound by memory and, at a few sequences, by the launch.
#include "glr_common.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kThreads = 128;

// kW = 4: rows of whole four-element pieces, aligned; 1: any.
template <typename T, int kW>
__global__ void __launch_bounds__(kThreads)
    k_glr_step(Args a, const T* __restrict__ x, const T* __restrict__ r, const T* __restrict__ i,
               const float* __restrict__ lam, float* state, const int* __restrict__ slots, long long num_slots, T* y) {
  const int c = (blockIdx.x * kThreads + threadIdx.x) * kW;
  if (c >= a.D) return;
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    const long long slot = slots ? slots[n] : n;
    const bool held = slot >= 0 && slot < num_slots;  // else: a place without a sequence, y = 0
    float* s = state + (held ? (size_t)slot * a.D : 0) + c;
    float h[kW], ksp[kW];
    load<float, kW>(lam + c, ksp);
    if (held) load<float, kW>(s, h);
#pragma unroll
    for (int k = 0; k < kW; ++k) ksp[k] = -a.scale * softplus_f(ksp[k]);
    for (int t = 0; t < a.T; ++t) {
      const size_t at = (size_t)n * a.T + t;
      if (held) {
        float xv[kW], rv[kW], iv[kW];
        load<T, kW>(x + at * a.xs + c, xv);
        load<T, kW>(r + at * a.rs + c, rv);
        load<T, kW>(i + at * a.is + c, iv);
#pragma unroll
        for (int k = 0; k < kW; ++k) {
          float av, m;
          gates<T>(rv[k], ksp[k], av, m);
          h[k] = fmaf(av, h[k], m * (sigmoid<T>(iv[k]) * xv[k]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < kW; ++k) h[k] = 0.f;
      }
      save<T, kW>(y + at * a.D + c, h);
    }
    if (held) save<float, kW>(s, h);
  }
}

template <typename T>
void launch(const Args& a, const void* x, const void* r, const void* i, const float* lam, float* state, const int32_t* slots,
            long long num_slots, void* y, cudaStream_t st) {
  const uintptr_t piece = 4 * sizeof(T);
  const bool whole = !(a.D % 4 || a.xs % 4 || a.rs % 4 || a.is % 4 || off(x, piece) || off(r, piece) || off(i, piece) ||
                       off(y, piece) || off(lam, 16) || off(state, 16));
  const int w = whole ? 4 : 1, groups = (a.D + w - 1) / w;
  const dim3 grid((groups + kThreads - 1) / kThreads, a.N < 65535 ? a.N : 65535);
  if (whole)
    SSD_LAUNCH("k_glr_step", st,
               k_glr_step<T, 4><<<grid, kThreads, 0, st>>>(a, (const T*)x, (const T*)r, (const T*)i, lam, state, slots,
                                                           num_slots, (T*)y));
  else
    SSD_LAUNCH("k_glr_step", st,
               k_glr_step<T, 1><<<grid, kThreads, 0, st>>>(a, (const T*)x, (const T*)r, (const T*)i, lam, state, slots,
                                                           num_slots, (T*)y));
}

}  // namespace
}  // namespace glr
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status ssd_glr_step(const ssd_glr_problem* prob, const void* x, const void* r, const void* i, const float* lam,
                                   float* state, const int32_t* slots, int64_t num_slots, float scale, void* y,
                                   void* cuda_stream) {
  glr::Args a;
  const ssd_status s = glr::make_args(prob, &a);
  if (s != SSD_OK) return s;
  if (a.packed || num_slots < 1 || (!slots && num_slots < a.N)) return SSD_ERR_INVALID_ARG;
  if (!x || !r || !i || !lam || !state || !y || !(scale >= 0.f) || scale > 3e38f) return SSD_ERR_INVALID_ARG;
  const uintptr_t elem = a.f32 ? 4 : 2;
  if (off(x, elem) || off(r, elem) || off(i, elem) || off(lam, 4) || off(state, 4) ||
      off(slots, 4) || off(y, elem))
    return SSD_ERR_ALIGNMENT;
  a.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (a.f32)
    glr::launch<float>(a, x, r, i, lam, state, slots, num_slots, y, st);
  else
    glr::launch<bf16>(a, x, r, i, lam, state, slots, num_slots, y, st);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
