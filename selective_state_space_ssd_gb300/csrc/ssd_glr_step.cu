// The gated linear recurrence's recurrent form, for serving: T >= 1 steps of every sequence of a batch on a cache of fp32
// states that is updated in place (formulas: ssd_glr.cu).  One thread has kW channels of a sequence; the state is read
// once, held in registers over all steps and written once.  Bound by memory and, at a few sequences, by the launch.
#include "glr_common.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kStepThreads = 128;

// kW = 4: rows of whole four-element pieces, aligned; 1: any.
template <typename T, int kW>
__global__ void __launch_bounds__(kStepThreads)
    k_glr_step(Args a, const T* __restrict__ x, const T* __restrict__ r, const T* __restrict__ i,
               const float* __restrict__ lam, float* state, const int* __restrict__ slots, long long num_slots, T* y) {
  const int c = (blockIdx.x * kStepThreads + threadIdx.x) * kW;
  if (c >= a.D) return;
  const int n = blockIdx.y;
  const long long slot = slots ? slots[n] : n;
  const bool held = slot >= 0 && slot < num_slots;  // else: a place without a sequence, y = 0
  float* s = state + (held ? (size_t)slot * a.D : 0) + c;
  constexpr int kP = (kW + 1) / 2;
  const auto two = [](const float(&v)[kW], int p) { return pair(v[2 * p], kW > 1 ? v[(2 * p + 1) % kW] : 0.f); };
  float h[kW] = {}, l[kW];
  load<float, kW>(lam + c, l);
  if (held) load<float, kW>(s, h);
  P rate[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    rate[p] = each(two(l, p), [&](float v) { return a.scale * softplus_f(v); });
  }
  for (int t = 0; t < a.T; ++t) {
    const size_t at = (size_t)n * a.T + t;
    if (held) {
      float xv[kW], rv[kW], iv[kW];
      load<T, kW>(x + at * a.xs + c, xv);
      load<T, kW>(r + at * a.rs + c, rv);
      load<T, kW>(i + at * a.is + c, iv);
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const P o = one_minus_exp<true>(rate[p] * sigmoid(two(rv, p))), av = one_less(o);
        const P m = each(o * one_more(av), [](float v) { return sqrt_f(v); });
        const P hn = fma(av, two(h, p), m * (sigmoid(two(iv, p)) * two(xv, p)));
        float h0, h1;
        split(hn, h0, h1);
        h[2 * p] = h0;
        if (kW > 1) h[(2 * p + 1) % kW] = h1;
      }
    }
    save<T, kW>(y + at * a.D + c, h);
  }
  if (held) save<float, kW>(s, h);
}

template <typename T>
void launch(const Args& a, const void* x, const void* r, const void* i, const float* lam, float* state, const int32_t* slots,
            long long num_slots, void* y, cudaStream_t st) {
  const uintptr_t piece = 4 * sizeof(T);
  const bool whole = !(a.D % 4 || a.xs % 4 || a.rs % 4 || a.is % 4 || off(x, piece) || off(r, piece) || off(i, piece) ||
                       off(y, piece) || off(lam, 16) || off(state, 16));
  const int w = whole ? 4 : 1, groups = (a.D + w - 1) / w;
  const dim3 grid((groups + kStepThreads - 1) / kStepThreads, a.N);  // (make_args: 65535 sequences at most)
  if (whole)
    SSD_LAUNCH("k_glr_step", st,
               k_glr_step<T, 4><<<grid, kStepThreads, 0, st>>>(a, (const T*)x, (const T*)r, (const T*)i, lam, state, slots,
                                                           num_slots, (T*)y));
  else
    SSD_LAUNCH("k_glr_step", st,
               k_glr_step<T, 1><<<grid, kStepThreads, 0, st>>>(a, (const T*)x, (const T*)r, (const T*)i, lam, state, slots,
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
