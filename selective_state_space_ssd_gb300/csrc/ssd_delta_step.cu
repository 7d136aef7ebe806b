// The gated delta rule's recurrent form, for serving: T >= 1 steps (one token, or a few drafted ones) of every sequence
// of a batch on a cache of fp32 states that is updated in place.  fp32 arithmetic throughout.
//
// Per (sequence, value head) and step, with Sd = e^g S:
//     r = beta (v - Sd^T k),   S <- Sd + k r^T,   o = scale S^T q = scale (Sd^T q + (k.q) r)
// so both products of the old state (with k and with q) come out of one pass over it: the state is read once, held in
// registers over all T steps and written once.  The state is nearly all that a call moves, and the kernel is bound by
// that: 192 sequences of 32 heads of 128 x 128 take 146 us, 5.5 TB/s read and written.  32 columns of a state a block: a
// warp reads whole 128-byte rows, and one sequence of 16 heads is still 64 blocks.
#include <initializer_list>

#include "delta_common.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kCols = 32;     // columns of V a block
constexpr int kThreads = 128; // 8 column groups of four x 16 row groups

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float* p, float x) { *p = x; }
__device__ __forceinline__ void stf(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T>
struct StepIn {
  const T *q, *k, *v;
  const void *g, *beta;
  const int* slots;
  long long num_slots;
  float scale;
};

// A block: 32 columns of one state, all of its K rows; thread (cg, rg) holds columns 4 cg .. + 3 of the rows
// rg, rg + 16, ...: a warp reads four rows of 128 bytes at a time.  kVec: rows of V are whole 16-byte pieces.
template <typename T, int KP, bool kVec>
__global__ void __launch_bounds__(kThreads) k_delta_step(Dims d, StepIn<T> in, float* state, T* o) {
  constexpr int kRows = KP / 16;
  __shared__ float s_k[2][KP], s_q[2][KP];
  __shared__ float s_part[4][8][9];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, cg = tid & 7, rg = tid >> 3;
  const int n = blockIdx.x / d.HV, hv = blockIdx.x - n * d.HV, hk = hv / d.G;
  const int v0 = blockIdx.y * kCols + 4 * cg;
  const long long slot = in.slots ? in.slots[n] : n;
  if (slot < 0 || slot >= in.num_slots) {  // a place that holds no sequence: no state, o = 0
    if (rg == 0)
      for (int t = 0; t < d.T; ++t)
        for (int j = 0; j < 4; ++j)
          if (v0 + j < d.V) stf(o + (((size_t)n * d.T + t) * d.HV + hv) * d.V + v0 + j, 0.f);
    return;
  }
  float* s = state + ((size_t)slot * d.HV + hv) * d.K * d.V;
  float S[kRows][4];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = rg + 16 * i;
    if (kVec) {
      const float4 x = r < d.K && v0 < d.V ? *reinterpret_cast<const float4*>(s + (size_t)r * d.V + v0)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i][0] = x.x;
      S[i][1] = x.y;
      S[i][2] = x.z;
      S[i][3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = r < d.K && v0 + j < d.V ? s[(size_t)r * d.V + v0 + j] : 0.f;
    }
  }
  for (int t = 0; t < d.T; ++t) {
    const long long tok = (long long)n * d.T + t;
    const int p = t & 1;
    if (tid < KP) {
      s_k[p][tid] = tid < d.K ? ldf(in.k + tok * d.ks + (long long)hk * d.K + tid) : 0.f;
      s_q[p][tid] = tid < d.K ? ldf(in.q + tok * d.qs + (long long)hk * d.K + tid) : 0.f;
    }
    const size_t gi = (size_t)tok * d.HV + hv;
    const float decay = expf(gate(in.g, gi, d.gate_bf16)), beta = gate(in.beta, gi, d.gate_bf16);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = v0 + j < d.V ? ldf(in.v + tok * d.vs + (long long)hv * d.V + v0 + j) : 0.f;
    __syncthreads();
    float a[9];  // k.S and q.S of the four columns, k.q
#pragma unroll
    for (int j = 0; j < 9; ++j) a[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float kr = s_k[p][rg + 16 * i], qr = s_q[p][rg + 16 * i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] *= decay;
        a[j] = fmaf(kr, S[i][j], a[j]);
        a[4 + j] = fmaf(qr, S[i][j], a[4 + j]);
      }
      a[8] = fmaf(kr, qr, a[8]);
    }
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      a[j] += __shfl_xor_sync(0xffffffffu, a[j], 8);
      a[j] += __shfl_xor_sync(0xffffffffu, a[j], 16);
    }
    if (lane < 8)
#pragma unroll
      for (int j = 0; j < 9; ++j) s_part[w][lane][j] = a[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 9; ++j)
      a[j] = (s_part[0][cg][j] + s_part[1][cg][j]) + (s_part[2][cg][j] + s_part[3][cg][j]);
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = beta * (v[j] - a[j]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float kr = s_k[p][rg + 16 * i];
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = fmaf(kr, r[j], S[i][j]);
    }
    if (rg == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v0 + j < d.V) stf(o + (size_t)gi * d.V + v0 + j, in.scale * fmaf(a[8], r[j], a[4 + j]));
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = rg + 16 * i;
    if (r >= d.K) continue;
    if (kVec) {
      if (v0 < d.V)
        *reinterpret_cast<float4*>(s + (size_t)r * d.V + v0) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v0 + j < d.V) s[(size_t)r * d.V + v0 + j] = S[i][j];
    }
  }
}

template <typename T, int KP>
void launch(const Dims& d, const StepIn<T>& in, float* state, T* o, cudaStream_t st) {
  const dim3 grid((unsigned)(d.N * d.HV), (unsigned)((d.V + kCols - 1) / kCols));
  if (d.V % 4 == 0)
    SSD_LAUNCH("k_delta_step", st, k_delta_step<T, KP, true><<<grid, kThreads, 0, st>>>(d, in, state, o));
  else
    SSD_LAUNCH("k_delta_step", st, k_delta_step<T, KP, false><<<grid, kThreads, 0, st>>>(d, in, state, o));
}
template <typename T>
void launch(const Dims& d, const void* q, const void* k, const void* v, const void* g, const void* beta, float* state,
            const int32_t* slots, long long num_slots, float scale, void* o, cudaStream_t st) {
  const StepIn<T> in{(const T*)q, (const T*)k, (const T*)v, g, beta, slots, num_slots, scale};
  if (d.KP == 64)
    launch<T, 64>(d, in, state, (T*)o, st);
  else
    launch<T, 128>(d, in, state, (T*)o, st);
}

}  // namespace
}  // namespace delta
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status ssd_delta_step(const ssd_delta_problem* prob, const void* q, const void* k, const void* v,
                                     const void* g, const void* beta, float* state, const int32_t* slots,
                                     int64_t num_slots, float scale, void* o, void* cuda_stream) {
  delta::Dims d;
  const ssd_status s = delta::make_dims(prob, true, &d);
  if (s != SSD_OK) return s;
  if (d.packed || num_slots < 1 || (!slots && num_slots < d.N)) return SSD_ERR_INVALID_ARG;
  const uintptr_t elem = d.f32 ? 4 : 2, gelem = d.gate_bf16 ? 2 : 4;
  const auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (!q || !k || !v || !g || !beta || !state || !o) return SSD_ERR_INVALID_ARG;
  if (off(q, elem) || off(k, elem) || off(v, elem) || off(g, gelem) || off(beta, gelem) || off(o, elem) ||
      off(slots, 4) || off(state, 16))
    return SSD_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (d.f32)
    delta::launch<float>(d, q, k, v, g, beta, state, slots, num_slots, scale, o, st);
  else
    delta::launch<delta::bf16>(d, q, k, v, g, beta, state, slots, num_slots, scale, o, st);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
