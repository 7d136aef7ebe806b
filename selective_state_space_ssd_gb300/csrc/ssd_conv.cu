// The causal short convolution of each channel (depthwise), with bias and SiLU:
//     z_t = bias + sum over j < K of w[K-1-j] x_{t-j},   y = silu(z) = z s(z), or y = z
//     dz = dy y'(z),  dx_t = sum over j of w[K-1-j] dz_{t+j},  dw[K-1-j] = sum over t of dz_t x_{t-j},  dbias = sum of dz
// where the steps are those of one sequence and x before its first one is its K - 1 taps (or zeros).
// All of it is bound by memory.  A warp takes kW channels a lane and a run of steps, and holds what the taps reach back to
// (and, backward, the K - 1 gradients that still miss terms) in registers, so a run reads K - 1 steps more than its own.
// Eight steps are loaded before the first is used.  The weight's gradient is summed by a thread over its run, by a block
// over its eight runs in order, and over blocks in order by k_conv_sums: nothing depends on timing.
#include <initializer_list>
#include <type_traits>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.h"
#include "vec_io.cuh"

namespace ssd {
namespace conv {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kAhead = 8;  // steps loaded at a time

struct Args {
  int N, T, D, K;
  bool packed, f32, wbf16, silu;
  long long xs;  // elements from a step of x to the next
  int run;       // steps a warp (a multiple of kAhead)
};

struct Call {
  Args a;
  const void *dy, *x, *w, *b, *taps;
  const int* cu;
  void *y, *taps_out, *dx, *dw, *db, *dtaps;
  float* part;
};

// The sequence that step t belongs to (-1: none) and its first and last + 1 step; 0 <= begin <= t < end <= T.
struct Seq {
  int n, begin, end;
};
__device__ __forceinline__ int clamp_cu(const int* cu, int n, int T) { return min(max(cu[n], 0), T); }
__device__ __forceinline__ Seq locate(const int* cu, int N, int T, int t) {
  int lo = 0, hi = N;  // the last n with cu[n] <= t, or -1
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (clamp_cu(cu, mid, T) <= t)
      lo = mid + 1;
    else
      hi = mid - 1;
  }
  if (hi < 0) return Seq{-1, 0, clamp_cu(cu, 0, T)};
  if (hi >= N) return Seq{-1, clamp_cu(cu, N, T), T};
  return Seq{hi, clamp_cu(cu, hi, T), clamp_cu(cu, hi + 1, T)};
}

// kW channels' weights, w[tap][channel], and bias.
template <int K, int kW>
__device__ __forceinline__ void load_weights(const void* w, const void* b, bool wbf16, int c, float (&wt)[K][kW],
                                             float (&bias)[kW]) {
  float flat[K * kW];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    float v[kW];
    if (wbf16)
      load<bf16, kW>(static_cast<const bf16*>(w) + (size_t)c * K + i * kW, v);
    else
      load<float, kW>(static_cast<const float*>(w) + (size_t)c * K + i * kW, v);
#pragma unroll
    for (int k = 0; k < kW; ++k) flat[i * kW + k] = v[k];
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int k = 0; k < kW; ++k) wt[j][k] = flat[k * K + j];
#pragma unroll
  for (int k = 0; k < kW; ++k) bias[k] = 0.f;
  if (b) {
    if (wbf16)
      load<bf16, kW>(static_cast<const bf16*>(b) + c, bias);
    else
      load<float, kW>(static_cast<const float*>(b) + c, bias);
  }
}

// win[j] = x_{t-1-j}: steps of the sequence, before its first one its taps.
template <typename T, int K, int kW>
__device__ __forceinline__ void load_window(const T* x, long long xs, const T* taps, int D, const Seq& q, int t,
                                            float (&win)[K - 1][kW]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int at = t - 1 - j;
#pragma unroll
    for (int k = 0; k < kW; ++k) win[j][k] = 0.f;
    if (q.n < 0) continue;
    if (at >= q.begin)
      load<T, kW>(x + (long long)at * xs, win[j]);
    else if (taps)
      load<T, kW>(taps + ((size_t)q.n * (K - 1) + (K - 1 + at - q.begin)) * D, win[j]);
  }
}
template <int K, int kW>
__device__ __forceinline__ void shift(float (&win)[K - 1][kW], const float (&x)[kW]) {
#pragma unroll
  for (int j = K - 2; j > 0; --j)
#pragma unroll
    for (int k = 0; k < kW; ++k) win[j][k] = win[j - 1][k];
#pragma unroll
  for (int k = 0; k < kW; ++k) win[0][k] = x[k];
}
template <int K, int kW>
__device__ __forceinline__ float product(const float (&wt)[K][kW], const float (&bias)[kW], const float (&win)[K - 1][kW],
                                         const float (&x)[kW], int k) {
  float z = fmaf(wt[K - 1][k], x[k], bias[k]);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) z = fmaf(wt[K - 2 - j][k], win[j][k], z);
  return z;
}
template <typename T>
__device__ __forceinline__ float exp_minus(float z) {  // e^-z, at most e^80
  const float e = z < -80.f ? 80.f : -z;
  return sizeof(T) == 4 ? expf(e) : __expf(e);
}
template <typename T>
__device__ __forceinline__ float act(float z, bool silu) {
  return silu ? __fdividef(z, 1.f + exp_minus<T>(z)) : z;
}
template <typename T>
__device__ __forceinline__ float slope(float z, bool silu) {  // s (1 + z (1 - s))
  const float e = exp_minus<T>(z), s = __fdividef(1.f, 1.f + e);
  return silu ? s * fmaf(z, e * s, 1.f) : 1.f;
}

// Elements as they lie in memory, loaded ahead of their use.
template <typename T, int kW>
struct __align__(kW * sizeof(T)) RawVec {
  T v[kW];
};
template <typename T, int kW>
__device__ __forceinline__ void widen(const RawVec<T, kW>& r, float (&v)[kW]) {
#pragma unroll
  for (int k = 0; k < kW; ++k) v[k] = (float)r.v[k];
}
template <typename T, int kW>
__device__ __forceinline__ RawVec<T, kW> raw(const T* p) {
  return *reinterpret_cast<const RawVec<T, kW>*>(p);
}

// A block: 32 kW channels, eight runs of steps one after another.  Grid: (chunks of eight runs x channel slabs, sequences).
template <typename T, int K, int kW>
__global__ void __launch_bounds__(kThreads) k_conv_forward(Args a, const T* __restrict__ x, const void* __restrict__ w,
                                                           const void* __restrict__ b, const T* __restrict__ taps,
                                                           const int* __restrict__ cu, T* y, T* taps_out, int slabs) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, axis = blockIdx.y;
  const int chunk = blockIdx.x / slabs, c = ((blockIdx.x - chunk * slabs) * 32 + lane) * kW;
  if (c >= a.D) return;
  if (a.packed && taps_out && chunk == 0)  // sequences without steps keep their taps
    for (int n = warp; n < a.N; n += kWarps)
      if (clamp_cu(cu, n + 1, a.T) <= clamp_cu(cu, n, a.T))
        for (int p = 0; p < K - 1; ++p) {
          float v[kW] = {};
          const size_t at = ((size_t)n * (K - 1) + p) * a.D + c;
          if (taps) load<T, kW>(taps + at, v);
          save<T, kW>(taps_out + at, v);
        }
  const long long first = ((long long)chunk * kWarps + warp) * a.run;
  if (first >= a.T) return;
  const int t0 = (int)first, t1 = (int)(first + a.run < a.T ? first + a.run : a.T);
  const T* px = x + (size_t)axis * a.T * a.xs + c;
  T* py = y + (size_t)axis * a.T * a.D + c;
  const T* pt = taps ? taps + c : nullptr;
  float wt[K][kW], bias[kW], win[K - 1][kW];
  load_weights<K, kW>(w, b, a.wbf16, c, wt, bias);
  Seq q = a.packed ? locate(cu, a.N, a.T, t0) : Seq{axis, 0, a.T};
  load_window<T, K, kW>(px, a.xs, pt, a.D, q, t0, win);
  for (int t = t0; t < t1; t += kAhead) {
    RawVec<T, kW> next[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
      if (t + s < t1) next[s] = raw<T, kW>(px + (long long)(t + s) * a.xs);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      if (t + s >= t1) break;
      if (t + s >= q.end) {
        q = locate(cu, a.N, a.T, t + s);
        load_window<T, K, kW>(px, a.xs, pt, a.D, q, t + s, win);
      }
      float v[kW], o[kW];
      widen(next[s], v);
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        o[k] = act<T>(product<K, kW>(wt, bias, win, v, k), a.silu);
        if (q.n < 0) o[k] = 0.f;
      }
      save<T, kW>(py + (size_t)(t + s) * a.D, o);
      shift<K, kW>(win, v);
      if (taps_out && t + s == q.end - 1 && q.n >= 0) {
#pragma unroll
        for (int p = 0; p < K - 1; ++p) save<T, kW>(taps_out + ((size_t)q.n * (K - 1) + p) * a.D + c, win[K - 2 - p]);
      }
    }
  }
}

template <typename T, int K, int kW>
__global__ void __launch_bounds__(kThreads) k_conv_backward(Args a, const T* __restrict__ dy, const T* __restrict__ x,
                                                            const void* __restrict__ w, const void* __restrict__ b,
                                                            const T* __restrict__ taps, const int* __restrict__ cu, T* dx,
                                                            float* part, int slabs) {
  __shared__ float red[kWarps][(K + 1) * kW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, axis = blockIdx.y;
  const int chunk = blockIdx.x / slabs, c = ((blockIdx.x - chunk * slabs) * 32 + lane) * kW;
  const long long first = ((long long)chunk * kWarps + warp) * a.run;
  float sum[K + 1][kW] = {};  // dw by tap, dbias
  if (c < a.D && first < a.T) {
    const int t0 = (int)first, t1 = (int)(first + a.run < a.T ? first + a.run : a.T);
    const T* px = x + (size_t)axis * a.T * a.xs + c;
    const T* pg = dy + (size_t)axis * a.T * a.D + c;
    T* pd = dx + (size_t)axis * a.T * a.D + c;
    const T* pt = taps ? taps + c : nullptr;
    float wt[K][kW], bias[kW], win[K - 1][kW], acc[K - 1][kW] = {};  // acc[j]: dx of step t - 1 - j so far
    load_weights<K, kW>(w, b, a.wbf16, c, wt, bias);
    Seq q = a.packed ? locate(cu, a.N, a.T, t0) : Seq{axis, 0, a.T};
    load_window<T, K, kW>(px, a.xs, pt, a.D, q, t0, win);
    for (int t = t0; t < t1 + K - 1; t += kAhead) {
      RawVec<T, kW> nx[kAhead], ng[kAhead];
#pragma unroll
      for (int s = 0; s < kAhead; ++s)
        if (t + s < t1 + K - 1 && t + s < a.T) {
          nx[s] = raw<T, kW>(px + (long long)(t + s) * a.xs);
          ng[s] = raw<T, kW>(pg + (size_t)(t + s) * a.D);
        }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        if (t + s >= t1 + K - 1) break;
        const bool real = t + s < a.T;
        if (real && t + s >= q.end) {
          q = locate(cu, a.N, a.T, t + s);
          load_window<T, K, kW>(px, a.xs, pt, a.D, q, t + s, win);
        }
        float v[kW] = {}, dz[kW] = {};
        if (real && q.n >= 0) {
          float g[kW];
          widen(nx[s], v);
          widen(ng[s], g);
#pragma unroll
          for (int k = 0; k < kW; ++k) {
            dz[k] = g[k] * slope<T>(product<K, kW>(wt, bias, win, v, k), a.silu);
            if (t + s < t1) {
              sum[K][k] += dz[k];
              sum[K - 1][k] = fmaf(dz[k], v[k], sum[K - 1][k]);
#pragma unroll
              for (int j = 0; j < K - 1; ++j) sum[K - 2 - j][k] = fmaf(dz[k], win[j][k], sum[K - 2 - j][k]);
            }
          }
        }
        // terms of dz for the steps before it, as far back as the sequence goes
        float out[kW];
#pragma unroll
        for (int j = K - 2; j >= 0; --j)
#pragma unroll
          for (int k = 0; k < kW; ++k) {
            const float more = t + s - 1 - j >= q.begin ? fmaf(wt[K - 2 - j][k], dz[k], acc[j][k]) : acc[j][k];
            if (j == K - 2)
              out[k] = more;
            else
              acc[j + 1][k] = more;
          }
#pragma unroll
        for (int k = 0; k < kW; ++k) acc[0][k] = wt[K - 1][k] * dz[k];
        if (t + s - (K - 1) >= t0) save<T, kW>(pd + (size_t)(t + s - (K - 1)) * a.D, out);
        shift<K, kW>(win, v);
      }
    }
  }
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int k = 0; k < kW; ++k) red[warp][j * kW + k][lane] = sum[j][k];
  __syncthreads();
  // part [rows, K + 1, D]
  float* to = part + ((size_t)axis * (gridDim.x / slabs) + chunk) * (K + 1) * a.D;
  for (int e = threadIdx.x; e < (K + 1) * kW * 32; e += kThreads) {
    const int j = e / (kW * 32), col = e - j * (kW * 32);  // col: channel of the slab
    const int ch = (blockIdx.x - chunk * slabs) * 32 * kW + col;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) s += red[v][j * kW + col % kW][col / kW];
    if (ch < a.D) to[(size_t)j * a.D + ch] = s;
  }
}

// dw[c][j] and db[c] from n rows of partial sums: 32 channels a block, 32 rows at a time; blockIdx.y: the tap, K: db.
__global__ void __launch_bounds__(1024) k_conv_sums(const float* __restrict__ part, int n, int D, int K, void* dw, void* db,
                                                     bool wbf16) {
  __shared__ float s[32][33];
  const int j = blockIdx.y;
  if (j == K ? !db : !dw) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int i = threadIdx.y; i < n; i += 32) v += part[((size_t)i * (K + 1) + j) * D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x != 0 || col >= D) return;
  const size_t at = j == K ? (size_t)col : (size_t)col * K + j;
  if (wbf16)
    static_cast<bf16*>(j == K ? db : dw)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(j == K ? db : dw)[at] = v;
}

// The gradients of the taps: a thread has a channel of a sequence, and its first K - 1 steps.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) k_conv_dtaps(Args a, const T* __restrict__ dy, const T* __restrict__ x,
                                                         const void* __restrict__ w, const void* __restrict__ b,
                                                         const T* __restrict__ taps, const int* __restrict__ cu, T* dtaps) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.D) return;
  float wt[K][1], bias[1];
  load_weights<K, 1>(w, b, a.wbf16, c, wt, bias);
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    const size_t row0 = a.packed ? 0 : (size_t)n * a.T;
    const Seq q = a.packed ? Seq{n, clamp_cu(cu, n, a.T), clamp_cu(cu, n + 1, a.T)} : Seq{n, 0, a.T};
    float win[K - 1][1], out[K - 1] = {};
    load_window<T, K, 1>(x + row0 * a.xs + c, a.xs, taps ? taps + c : nullptr, a.D, q, q.begin, win);
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
      if (q.begin + t >= q.end) break;
      float v[1], g[1];
      load<T, 1>(x + (row0 + q.begin + t) * a.xs + c, v);
      load<T, 1>(dy + (row0 + q.begin + t) * a.D + c, g);
      const float dz = g[0] * slope<T>(product<K, 1>(wt, bias, win, v, 0), a.silu);
#pragma unroll
      for (int j = t + 1; j < K; ++j) out[K - 1 + t - j] = fmaf(wt[K - 1 - j][0], dz, out[K - 1 + t - j]);
      shift<K, 1>(win, v);
    }
#pragma unroll
    for (int p = 0; p < K - 1; ++p) {
      const float o[1] = {out[p]};
      save<T, 1>(dtaps + ((size_t)n * (K - 1) + p) * a.D + c, o);
    }
  }
}

// Steps of every sequence on its slot of a cache of taps [slots, K - 1, D], for serving.
template <typename T, int K, int kW>
__global__ void __launch_bounds__(128) k_conv_step(Args a, const T* __restrict__ x, const void* __restrict__ w,
                                                   const void* __restrict__ b, T* state, const int* __restrict__ slots,
                                                   long long num_slots, T* y) {
  const int c = (blockIdx.x * 128 + threadIdx.x) * kW;
  if (c >= a.D) return;
  float wt[K][kW], bias[kW];
  load_weights<K, kW>(w, b, a.wbf16, c, wt, bias);
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    const long long slot = slots ? slots[n] : n;
    const bool held = slot >= 0 && slot < num_slots;  // else: a place without a sequence, y = 0
    T* s = state + (held ? (size_t)slot * (K - 1) * a.D : 0) + c;
    float win[K - 1][kW] = {};
    if (held) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) load<T, kW>(s + (size_t)(K - 2 - j) * a.D, win[j]);
    }
    for (int t = 0; t < a.T; ++t) {
      const size_t at = (size_t)n * a.T + t;
      float v[kW] = {}, o[kW] = {};
      if (held) {
        load<T, kW>(x + at * a.xs + c, v);
#pragma unroll
        for (int k = 0; k < kW; ++k) o[k] = act<T>(product<K, kW>(wt, bias, win, v, k), a.silu);
        shift<K, kW>(win, v);
      }
      save<T, kW>(y + at * a.D + c, o);
    }
    if (held) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) save<T, kW>(s + (size_t)(K - 2 - j) * a.D, win[j]);
    }
  }
}

int axes(const Args& a) { return a.packed ? 1 : a.N; }
long long chunks(const Args& a) { return ((long long)a.T + (long long)a.run * kWarps - 1) / ((long long)a.run * kWarps); }
int slabs(const Args& a, int kW) { return (a.D + 32 * kW - 1) / (32 * kW); }

template <typename T, int K, int kW>
void forward_of(const Call& c, cudaStream_t st) {
  const int s = slabs(c.a, kW);
  const dim3 grid((unsigned)(chunks(c.a) * s), axes(c.a));
  SSD_LAUNCH("k_conv_forward", st,
             k_conv_forward<T, K, kW><<<grid, kThreads, 0, st>>>(c.a, (const T*)c.x, c.w, c.b, (const T*)c.taps, c.cu,
                                                                 (T*)c.y, (T*)c.taps_out, s));
}
template <typename T, int K, int kW>
void backward_of(const Call& c, cudaStream_t st) {
  const int s = slabs(c.a, kW);
  const dim3 grid((unsigned)(chunks(c.a) * s), axes(c.a));
  SSD_LAUNCH("k_conv_backward", st,
             k_conv_backward<T, K, kW><<<grid, kThreads, 0, st>>>(c.a, (const T*)c.dy, (const T*)c.x, c.w, c.b,
                                                                  (const T*)c.taps, c.cu, (T*)c.dx, c.part, s));
  if (c.dw || c.db)
    SSD_LAUNCH("k_conv_sums", st,
               k_conv_sums<<<dim3((c.a.D + 31) / 32, K + 1), dim3(32, 32), 0, st>>>(
                   c.part, (int)(axes(c.a) * chunks(c.a)), c.a.D, K, c.dw, c.db, c.a.wbf16));
  if (c.dtaps)
    SSD_LAUNCH("k_conv_dtaps", st,
               k_conv_dtaps<T, K><<<dim3((c.a.D + kThreads - 1) / kThreads, c.a.N < 65535 ? c.a.N : 65535), kThreads, 0, st>>>(
                   c.a, (const T*)c.dy, (const T*)c.x, c.w, c.b, (const T*)c.taps, c.cu, (T*)c.dtaps));
}
template <typename T, int K, int kW>
void step_of(const Call& c, void* state, const int32_t* slots, long long num_slots, cudaStream_t st) {
  const int groups = (c.a.D + kW - 1) / kW;
  SSD_LAUNCH("k_conv_step", st,
             k_conv_step<T, K, kW><<<dim3((groups + 127) / 128, c.a.N < 65535 ? c.a.N : 65535), 128, 0, st>>>(
                 c.a, (const T*)c.x, c.w, c.b, (T*)state, slots, num_slots, (T*)c.y));
}

// Runs f<T, K, kW> for a call's type, taps and width: four channels a thread where every row is whole, aligned pieces.
template <typename F>
void by_shape(const Call& c, bool whole, const F& f) {
  const auto width = [&](auto t, auto k) {
    if (whole)
      f(t, k, std::integral_constant<int, 4>());
    else
      f(t, k, std::integral_constant<int, 1>());
  };
  const auto taps = [&](auto t) {
    if (c.a.K == 2)
      width(t, std::integral_constant<int, 2>());
    else if (c.a.K == 3)
      width(t, std::integral_constant<int, 3>());
    else
      width(t, std::integral_constant<int, 4>());
  };
  if (c.a.f32)
    taps(float());
  else
    taps(bf16());
}

ssd_status make_args(const ssd_conv_problem* p, Args* a) {
  if (!p) return SSD_ERR_INVALID_ARG;
  for (const int32_t d : {p->io_dtype, p->weight_dtype})
    if (d != SSD_F32 && d != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if ((p->packed != 0 && p->packed != 1) || (p->activation != SSD_ACT_NONE && p->activation != SSD_ACT_SILU))
    return SSD_ERR_INVALID_ARG;
  if (p->batch < 1 || p->seqlen < 1 || p->dim < 1 || p->taps < 1 || p->x_stride < 0) return SSD_ERR_INVALID_ARG;
  if (p->taps < 2 || p->taps > 4 || (p->x_stride && p->x_stride < p->dim)) return SSD_ERR_SHAPE;
  if (p->seqlen > 0x7ffff000ll || p->batch > 0x1fffffffll || p->dim > (1 << 20)) return SSD_ERR_SHAPE;
  if (!p->packed && (p->batch > 65535 || p->batch * p->seqlen > 0x7fffffffll)) return SSD_ERR_SHAPE;
  *a = Args{};
  a->N = (int)p->batch;
  a->T = (int)p->seqlen;
  a->D = (int)p->dim;
  a->K = (int)p->taps;
  a->packed = p->packed == 1;
  a->f32 = p->io_dtype == SSD_F32;
  a->wbf16 = p->weight_dtype == SSD_BF16;
  a->silu = p->activation == SSD_ACT_SILU;
  a->xs = p->x_stride ? p->x_stride : p->dim;
  // Long runs read little twice, short ones give work to the whole GPU: the longest of 64, 32, 16 and 8 steps that leaves
  // about 24 warps an SM.  The grid and the rows of partial sums stay within bounds by longer runs.
  long long run = 64;
  const long long rows = (long long)axes(*a) * a->T, warps = 152 * 24;
  while (run > 8 && rows / run * ((a->D + 127) / 128) < warps) run /= 2;
  while (rows / (run * kWarps) > 4096) run *= 2;
  a->run = (int)(run < 0x40000000ll ? run : 0x40000000ll);
  return SSD_OK;
}

size_t workspace(Call* c, void* ws) {
  Carver cv(ws);
  c->part = cv.take<float>((size_t)axes(c->a) * chunks(c->a) * (c->a.K + 1) * c->a.D);
  return cv.off;
}

ssd_status check_inputs(const Call& c) {
  const uintptr_t elem = c.a.f32 ? 4 : 2, we = c.a.wbf16 ? 2 : 4;
  if (!c.x || !c.w) return SSD_ERR_INVALID_ARG;
  if (off(c.x, elem) || off(c.w, we) || off(c.b, we) || off(c.taps, elem) || off(c.cu, 4)) return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}
// Rows of whole four-element pieces that lie at multiples of their size.
bool whole(const Call& c, std::initializer_list<const void*> tensors) {
  const uintptr_t piece = c.a.f32 ? 16 : 8, wp = c.a.wbf16 ? 8 : 16;
  if (c.a.D % 4 || c.a.xs % 4 || off(c.w, wp) || off(c.b, wp)) return false;
  for (const void* p : tensors)
    if (off(p, piece)) return false;
  return true;
}

}  // namespace
}  // namespace conv
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_conv_workspace_size(const ssd_conv_problem* prob, size_t* bytes) {
  conv::Call c = {};
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = conv::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  *bytes = conv::workspace(&c, nullptr);
  return SSD_OK;
}

ssd_status ssd_conv_forward(const ssd_conv_problem* prob, const void* x, const void* weight, const void* bias, const void* taps,
                            const int32_t* cu_seqlens, void* y, void* taps_final, void* cuda_stream) {
  conv::Call c = {};
  ssd_status s = conv::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.x = x, c.w = weight, c.b = bias, c.taps = taps, c.cu = cu_seqlens, c.y = y, c.taps_out = taps_final;
  if (!y || c.a.packed != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
  if ((s = conv::check_inputs(c)) != SSD_OK) return s;
  if (off(y, c.a.f32 ? 4 : 2) || off(taps_final, c.a.f32 ? 4 : 2)) return SSD_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  conv::by_shape(c, conv::whole(c, {x, taps, y, taps_final}), [&](auto t, auto k, auto w) {
    conv::forward_of<decltype(t), decltype(k)::value, decltype(w)::value>(c, st);
  });
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_conv_backward(const ssd_conv_problem* prob, const void* dy, const void* x, const void* weight, const void* bias,
                             const void* taps, const int32_t* cu_seqlens, void* dx, void* dw, void* db, void* dtaps, void* ws,
                             size_t ws_bytes, void* cuda_stream) {
  conv::Call c = {};
  ssd_status s = conv::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.dy = dy, c.x = x, c.w = weight, c.b = bias, c.taps = taps, c.cu = cu_seqlens;
  c.dx = dx, c.dw = dw, c.db = db, c.dtaps = dtaps;
  if (!dy || !dx || !ws || c.a.packed != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
  if ((s = conv::check_inputs(c)) != SSD_OK) return s;
  const uintptr_t elem = c.a.f32 ? 4 : 2, we = c.a.wbf16 ? 2 : 4;
  if (off(dy, elem) || off(dx, elem) || off(dw, we) || off(db, we) || off(dtaps, elem) || off(ws, 16)) return SSD_ERR_ALIGNMENT;
  if (ws_bytes < conv::workspace(&c, nullptr)) return SSD_ERR_WORKSPACE;
  conv::workspace(&c, ws);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  conv::by_shape(c, conv::whole(c, {x, taps, dy, dx}), [&](auto t, auto k, auto w) {
    conv::backward_of<decltype(t), decltype(k)::value, decltype(w)::value>(c, st);
  });
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_conv_step(const ssd_conv_problem* prob, const void* x, const void* weight, const void* bias, void* state,
                         const int32_t* slots, int64_t num_slots, void* y, void* cuda_stream) {
  conv::Call c = {};
  ssd_status s = conv::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.x = x, c.w = weight, c.b = bias, c.y = y;
  if (c.a.packed || num_slots < 1 || (!slots && num_slots < c.a.N) || !state || !y) return SSD_ERR_INVALID_ARG;
  if ((s = conv::check_inputs(c)) != SSD_OK) return s;
  const uintptr_t elem = c.a.f32 ? 4 : 2;
  if (off(state, elem) || off(y, elem) || off(slots, 4)) return SSD_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  conv::by_shape(c, conv::whole(c, {x, state, y}), [&](auto t, auto k, auto w) {
    conv::step_of<decltype(t), decltype(k)::value, decltype(w)::value>(c, state, slots, num_slots, st);
  });
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
