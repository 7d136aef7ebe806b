// The causal short convolution of each channel (depthwise), with bias and SiLU:
//     z_t = bias + sum over j < K of w[K-1-j] x_{t-j},   y = silu(z) = z s(z), or y = z
//     dz = dy y'(z),  dx_t = sum over j of w[K-1-j] dz_{t+j},  dw[K-1-j] = sum over t of dz_t x_{t-j},  dbias = sum of dz
// where the steps are those of one sequence and x before its first one is its K - 1 taps (or zeros).
// All of it is bound by memory.  A warp takes kW channels a lane and a run of steps, and holds what the taps reach back to
// (and, backward, the K - 1 gradients that still miss terms) in registers, so a run reads K - 1 steps more than its own.
// Steps are loaded well before they are used.  The weight's gradient is summed by a thread over its run, by a block
// over its eight runs in order, and over blocks in order by k_conv_sums: nothing depends on timing.
#include <initializer_list>
#include <type_traits>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.h"
#include "pair.cuh"
#include "vec_io.cuh"

namespace ssd {
namespace conv {
namespace {

constexpr int kThreads = 256, kWarps = 8;
// Steps loaded ahead, channels a thread has (where rows are whole pieces of them) and blocks an SM.  Measured, L2 flushed:
// 4 x 4096 steps of 5120 channels forward 66 us with eight steps and 3 blocks (four steps 66, 2 blocks 66, two channels a
// thread 73), 11811 of 1582, one channel a thread, 33 us (four steps 41); backward 112 us with four channels, four steps and 2
// blocks (two channels 137; registers for 3 blocks spill, 300).
constexpr int kAhead = 8, kFwdBlocks = 3, kWide = 4;
constexpr int kBack = 4, kBackBlocks = 2;

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

// kW channels (four, two or one) as pairs; of one channel the second number is idle.
template <int kW>
struct Chan {
  static constexpr int kP = (kW + 1) / 2;
  P p[kP];
};
template <int kW>
__device__ __forceinline__ Chan<kW> chan(const float (&v)[kW]) {
  Chan<kW> c;
#pragma unroll
  for (int i = 0; i < Chan<kW>::kP; ++i) c.p[i] = pair(v[2 * i], kW > 1 ? v[(2 * i + 1) % kW] : 0.f);
  return c;
}
template <int kW>
__device__ __forceinline__ Chan<kW> none() {
  Chan<kW> c;
#pragma unroll
  for (int i = 0; i < Chan<kW>::kP; ++i) c.p[i] = both(0.f);
  return c;
}
template <typename T, int kW>
__device__ __forceinline__ Chan<kW> get(const T* p) {
  float v[kW];
  load<T, kW>(p, v);
  return chan<kW>(v);
}
template <typename T, int kW>
__device__ __forceinline__ void put(T* p, const Chan<kW>& c) {
  float v[kW + 1];
#pragma unroll
  for (int i = 0; i < Chan<kW>::kP; ++i) split(c.p[i], v[2 * i], v[2 * i + 1]);
  float o[kW];
#pragma unroll
  for (int k = 0; k < kW; ++k) o[k] = v[k];
  save<T, kW>(p, o);
}
// As they lie in memory, for steps that are loaded ahead.
template <int kBytes>
struct RawOf;
template <>
struct RawOf<2> {
  using Type = uint16_t;
};
template <>
struct RawOf<4> {
  using Type = uint32_t;
};
template <>
struct RawOf<8> {
  using Type = uint2;
};
template <>
struct RawOf<16> {
  using Type = uint4;
};
template <typename T, int kW>
using Raw = typename RawOf<kW * sizeof(T)>::Type;
template <typename T, int kW>
__device__ __forceinline__ Raw<T, kW> raw(const T* p) {
  return *reinterpret_cast<const Raw<T, kW>*>(p);
}
__device__ __forceinline__ P two(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ P two(uint32_t x, uint32_t y) { return pair(__uint_as_float(x), __uint_as_float(y)); }
template <typename T, int kW>
__device__ __forceinline__ Chan<kW> open(const Raw<T, kW>& r) {
  Chan<kW> c;
  if constexpr (sizeof(T) == 2) {
    if constexpr (kW == 1) c.p[0] = two((uint32_t)r << 16, 0u);
    if constexpr (kW == 2) c.p[0] = two(r);
    if constexpr (kW == 4) c.p[0] = two(r.x), c.p[1] = two(r.y);
  } else {
    if constexpr (kW == 1) c.p[0] = two(r, 0u);
    if constexpr (kW == 2) c.p[0] = two(r.x, r.y);
    if constexpr (kW == 4) c.p[0] = two(r.x, r.y), c.p[1] = two(r.z, r.w);
  }
  return c;
}

template <int K, int kW>
struct Weights {
  Chan<kW> w[K], b;
  __device__ __forceinline__ Weights(const void* wp, const void* bp, bool wbf16, int c) {
    float flat[K * kW];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float v[kW];
      if (wbf16)
        load<bf16, kW>(static_cast<const bf16*>(wp) + (size_t)c * K + i * kW, v);
      else
        load<float, kW>(static_cast<const float*>(wp) + (size_t)c * K + i * kW, v);
#pragma unroll
      for (int k = 0; k < kW; ++k) flat[i * kW + k] = v[k];
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float v[kW];
#pragma unroll
      for (int k = 0; k < kW; ++k) v[k] = flat[k * K + j];
      w[j] = chan<kW>(v);
    }
    b = none<kW>();
    if (bp) b = wbf16 ? get<bf16, kW>(static_cast<const bf16*>(bp) + c) : get<float, kW>(static_cast<const float*>(bp) + c);
  }
};

// win[j] = x_{t-1-j}: steps of the sequence, before its first one its taps.
template <typename T, int K, int kW>
__device__ __forceinline__ void load_window(const T* x, long long xs, const T* taps, int D, const Seq& q, int t,
                                            Chan<kW> (&win)[K - 1]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int at = t - 1 - j;
    win[j] = none<kW>();
    if (q.n < 0) continue;
    if (at >= q.begin)
      win[j] = get<T, kW>(x + (long long)at * xs);
    else if (taps)
      win[j] = get<T, kW>(taps + ((size_t)q.n * (K - 1) + (K - 1 + at - q.begin)) * D);
  }
}
template <int K, int kW>
__device__ __forceinline__ void shift(Chan<kW> (&win)[K - 1], const Chan<kW>& x) {
#pragma unroll
  for (int j = K - 2; j > 0; --j) win[j] = win[j - 1];
  win[0] = x;
}
template <int K, int kW>
__device__ __forceinline__ P product(const Weights<K, kW>& wt, const Chan<kW> (&win)[K - 1], const Chan<kW>& x, int i) {
  P z = fma(wt.w[K - 1].p[i], x.p[i], wt.b.p[i]);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) z = fma(wt.w[K - 2 - j].p[i], win[j].p[i], z);
  return z;
}
__device__ __forceinline__ P act(P z, bool silu) { return silu ? z * sigmoid(z) : z; }
__device__ __forceinline__ P slope(P z, bool silu) {  // s (1 + z (1 - s))
  const P s = sigmoid(z);
  return silu ? s * fma(z, one_less(s), both(1.f)) : both(1.f);
}

// A block: 32 kW channels, eight runs of steps one after another (those of all sequences on one axis, `runs` of each).
// Grid: chunks of eight runs x channel slabs.
template <typename T, int K, int kW>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) k_conv_forward(Args a, const T* __restrict__ x, const void* __restrict__ w,
                                                           const void* __restrict__ b, const T* __restrict__ taps,
                                                           const int* __restrict__ cu, T* y, T* taps_out, int slabs,
                                                           int runs) {
  constexpr int kP = Chan<kW>::kP;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x / slabs, c = ((blockIdx.x - chunk * slabs) * 32 + lane) * kW;
  if (c >= a.D) return;
  if (a.packed && taps_out && chunk == 0)  // sequences without steps keep their taps
    for (int n = warp; n < a.N; n += kWarps)
      if (clamp_cu(cu, n + 1, a.T) <= clamp_cu(cu, n, a.T))
        for (int p = 0; p < K - 1; ++p) {
          const size_t at = ((size_t)n * (K - 1) + p) * a.D + c;
          put<T, kW>(taps_out + at, taps ? get<T, kW>(taps + at) : none<kW>());
        }
  const long long id = (long long)chunk * kWarps + warp;
  const int axis = (int)(id / runs);
  if (axis >= (a.packed ? 1 : a.N)) return;
  const int t0 = (int)(id - (long long)axis * runs) * a.run, t1 = a.T - t0 > a.run ? t0 + a.run : a.T;
  const T* px = x + ((size_t)axis * a.T + t0) * a.xs + c;
  T* py = y + ((size_t)axis * a.T + t0) * a.D + c;
  const T *x0 = x + (size_t)axis * a.T * a.xs + c, *pt = taps ? taps + c : nullptr;
  Seq q = a.packed ? locate(cu, a.N, a.T, t0) : Seq{axis, 0, a.T};
  Raw<T, kW> next[kAhead];
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    if (t0 + s < t1) next[s] = raw<T, kW>(px + s * a.xs);
  const Weights<K, kW> wt(w, b, a.wbf16, c);
  Chan<kW> win[K - 1];
  load_window<T, K, kW>(x0, a.xs, pt, a.D, q, t0, win);
  for (int t = t0; t < t1; t += kAhead) {
    Raw<T, kW> now[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) now[s] = next[s];
    px += kAhead * a.xs;
    if (t + 2 * kAhead <= t1) {
#pragma unroll
      for (int s = 0; s < kAhead; ++s) next[s] = raw<T, kW>(px + s * a.xs);
    } else {
#pragma unroll
      for (int s = 0; s < kAhead; ++s)
        if (t + kAhead + s < t1) next[s] = raw<T, kW>(px + s * a.xs);
    }
    if (t + kAhead <= t1 && t + kAhead < q.end && q.n >= 0) {  // eight steps of one sequence, not its last ones
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const Chan<kW> v = open<T, kW>(now[s]);
        Chan<kW> o;
#pragma unroll
        for (int i = 0; i < kP; ++i) o.p[i] = act(product<K, kW>(wt, win, v, i), a.silu);
        put<T, kW>(py + s * (long long)a.D, o);
        shift<K, kW>(win, v);
      }
    } else {
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        if (t + s >= t1) break;
        if (t + s >= q.end) {
          q = locate(cu, a.N, a.T, t + s);
          load_window<T, K, kW>(x0, a.xs, pt, a.D, q, t + s, win);
        }
        const Chan<kW> v = open<T, kW>(now[s]);
        Chan<kW> o = none<kW>();
        if (q.n >= 0) {
#pragma unroll
          for (int i = 0; i < kP; ++i) o.p[i] = act(product<K, kW>(wt, win, v, i), a.silu);
        }
        put<T, kW>(py + s * (long long)a.D, o);
        shift<K, kW>(win, v);
        if (taps_out && t + s == q.end - 1 && q.n >= 0) {
#pragma unroll
          for (int p = 0; p < K - 1; ++p)
            put<T, kW>(taps_out + ((size_t)q.n * (K - 1) + p) * a.D + c, win[K - 2 - p]);
        }
      }
    }
    py += kAhead * (long long)a.D;
  }
}

template <typename T, int K, int kW>
__global__ void __launch_bounds__(kThreads, kBackBlocks)
    k_conv_backward(Args a, const T* __restrict__ dy, const T* __restrict__ x, const void* __restrict__ w,
                    const void* __restrict__ b, const T* __restrict__ taps, const int* __restrict__ cu, T* dx, float* part,
                    int slabs, int runs) {
  constexpr int kP = Chan<kW>::kP;
  __shared__ float red[kWarps][(K + 1) * kW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x / slabs, c = ((blockIdx.x - chunk * slabs) * 32 + lane) * kW;
  Chan<kW> sum[K + 1];  // dw by tap, dbias
#pragma unroll
  for (int j = 0; j <= K; ++j) sum[j] = none<kW>();
  const long long id = (long long)chunk * kWarps + warp;
  const int axis = (int)(id / runs);
  if (c < a.D && axis < (a.packed ? 1 : a.N)) {
    const int t0 = (int)(id - (long long)axis * runs) * a.run, t1 = a.T - t0 > a.run ? t0 + a.run : a.T;
    const T *x0 = x + (size_t)axis * a.T * a.xs + c, *pt = taps ? taps + c : nullptr;
    const T* px = x0 + (long long)t0 * a.xs;
    const T* pg = dy + ((size_t)axis * a.T + t0) * a.D + c;
    T* pd = dx + (size_t)axis * a.T * a.D + c;
    const Weights<K, kW> wt(w, b, a.wbf16, c);
    Chan<kW> win[K - 1], acc[K - 1];  // acc[j]: dx of step t - 1 - j so far
#pragma unroll
    for (int j = 0; j < K - 1; ++j) acc[j] = none<kW>();
    Seq q = a.packed ? locate(cu, a.N, a.T, t0) : Seq{axis, 0, a.T};
    load_window<T, K, kW>(x0, a.xs, pt, a.D, q, t0, win);
    // A step's dz into the sums and into dx of the steps before it; what is complete by it.
    const auto spread = [&](const Chan<kW>& v, const Chan<kW>& dz, int back, bool own) {
      if (own) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          sum[K].p[i] = sum[K].p[i] + dz.p[i];
          sum[K - 1].p[i] = fma(dz.p[i], v.p[i], sum[K - 1].p[i]);
#pragma unroll
          for (int j = 0; j < K - 1; ++j) sum[K - 2 - j].p[i] = fma(dz.p[i], win[j].p[i], sum[K - 2 - j].p[i]);
        }
      }
      Chan<kW> out;
#pragma unroll
      for (int j = K - 2; j >= 0; --j)
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          // (back: steps of the sequence that lie before this one)
          const P more = j < back ? fma(wt.w[K - 2 - j].p[i], dz.p[i], acc[j].p[i]) : acc[j].p[i];
          if (j == K - 2)
            out.p[i] = more;
          else
            acc[j + 1].p[i] = more;
        }
#pragma unroll
      for (int i = 0; i < kP; ++i) acc[0].p[i] = wt.w[K - 1].p[i] * dz.p[i];
      shift<K, kW>(win, v);
      return out;
    };
    const int last = t1 + K - 1 < a.T ? t1 + K - 1 : a.T;  // of the steps that are read
    Raw<T, kW> nx[kBack], ng[kBack];
#pragma unroll
    for (int s = 0; s < kBack; ++s)
      if (t0 + s < last) {
        nx[s] = raw<T, kW>(px + s * a.xs);
        ng[s] = raw<T, kW>(pg + s * (long long)a.D);
      }
    for (int t = t0; t < t1 + K - 1; t += kBack) {
      Raw<T, kW> rx[kBack], rg[kBack];
#pragma unroll
      for (int s = 0; s < kBack; ++s) rx[s] = nx[s], rg[s] = ng[s];
      px += kBack * a.xs, pg += kBack * (long long)a.D;
      if (t + 2 * kBack <= last) {
#pragma unroll
        for (int s = 0; s < kBack; ++s) {
          nx[s] = raw<T, kW>(px + s * a.xs);
          ng[s] = raw<T, kW>(pg + s * (long long)a.D);
        }
      } else {
#pragma unroll
        for (int s = 0; s < kBack; ++s)
          if (t + kBack + s < last) {
            nx[s] = raw<T, kW>(px + s * a.xs);
            ng[s] = raw<T, kW>(pg + s * (long long)a.D);
          }
      }
      const bool all = t + kBack <= t1;
      if (all && t + kBack <= q.end && q.n >= 0 && t - q.begin >= K - 1) {
        const bool later = t != t0;  // (of the first steps' terms, those for steps before the run are another warp's)
#pragma unroll
        for (int s = 0; s < kBack; ++s) {
          const Chan<kW> v = open<T, kW>(rx[s]), g = open<T, kW>(rg[s]);
          Chan<kW> dz;
#pragma unroll
          for (int i = 0; i < kP; ++i) dz.p[i] = g.p[i] * slope(product<K, kW>(wt, win, v, i), a.silu);
          const Chan<kW> out = spread(v, dz, K, true);
          if (later || s >= K - 1) put<T, kW>(pd + (size_t)(t + s - (K - 1)) * a.D, out);
        }
        continue;
      }
#pragma unroll
      for (int s = 0; s < kBack; ++s) {
        if (t + s >= t1 + K - 1) break;
        const bool real = t + s < a.T;
        if (real && t + s >= q.end) {
          q = locate(cu, a.N, a.T, t + s);
          load_window<T, K, kW>(x0, a.xs, pt, a.D, q, t + s, win);
        }
        Chan<kW> v = none<kW>(), dz = none<kW>();
        if (real && q.n >= 0) {
          v = open<T, kW>(rx[s]);
          const Chan<kW> g = open<T, kW>(rg[s]);
#pragma unroll
          for (int i = 0; i < kP; ++i) dz.p[i] = g.p[i] * slope(product<K, kW>(wt, win, v, i), a.silu);
        }
        const Chan<kW> out = spread(v, dz, t + s - q.begin, real && q.n >= 0 && t + s < t1);
        if (t + s - (K - 1) >= t0) put<T, kW>(pd + (size_t)(t + s - (K - 1)) * a.D, out);
      }
    }
  }
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    float v[2 * kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) split(sum[j].p[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int k = 0; k < kW; ++k) red[warp][j * kW + k][lane] = v[k];
  }
  __syncthreads();
  // part [rows, K + 1, D]
  float* to = part + (size_t)chunk * (K + 1) * a.D;
  for (int e = threadIdx.x; e < (K + 1) * kW * 32; e += kThreads) {
    const int j = e / (kW * 32), col = e - j * (kW * 32);  // col: channel of the slab
    const int ch = (blockIdx.x - chunk * slabs) * 32 * kW + col;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) s += red[v][j * kW + col % kW][col / kW];
    if (ch < a.D) to[(size_t)j * a.D + ch] = s;
  }
}

// dw[c][j] and db[c] from n rows of partial sums: 32 channels a block, blockDim.y rows at a time; blockIdx.y: the tap, K: db.
__global__ void __launch_bounds__(1024) k_conv_sums(const float* __restrict__ part, int n, int D, int K, void* dw, void* db,
                                                     bool wbf16) {
  __shared__ float s[32][32];
  const int j = blockIdx.y;
  if (j == K ? !db : !dw) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int i = threadIdx.y; i < n; i += blockDim.y) v += part[((size_t)i * (K + 1) + j) * D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= D) return;
  for (int i = 1; i < blockDim.y; ++i) v += s[i][threadIdx.x];
  const size_t at = j == K ? (size_t)c : (size_t)c * K + j;
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
  const Weights<K, 1> wt(w, b, a.wbf16, c);
  for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
    const size_t row0 = a.packed ? 0 : (size_t)n * a.T;
    const Seq q = a.packed ? Seq{n, clamp_cu(cu, n, a.T), clamp_cu(cu, n + 1, a.T)} : Seq{n, 0, a.T};
    Chan<1> win[K - 1], out[K - 1];
#pragma unroll
    for (int p = 0; p < K - 1; ++p) out[p] = none<1>();
    load_window<T, K, 1>(x + row0 * a.xs + c, a.xs, taps ? taps + c : nullptr, a.D, q, q.begin, win);
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
      if (q.begin + t >= q.end) break;
      const Chan<1> v = get<T, 1>(x + (row0 + q.begin + t) * a.xs + c);
      const P dz = get<T, 1>(dy + (row0 + q.begin + t) * a.D + c).p[0] * slope(product<K, 1>(wt, win, v, 0), a.silu);
#pragma unroll
      for (int j = t + 1; j < K; ++j) out[K - 1 + t - j].p[0] = fma(wt.w[K - 1 - j].p[0], dz, out[K - 1 + t - j].p[0]);
      shift<K, 1>(win, v);
    }
#pragma unroll
    for (int p = 0; p < K - 1; ++p) put<T, 1>(dtaps + ((size_t)n * (K - 1) + p) * a.D + c, out[p]);
  }
}

// Steps of every sequence on its slot of a cache of taps [slots, K - 1, D], for serving.
template <typename T, int K, int kW>
__global__ void __launch_bounds__(128) k_conv_step(Args a, const T* __restrict__ x, const void* __restrict__ w,
                                                   const void* __restrict__ b, T* state, const int* __restrict__ slots,
                                                   long long num_slots, T* y) {
  const int c = (blockIdx.x * 128 + threadIdx.x) * kW;
  if (c >= a.D) return;
  const Weights<K, kW> wt(w, b, a.wbf16, c);
  const int n = blockIdx.y;
  const long long slot = slots ? slots[n] : n;
  const bool held = slot >= 0 && slot < num_slots;  // else: a place without a sequence, y = 0
  T* s = state + (held ? (size_t)slot * (K - 1) * a.D : 0) + c;
  Chan<kW> win[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) win[j] = held ? get<T, kW>(s + (size_t)(K - 2 - j) * a.D) : none<kW>();
  for (int t = 0; t < a.T; ++t) {
    const size_t at = (size_t)n * a.T + t;
    Chan<kW> o = none<kW>();
    if (held) {
      const Chan<kW> v = get<T, kW>(x + at * a.xs + c);
#pragma unroll
      for (int i = 0; i < Chan<kW>::kP; ++i) o.p[i] = act(product<K, kW>(wt, win, v, i), a.silu);
      shift<K, kW>(win, v);
    }
    put<T, kW>(y + at * a.D + c, o);
  }
  if (held) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) put<T, kW>(s + (size_t)(K - 2 - j) * a.D, win[j]);
  }
}

int axes(const Args& a) { return a.packed ? 1 : a.N; }
int runs(const Args& a) { return (int)(((long long)a.T + a.run - 1) / a.run); }
long long chunks(const Args& a) { return ((long long)axes(a) * runs(a) + kWarps - 1) / kWarps; }
int slabs(const Args& a, int kW) { return (a.D + 32 * kW - 1) / (32 * kW); }

template <typename T, int K, int kW>
void forward_of(const Call& c, cudaStream_t st) {
  const int s = slabs(c.a, kW);
  SSD_LAUNCH("k_conv_forward", st,
             k_conv_forward<T, K, kW><<<(unsigned)(chunks(c.a) * s), kThreads, 0, st>>>(
                 c.a, (const T*)c.x, c.w, c.b, (const T*)c.taps, c.cu, (T*)c.y, (T*)c.taps_out, s, runs(c.a)));
}
template <typename T, int K, int kW>
void backward_of(const Call& c, cudaStream_t st) {
  const int s = slabs(c.a, kW);
  SSD_LAUNCH("k_conv_backward", st,
             k_conv_backward<T, K, kW><<<(unsigned)(chunks(c.a) * s), kThreads, 0, st>>>(
                 c.a, (const T*)c.dy, (const T*)c.x, c.w, c.b, (const T*)c.taps, c.cu, (T*)c.dx, c.part, s, runs(c.a)));
  if (c.dw || c.db) {
    const int n = (int)chunks(c.a);
    SSD_LAUNCH("k_conv_sums", st,
               k_conv_sums<<<dim3((c.a.D + 31) / 32, K + 1), dim3(32, n > 256 ? 32 : 8), 0, st>>>(c.part, n, c.a.D, K, c.dw, c.db,
                                                                                                c.a.wbf16));
  }
  if (c.dtaps)
    SSD_LAUNCH("k_conv_dtaps", st,
               k_conv_dtaps<T, K><<<dim3((c.a.D + kThreads - 1) / kThreads, c.a.N < 65535 ? c.a.N : 65535), kThreads, 0, st>>>(
                   c.a, (const T*)c.dy, (const T*)c.x, c.w, c.b, (const T*)c.taps, c.cu, (T*)c.dtaps));
}
template <typename T, int K, int kW>
void step_of(const Call& c, void* state, const int32_t* slots, long long num_slots, cudaStream_t st) {
  const int groups = (c.a.D + kW - 1) / kW;  // (make_args: 65535 sequences at most)
  SSD_LAUNCH("k_conv_step", st,
             k_conv_step<T, K, kW><<<dim3((groups + 127) / 128, c.a.N), 128, 0, st>>>(
                 c.a, (const T*)c.x, c.w, c.b, (T*)state, slots, num_slots, (T*)c.y));
}

// Runs f<T, K, kW> for a call's type, taps and width: kWide channels a thread where every row is whole, aligned pieces.
template <typename F>
void by_shape(const Call& c, bool whole, const F& f) {
  const auto width = [&](auto t, auto k) {
    if (whole)
      f(t, k, std::integral_constant<int, kWide>());
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
  return SSD_OK;
}
// Steps of a run (a multiple of kAhead): those with which the blocks that fit the GPU at once end soonest, turn after turn; a
// run starts with loads that take about as long as 16 steps.  Forward and backward, us: 20011 steps of 2560 channels 43 and
// 68, in runs of 64 46 and 85; 16384 of 2560 39 and 60, 45 and 74; 4 x 4096 of 5120 66 and 112, 66 and 123.  Planned for four
// channels a thread also where one is taken, which has four times the blocks: 11811 of 1582 33 and 67, in runs of 64 32 and
// 68.  Longer ones where the grid would pass 2^31 blocks.
constexpr int kStart = 16, kMostRun = 256;
void set_run(Args* a, int blocks_of_an_sm) {
  const long long slots = 152 * blocks_of_an_sm;
  long long least = -1;
  int run = kAhead;
  for (a->run = kAhead; a->run <= kMostRun; a->run += kAhead) {
    const long long turns = (chunks(*a) * slabs(*a, kWide) + slots - 1) / slots, end = turns * (a->run + kStart);
    if (least < 0 || end < least) least = end, run = a->run;
    if (turns == 1) break;
  }
  a->run = run;
  while (chunks(*a) * slabs(*a, 1) > 0x7fffffffll) a->run *= 2;
}

size_t workspace(Call* c, void* ws) {
  Carver cv(ws);
  set_run(&c->a, kBackBlocks);
  c->part = cv.take<float>((size_t)chunks(c->a) * (c->a.K + 1) * c->a.D);
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
  conv::set_run(&c.a, conv::kFwdBlocks);
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
  if (ws_bytes < conv::workspace(&c, ws)) return SSD_ERR_WORKSPACE;
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
