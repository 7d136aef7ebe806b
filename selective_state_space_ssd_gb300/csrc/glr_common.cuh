// What the files of the gated linear recurrence share: a call's sizes, the gates of a step, tiles and maps of the scans.
//
// Per channel, with s the sigmoid and n = -g = scale softplus(lam) s(r):
//     a = e^-n,  m = sqrt(1 - a^2),  u = s(i) x,   h_t = a_t h_{t-1} + m_t u_t,   y = h
// o = 1 - e^-n is summed as a series where n is small, a = 1 - o and m^2 = o (1 + a): 1 - a^2 of a rounded a would lose what
// a slow decay (a near 1) is about.
//
// A step is an affine map h -> a h + b of each channel, and maps compose: (A, B) after (A', B') is (A A', A B' + B).  A
// block takes 64 channels, two a lane, and walks a sequence in tiles; each of its 8 or 16 warps has a run of a tile's steps.
// The runs' maps are joined in order through shared memory, and the tiles' maps, where several blocks of a cluster share the
// sequence, through their shared memories.
// In packed batches the first step of a sequence starts anew (b + a h0, and steps of no sequence with zero); the map of a
// run that holds one has A = -0, which says that nothing before it counts, not even a NaN.
#pragma once

#include <cuda_bf16.h>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.h"
#include "pair.cuh"
#include "vec_io.cuh"

namespace ssd {
namespace glr {

// The stash holds the state that enters every so many steps: each run of the backward's threads.
constexpr int mark_of(bool f32) { return f32 ? 4 : 8; }
constexpr int kWidth = 64;     // channels of a block
constexpr int kMostShare = 8;  // blocks that share a sequence, at most
constexpr int kFewWarps = 8, kManyWarps = 16;  // of a block
constexpr long long kMostStride = 1 << 24;  // elements from a step to the next: those of a tile's 256 steps fit 32 bits
constexpr long long kMostSteps = 0x7fff0000;  // of an axis: a few tiles more than it has are counted in 32 bits

struct Args {
  int N, T, D;  // sequences, steps (of each, or of the packed axis), channels
  bool packed, f32;
  long long xs, rs, is;  // elements from a step to the next of x, r, i
  float scale;
  int share;  // blocks of a cluster, which share a sequence's tiles
  int len;    // a packed axis without bounds: its sequences have so many steps each
};

struct Call {
  Args a;
  const void *dy, *x, *r, *i;
  const float *lam, *h0, *dh_final;
  const int* cu;
  void *y, *dx, *dr, *di;
  float *h_final, *marks, *dh0, *dlam, *part;  // part: room for [axes kMostShare, D]
};

inline int axes(const Args& a) { return a.packed ? 1 : a.N; }
inline int slabs(const Args& a) { return (a.D + kWidth - 1) / kWidth; }

ssd_status make_args(const ssd_glr_problem* p, Args* a);  // checks a problem's numbers
cudaError_t forward(const Call& c, cudaStream_t st);
cudaError_t backward(const Call& c, cudaStream_t st, int* rows);  // without the last step of dlam; rows of part

// ------------------------------------------------------------ gates
// 1 - e^-n for n >= 0: the series to n^5 / 5! where n < 1/8 (what is left out is below 5e-8 of the sum), else from e^-n
// itself; kFar: there are channels whose n can be beyond 1/8 (a warp's lanes go one way; most layers' channels are slower).
constexpr float kNear = 0.125f;
template <bool kFar>
__device__ __forceinline__ P one_minus_exp(P n) {
  P s = fma(n, both(1.f / 120.f), both(-1.f / 24.f));
  s = fma(n, s, both(1.f / 6.f));
  s = fma(n, s, both(-0.5f));
  s = fma(n, s, both(1.f));
  s = n * s;
  if (kFar) {
    float n0, n1, s0, s1;
    split(n, n0, n1);
    split(s, s0, s1);
    const float f0 = 1.f - exp2_f(-kLog2e * n0), f1 = 1.f - exp2_f(-kLog2e * n1);
    s = pair(n0 < kNear ? s0 : f0, n1 < kNear ? s1 : f1);
  }
  return s;
}

// scale softplus(lam) of two channels, and whether some lane's n can be beyond 1/8 (n lies between 0 and that).
__device__ __forceinline__ P load_rate(const float* lam, int c, int D, float scale) {
  return pair(c < D ? scale * softplus_f(lam[c]) : 0.f, c + 1 < D ? scale * softplus_f(lam[c + 1]) : 0.f);
}
__device__ __forceinline__ bool any_far(P rate) {
  float x, y;
  split(rate, x, y);
  return __any_sync(0xffffffffu, !(x < kNear) || !(y < kNear));
}

// ------------------------------------------------------------ words: two channels as they lie in memory
template <typename T>
struct Words;
template <>
struct Words<float> {
  using Word = float2;
  static __device__ __forceinline__ P open(float2 w) { return pair(w.x, w.y); }
  static __device__ __forceinline__ float2 close(P p) {
    float2 w;
    split(p, w.x, w.y);
    return w;
  }
};
template <>
struct Words<bf16> {
  using Word = uint32_t;
  static __device__ __forceinline__ P open(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
  static __device__ __forceinline__ uint32_t close(P p) {
    float x, y;
    split(p, x, y);
    return pack2(x, y);
  }
};
// Two channels to p, the second of them if there is one.  kVec: rows are whole words.
template <typename T, bool kVec>
__device__ __forceinline__ void store_row(T* p, bool second, P v) {
  if (kVec) {
    *reinterpret_cast<typename Words<T>::Word*>(p) = Words<T>::close(v);
  } else {
    float x[1], y[1];
    split(v, x[0], y[0]);
    save<T, 1>(p, x);
    if (second) save<T, 1>(p + 1, y);
  }
}
__device__ __forceinline__ P load_two(const float* p, int c, int D) {
  return pair(c < D ? p[c] : 0.f, c + 1 < D ? p[c + 1] : 0.f);
}
__device__ __forceinline__ void store_two(float* p, int c, int D, P v) {
  if (c < D) store_row<float, false>(p + c, c + 1 < D, v);
}

// ------------------------------------------------------------ maps
struct alignas(16) Map {
  P a, b;
};
__device__ __forceinline__ P anew() { return both(-0.f); }  // A of a map that forgets what comes before it
__device__ __forceinline__ bool is_anew(P a) { return __float_as_uint(low(a)) == 0x80000000u; }
template <bool kPacked>
__device__ __forceinline__ P through(const Map& m, P h) {
  const P n = fma(m.a, h, m.b);
  return kPacked && is_anew(m.a) ? m.b : n;
}
// First m, then n.
template <bool kPacked>
__device__ __forceinline__ Map after(const Map& m, const Map& n) {
  Map r;
  r.b = through<kPacked>(n, m.b);
  r.a = kPacked && (is_anew(m.a) || is_anew(n.a)) ? anew() : n.a * m.a;
  return r;
}

// ------------------------------------------------------------ clusters of blocks
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// For warps that wrote nothing the other blocks read: they do not wait for their stores first.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Writes to the place of `p` in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ void store_to(Map* p, int rank, const Map& m) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(m.a.v.x), "f"(m.a.v.y), "f"(m.b.v.x),
               "f"(m.b.v.y)
               : "memory");
}

// ------------------------------------------------------------ steps of a packed axis
// A step's sequence, with whether it is its first or last one; -1: of no sequence.
constexpr int kFirst = 1 << 30, kLast = 1 << 29, kSeq = kLast - 1;
__device__ __forceinline__ int clamp_cu(const int* cu, int n, int T) { return min(max(cu[n], 0), T); }
// n: where to look first (the sequence of a step not far from this one), and what was found.
__device__ __forceinline__ int code_of(const int* cu, const Args& a, int t, int& n) {
  const int N = a.N, T = a.T;
  if (t < 0 || t >= T) return -1;
  if (!cu) {
    const int q = t / a.len, at = t - q * a.len;
    return q | (at == 0 ? kFirst : 0) | (at == a.len - 1 ? kLast : 0);
  }
  int begin = clamp_cu(cu, n, T), end = clamp_cu(cu, n + 1, T);
  if (t < begin || t >= end) {
    int lo = 0, hi = N;  // the last n with cu[n] <= t, or -1
    while (lo <= hi) {
      const int mid = (lo + hi) >> 1;
      if (clamp_cu(cu, mid, T) <= t)
        lo = mid + 1;
      else
        hi = mid - 1;
    }
    if (hi < 0 || hi >= N) return -1;
    n = hi;
    begin = clamp_cu(cu, n, T), end = clamp_cu(cu, n + 1, T);
  }
  return n | (begin == t ? kFirst : 0) | (end == t + 1 ? kLast : 0);
}
// Brings 64 channels of a sequence's state near, for a tile that will read it soon.
__device__ __forceinline__ void prefetch_state(const float* p, int code, int c0, int D) {
  const float* at = p + (size_t)(code & kSeq) * D + c0;
#pragma unroll
  for (int c = 0; c < kWidth; c += 32)
    if (c0 + c < D) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c));
}
// What sequences without steps leave behind: their first state (the backward: the last state's gradient), or zeros.
__device__ __forceinline__ void empty_sequences(const int* cu, const Args& a, int c0, const float* from, float* to) {
  if (!cu) return;
  for (int n = threadIdx.x; n < a.N; n += blockDim.x)
    if (clamp_cu(cu, n + 1, a.T) <= clamp_cu(cu, n, a.T))
      for (int c = c0; c < c0 + kWidth && c < a.D; ++c) to[(size_t)n * a.D + c] = from ? from[(size_t)n * a.D + c] : 0.f;
}
// The steps of a run that begin a sequence, end one, or belong to none (bit s: step s).
struct Bits {
  uint32_t first, last, none;
  int code;  // lane s: step s's
  __device__ __forceinline__ int seq(int s) const { return __shfl_sync(0xffffffffu, code, s) & kSeq; }
};
template <bool kPacked, int kRun>
__device__ __forceinline__ Bits bits_of(const int* code, int t0, int T, int lane) {
  Bits b = {0, 0, 0, 0};
  if (kPacked) {
    const int cd = b.code = lane < kRun ? code[lane] : 0;
    b.none = __ballot_sync(0xffffffffu, cd < 0);
    b.first = __ballot_sync(0xffffffffu, cd < 0 || (cd & kFirst));
    b.last = __ballot_sync(0xffffffffu, cd >= 0 && (cd & kLast));
  } else if (t0 + kRun >= T) {
    const int left = T - t0 > 0 ? T - t0 : 0;  // steps of the run that there are
    b.none = left < kRun ? (1u << kRun) - (1u << left) : 0;
    b.last = left > 0 ? 1u << (left - 1) : 0;
  }
  return b;
}

// ------------------------------------------------------------ tiles on their way to shared memory
// A stage holds a tile of each of kArrays arrays: [array][step][32 words].  kVec: 16-byte pieces; otherwise each thread
// copies the words that it reads itself, four bytes at a time or, where rows of bf16 begin inside such, element by element
// (11811 packed steps forward: 157 us with 1582 channels, 345 with 1583).  Steps outside 0 .. T - 1 are left as they are
// (whatever they hold is masked), channels from D on are zeros.
template <typename T, bool kVec, int kWarps, int kRun, int kArrays>
struct Tiles {
  static constexpr int kThreads = 32 * kWarps, L = kRun * kWarps;
  using Word = typename Words<T>::Word;
  static constexpr int kBytes = kArrays * L * 32 * (int)sizeof(Word);
  static constexpr int PP = 32 * sizeof(Word) / 16, kRows = kThreads / PP, kPasses = kVec ? L / kRows : kRun;
  const T* src[kArrays];      // the first step and channel of the next tile
  uint32_t stride[kArrays];   // elements from a step to the next
  uint32_t from[kArrays];     // elements from src to what this thread copies first
  int t, hop, steps, left;    // the step of that; steps from a tile to the block's next; T; channels from this thread's on
  uint32_t at;                // this thread's place in a stage
  bool inside;                // rows of bf16 begin inside four bytes

  // first: the first tile's first step; hop_tiles: tiles from one to the next (below 0: towards the beginning).
  __device__ __forceinline__ Tiles(const T* const (&rows)[kArrays], const uint32_t (&step)[kArrays], int c0, int D, int T_,
                                   int first, int hop_tiles) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = kVec ? (int)(threadIdx.x % PP) * (16 / (int)sizeof(T)) : 2 * lane, row = kVec ? threadIdx.x / PP : w * kRun;
    left = D - c0 - c;
    t = first + row;
    hop = hop_tiles * L;
    steps = T_;
    at = kVec ? row * 32 * sizeof(Word) + (threadIdx.x % PP) * 16 : (row * 32 + lane) * sizeof(Word);
    inside = false;
#pragma unroll
    for (int a = 0; a < kArrays; ++a) {
      stride[a] = step[a];
      src[a] = rows[a] + c0 + (long long)first * step[a];
      from[a] = row * step[a] + (left > 0 ? c : 0);
      if (!kVec && sizeof(T) == 2 && ((reinterpret_cast<uintptr_t>(rows[a]) & 3) || step[a] % 2)) inside = true;
    }
  }
  // The next tile, to a stage.
  __device__ __forceinline__ void bring(uint8_t* stage) {
#pragma unroll
    for (int q = 0; q < kPasses; ++q) {
      const int tq = t + q * (kVec ? kRows : 1);
      if (tq >= 0 && tq < steps) {
#pragma unroll
        for (int a = 0; a < kArrays; ++a) {
          uint8_t* to = stage + at + (a * L + q * (kVec ? kRows : 1)) * 32 * sizeof(Word);
          const T* p = src[a] + (from[a] + q * (kVec ? kRows : 1) * stride[a]);
          if constexpr (kVec) {
            copy16(to, p, left > 0);
          } else if constexpr (sizeof(T) == 4) {
            copy4(to, p, left > 0);
            copy4(to + 4, left > 1 ? p + 1 : p, left > 1);
          } else if (!inside) {
            copy4_of(to, p, left > 1 ? 4 : left > 0 ? 2 : 0);
          } else {
            uint32_t v = 0;
            if (left > 0) v = *reinterpret_cast<const uint16_t*>(p);
            if (left > 1) v |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 1) << 16;
            *reinterpret_cast<uint32_t*>(to) = v;
          }
        }
      }
    }
    t += hop;
#pragma unroll
    for (int a = 0; a < kArrays; ++a) src[a] += (long long)hop * stride[a];
  }
};

// A number that goes round 0 .. kN - 1.
template <int kN>
struct Ring {
  int at = 0;
  __device__ __forceinline__ void next() { at = at + 1 == kN ? 0 : at + 1; }
};

template <typename... KArgs>
cudaLaunchConfig_t config_of(void (*kernel)(KArgs...), int threads, int smem, cudaLaunchAttribute* attr, int share) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.gridDim = dim3(share);
  cfg.dynamicSmemBytes = smem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = share;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = share > 1 ? 1 : 0;
  return cfg;
}
struct Fit {  // of one kernel: clusters of 1 .. kMostShare blocks that fit at once
  int clusters[kMostShare + 1] = {};
  cudaError_t error = cudaSuccess;
  mutable std::atomic<unsigned long long> allowed{0};
  template <typename Kernel>
  Fit(Kernel kernel, int threads, int smem) {
    error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    for (int s = 1; s <= kMostShare && error == cudaSuccess; ++s) {
      cudaLaunchAttribute attr;
      const cudaLaunchConfig_t cfg = config_of(kernel, threads, smem, &attr, s);
      error = cudaOccupancyMaxActiveClusters(&clusters[s], kernel, &cfg);
    }
  }
  int sharers(const Args& a, int L) const {
    const long long groups = (long long)slabs(a) * axes(a);
    int s = kMostShare;
    while (s > 1 && (clusters[s] < groups || s > (a.T + L - 1) / L)) --s;
    return s;
  }
  bool room(const Args& a, int L) const { return clusters[sharers(a, L)] >= (long long)slabs(a) * axes(a); }
  int rounds(const Args& a, int L) const {  // tiles that a block takes one after another
    const int s = sharers(a, L);
    return ((a.T + L - 1) / L + s - 1) / s;
  }
};
template <typename Shape, typename... Args_>
cudaError_t launch_shape(const char* name, const Fit& fit, Args& a, cudaStream_t st, Args_... args) {
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(Shape::kernel), Shape::smem, fit.allowed);
  if (e == cudaSuccess) e = fit.error;
  if (e != cudaSuccess) return e;
  a.share = fit.sharers(a, Shape::run * Shape::warps);
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config_of(Shape::kernel, 32 * Shape::warps, Shape::smem, &attr, a.share);
  cfg.gridDim = dim3(slabs(a) * a.share, axes(a));
  cfg.stream = st;
  SSD_LAUNCH(name, st, e = cudaLaunchKernelEx(&cfg, Shape::kernel, a, args...));
  return e;
}
// Launches a kernel in clusters of a.share blocks (1: none), which it sets: as many as leave every block a tile and all
// clusters room on the GPU at once, by the runtime's count.  A cluster that has to wait for its turn costs more than it
// brings: 40 slabs of one sequence of 16384 steps take 90 us forward and 166 backward in clusters of six, 110 and 246 in
// clusters of eight, of which only 36 fit.  Blocks of twice the warps, one an SM, where all have room and take fewer tiles
// one after another: 16384 steps of 1024 channels take 62 and 100 us, 66 and 128 in blocks of eight warps; 24318 packed ones
// of 320 79 and 125, 93 and 170.  (16 sequences of 512 steps of 1024 channels, which have no room, would take 33 and 41
// in place of 23 and 33.)
template <typename Few, typename Many, typename... Args_>
cudaError_t launch_cluster(const char* name, Args& a, cudaStream_t st, Args_... args) {
  static const Fit few(Few::kernel, 32 * Few::warps, Few::smem), many(Many::kernel, 32 * Many::warps, Many::smem);
  if (many.room(a, Many::run * Many::warps) && many.rounds(a, Many::run * Many::warps) < few.rounds(a, Few::run * Few::warps))
    return launch_shape<Many>(name, many, a, st, args...);
  return launch_shape<Few>(name, few, a, st, args...);
}
// Many short sequences are taken as one packed axis, as which they lie in memory: in tiles of their own most of a block would
// have no step.  By the tiles that one SM's blocks take one after another, either way (two blocks an SM, and as many sharers
// of the one axis as give them all one): 4096 sequences of 5 steps of 2560 channels take 171 us in place of 2260, 64 of 40
// steps 23 in place of 38, but 1000 of 60 steps of 1024 channels would take 307 in place of 228.
inline Args flattened(const Args& a) {
  const int L = 8 * mark_of(a.f32);
  Args f = a;
  if (a.packed || a.N < 2 || a.T >= L || (long long)a.N * a.T > kMostSteps) return f;
  const long long room = 2 * 152, wide = slabs(a);
  const long long share = room / wide < 1 ? 1 : room / wide < kMostShare ? room / wide : kMostShare;
  const long long apart = (wide * a.N + room - 1) / room;
  const long long joined = ((long long)a.N * a.T + L * share - 1) / (L * share) * ((wide + room - 1) / room);
  if (joined > apart) return f;
  f.packed = true;
  f.len = a.T;
  f.T = a.N * a.T;
  return f;
}
// Whole 16-byte pieces of every row: tiles are copied by them.
inline bool whole(const Call& c, bool back) {
  const int w = c.a.f32 ? 4 : 8;
  return !(c.a.D % w || c.a.xs % w || c.a.rs % w || c.a.is % w || off(c.x, 16) || off(c.r, 16) || off(c.i, 16) ||
           (back && off(c.dy, 16)));
}

}  // namespace glr
}  // namespace ssd
