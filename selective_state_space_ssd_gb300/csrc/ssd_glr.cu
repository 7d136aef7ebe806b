// The gated linear recurrence with one decay per channel: over whole sequences, forward and backward.
//
// Per channel, with s the sigmoid and ksp = -scale softplus(lam):
//     g = ksp s(r),  a = e^g,  m = sqrt(1 - a^2),  u = s(i) x,   h_t = a_t h_{t-1} + m_t u_t,   y = h
//     dh_t = dy_t + D_{t+1},  D_t = a_t dh_t,   q = dL/dg g = dh (a h_{t-1} g - a^2 u g / m)
//     dx = dh m s(i),  di = dh m u (1 - s(i)),  dr = q (1 - s(r)),  dlam = s(lam) / softplus(lam) sum q
// p = e^g - 1 is summed as a series where g is small, a = 1 + p and m^2 = -p (2 + p): 1 - a^2 of a rounded a would lose
// what a slow decay (a near 1) is about.  g / m goes to 0 with g, so a gate that is shut has finite gradients.
//
// A step is an affine map h -> a h + b of each channel, and maps compose: (A, B) after (A', B') is (A A', A B' + B).  A
// block takes 32 words of channels (64 in bf16, 32 in fp32: rows of 128 bytes) and walks the sequence in tiles; a warp has
// kRun steps of a tile, a thread its word's channels.  The runs' maps are joined through shared memory in order, and the
// state goes from tile to tile in registers.
// In packed batches the first step of a sequence starts anew (b + a h0); the map of a run that holds one has A = -0, which
// says that nothing before it counts, not even a NaN.
#include <initializer_list>

#include "glr_common.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kFwdRun = 8, kBwdRun = 4;  // steps a thread has of a tile of 8 warps
static_assert(kMark == kBwdRun * kWarps && kFwdRun * kWarps % kMark == 0, "the backward's tiles begin where states are kept");
constexpr int kStages = 3;  // tiles in shared memory or on their way there

// A step's place in a packed batch: its sequence, whether it is its first or last one; -1: of no sequence.
constexpr int kFirst = 1 << 30, kLast = 1 << 29, kSeq = kLast - 1;
__device__ __forceinline__ int clamp_cu(const int* cu, int n, int T) { return min(max(cu[n], 0), T); }
__device__ __forceinline__ int code_of(const int* cu, int N, int T, int t) {
  if (t >= T) return -1;
  int lo = 0, hi = N;  // the last n with cu[n] <= t, or -1
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (clamp_cu(cu, mid, T) <= t)
      lo = mid + 1;
    else
      hi = mid - 1;
  }
  if (hi < 0 || hi >= N) return -1;
  return hi | (clamp_cu(cu, hi, T) == t ? kFirst : 0) | (clamp_cu(cu, hi + 1, T) == t + 1 ? kLast : 0);
}

// (A, B) before (a, b): what comes first is forgotten where A of the later map is -0.
__device__ __forceinline__ float apply(float a, float b, float h) { return signbit(a) ? b : fmaf(a, h, b); }

// Copies a tile of `kArrays` arrays to a stage: [array][step][32 words].  kVec: 16-byte pieces; otherwise each thread copies
// the words that it reads itself, element by element.  Steps from T on and channels from D on are zeros.
template <typename T, bool kVec, int kRun, int kArrays>
__device__ __forceinline__ void fetch(uint32_t* stage, const T* const (&src)[kArrays], const long long (&stride)[kArrays],
                                      int t0, int steps, int c0, int D) {
  constexpr int L = kRun * kWarps, CPT = 4 / sizeof(T);
  if constexpr (kVec) {
    constexpr int PW = 16 / sizeof(T);
#pragma unroll
    for (int p = threadIdx.x; p < L * 8; p += kThreads) {
      const int row = p >> 3, c = c0 + (p & 7) * PW;
      const bool ok = t0 + row < steps && c < D;
#pragma unroll
      for (int a = 0; a < kArrays; ++a)
        copy16(stage + (a * L + row) * 32 + (p & 7) * 4, ok ? src[a] + (long long)(t0 + row) * stride[a] + c : src[a], ok);
    }
  } else {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = c0 + lane * CPT;
#pragma unroll
    for (int s = 0; s < kRun; ++s) {
      const int row = w * kRun + s;
#pragma unroll
      for (int a = 0; a < kArrays; ++a) {
        const T* p = src[a] + (long long)(t0 + row) * stride[a] + c;
        uint32_t* to = stage + (a * L + row) * 32 + lane;
        if constexpr (CPT == 1) {
          const bool ok = t0 + row < steps && c < D;
          copy4(to, ok ? p : src[a], ok);
        } else {
          uint32_t v = 0;
          if (t0 + row < steps) {
            if (c < D) v = *reinterpret_cast<const uint16_t*>(p);
            if (c + 1 < D) v |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 1) << 16;
          }
          *to = v;
        }
      }
    }
  }
}

// Stores a thread's channels of a step (CPT of them from channel c on; pair: rows are whole words).
template <typename T>
__device__ __forceinline__ void store(T* row, int c, int D, bool pair, const float (&v)[4 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    if (c < D) row[c] = v[0];
  } else if (pair) {
    if (c < D) *reinterpret_cast<uint32_t*>(row + c) = pack2(v[0], v[1]);
  } else {
    if (c < D) row[c] = __float2bfloat16_rn(v[0]);
    if (c + 1 < D) row[c + 1] = __float2bfloat16_rn(v[1]);
  }
}

// What sequences without steps leave behind: their first state, or zeros (the backward: the last state's gradient).
template <int W>
__device__ __forceinline__ void empty_sequences(const int* cu, const Args& a, int c0, const float* from, float* to) {
  for (long long e = threadIdx.x; e < (long long)a.N * W; e += kThreads) {
    const int n = (int)(e / W), c = c0 + (int)(e % W);
    if (c < a.D && clamp_cu(cu, n + 1, a.T) <= clamp_cu(cu, n, a.T))
      to[(size_t)n * a.D + c] = from ? from[(size_t)n * a.D + c] : 0.f;
  }
}

// y, the final states and the marks (the states that enter every kMark-th step).  Grid: 32-word slabs x sequences (one for
// a packed batch).
template <typename T, bool kVec, bool kPacked>
__global__ void __launch_bounds__(kThreads, 2)
    k_glr_forward(Args a, const T* __restrict__ x, const T* __restrict__ r, const T* __restrict__ i,
                  const float* __restrict__ lam, const float* __restrict__ h0, const int* __restrict__ cu, T* y,
                  float* h_final, float* marks) {
  constexpr int CPT = 4 / sizeof(T), W = 32 * CPT, L = kFwdRun * kWarps, kA = 3;
  extern __shared__ uint32_t ring[];  // [kStages][kA][L][32]
  __shared__ float agg[2][kWarps][2 * CPT][32];
  __shared__ int code[3][L];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c0 = blockIdx.x * W, c = c0 + lane * CPT, axis = blockIdx.y;
  const bool pair = a.D % 2 == 0;
  const size_t row0 = (size_t)axis * a.T;
  const T* const src[kA] = {x + row0 * a.xs, r + row0 * a.rs, i + row0 * a.is};
  const long long stride[kA] = {a.xs, a.rs, a.is};
  const int nt = (a.T + L - 1) / L, nm = (a.T + kMark - 1) / kMark;
  float ksp[CPT], carry[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    ksp[k] = c + k < a.D ? -a.scale * softplus_f(lam[c + k]) : 0.f;
    carry[k] = !kPacked && h0 && c + k < a.D ? h0[(size_t)axis * a.D + c + k] : 0.f;
  }
  if (kPacked && h_final) empty_sequences<W>(cu, a, c0, h0, h_final);
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    fetch<T, kVec, kFwdRun, kA>(ring + s * kA * L * 32, src, stride, s * L, a.T, c0, a.D);
    copies_commit();
  }
  if (kPacked && threadIdx.x < L) code[0][threadIdx.x] = code_of(cu, a.N, a.T, threadIdx.x);
  copies_wait<kStages - 1>();
  __syncthreads();
  for (int j = 0; j < nt; ++j) {
    const uint32_t* stage = ring + (j % kStages) * kA * L * 32;
    const int t0 = j * L + w * kFwdRun;
    uint32_t first = 0, last = 0, dead = 0;
    if (kPacked) {
      const int cd = lane < kFwdRun ? code[j % 3][w * kFwdRun + lane] : 0;
      dead = __ballot_sync(0xffffffffu, cd < 0);
      first = __ballot_sync(0xffffffffu, cd < 0 || (cd & kFirst));
      last = __ballot_sync(0xffffffffu, cd >= 0 && (cd & kLast));
    }
    float av[kFwdRun][CPT], bv[kFwdRun][CPT], A[CPT], B[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) A[k] = 1.f, B[k] = 0.f;
#pragma unroll
    for (int s = 0; s < kFwdRun; ++s) {
      float xv[CPT], rv[CPT], iv[CPT];
      const uint32_t* p = stage + (w * kFwdRun + s) * 32 + lane;
      unpack(p[0], xv);
      unpack(p[L * 32], rv);
      unpack(p[2 * L * 32], iv);
      const bool start = kPacked && (first >> s & 1), none = kPacked ? (dead >> s & 1) : t0 + s >= a.T;
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        float m;
        gates<T>(rv[k], ksp[k], av[s][k], m);
        bv[s][k] = m * (sigmoid<T>(iv[k]) * xv[k]);
        if (none) av[s][k] = 1.f, bv[s][k] = 0.f;
      }
      if (kPacked && start) {
        if (h0 && !none) {
          const float* from = h0 + (size_t)(code[j % 3][w * kFwdRun + s] & kSeq) * a.D + c;
#pragma unroll
          for (int k = 0; k < CPT; ++k)
            if (c + k < a.D) bv[s][k] = fmaf(av[s][k], from[k], bv[s][k]);
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) av[s][k] = -0.f, A[k] = -0.f, B[k] = bv[s][k];
      } else {
#pragma unroll
        for (int k = 0; k < CPT; ++k) A[k] *= av[s][k], B[k] = fmaf(av[s][k], B[k], bv[s][k]);
      }
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) agg[j & 1][w][2 * k][lane] = A[k], agg[j & 1][w][2 * k + 1][lane] = B[k];
    if (kPacked && threadIdx.x < L) code[(j + 1) % 3][threadIdx.x] = code_of(cu, a.N, a.T, (j + 1) * L + threadIdx.x);
    // one barrier a tile: the runs' maps are there, the next tile has come, and this one's stage is free
    copies_wait<kStages - 2>();
    __syncthreads();
    fetch<T, kVec, kFwdRun, kA>(ring + (j % kStages) * kA * L * 32, src, stride, (j + kStages) * L, a.T, c0, a.D);
    copies_commit();
    float h[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) h[k] = carry[k];
#pragma unroll
    for (int v = 0; v < kWarps; ++v)
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        if (v == w) h[k] = carry[k];
        const float Av = agg[j & 1][v][2 * k][lane], Bv = agg[j & 1][v][2 * k + 1][lane];
        carry[k] = kPacked ? apply(Av, Bv, carry[k]) : fmaf(Av, carry[k], Bv);
      }
    if (marks && t0 % kMark == 0 && t0 < a.T) {
      float* to = marks + ((size_t)axis * nm + t0 / kMark) * a.D + c;
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (c + k < a.D) to[k] = h[k];
    }
#pragma unroll
    for (int s = 0; s < kFwdRun; ++s) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) h[k] = kPacked ? apply(av[s][k], bv[s][k], h[k]) : fmaf(av[s][k], h[k], bv[s][k]);
      if (t0 + s >= a.T) continue;
      if (y) store<T>(y + (row0 + t0 + s) * a.D, c, a.D, pair, h);
      if (h_final && (kPacked ? (last >> s & 1) : t0 + s == a.T - 1)) {
        const int n = kPacked ? code[j % 3][w * kFwdRun + s] & kSeq : axis;
        float* to = h_final + (size_t)n * a.D + c;
#pragma unroll
        for (int k = 0; k < CPT; ++k)
          if (c + k < a.D) to[k] = h[k];
      }
    }
  }
  copies_wait<0>();
}

// The gradients, tile by tile from the end.  The states of a tile are made again from its mark, and the upstream gradients'
// runs are joined as the states' are, in the other direction.  part [axes, D]: the sums of q for dlam.
template <typename T, bool kVec, bool kPacked>
__global__ void __launch_bounds__(kThreads, 2)
    k_glr_backward(Args a, const T* __restrict__ dy, const float* __restrict__ dh_final, const T* __restrict__ x,
                   const T* __restrict__ r, const T* __restrict__ i, const float* __restrict__ lam,
                   const float* __restrict__ h0, const int* __restrict__ cu, const float* __restrict__ marks, T* dx, T* dr,
                   T* di, float* dh0, float* part) {
  constexpr int CPT = 4 / sizeof(T), W = 32 * CPT, L = kBwdRun * kWarps, kA = 4;
  extern __shared__ uint32_t ring[];  // [kStages][kA][L][32]
  __shared__ float agg[2][kWarps][3 * CPT][32];
  __shared__ int code[3][L];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c0 = blockIdx.x * W, c = c0 + lane * CPT, axis = blockIdx.y;
  const bool pair = a.D % 2 == 0;
  const size_t row0 = (size_t)axis * a.T;
  const T* const src[kA] = {x + row0 * a.xs, r + row0 * a.rs, i + row0 * a.is, dy + row0 * a.D};
  const long long stride[kA] = {a.xs, a.rs, a.is, a.D};
  const int nt = (a.T + L - 1) / L;
  float ksp[CPT], back[CPT], qsum[CPT];  // back: D of the step behind the tile
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    ksp[k] = c + k < a.D ? -a.scale * softplus_f(lam[c + k]) : 0.f;
    back[k] = !kPacked && dh_final && c + k < a.D ? dh_final[(size_t)axis * a.D + c + k] : 0.f;
    qsum[k] = 0.f;
  }
  if (kPacked && dh0) empty_sequences<W>(cu, a, c0, dh_final, dh0);
  const auto tile = [&](int j) { return (nt - 1 - j) * L; };  // the first step of the j-th tile from the end
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    if (s < nt) fetch<T, kVec, kBwdRun, kA>(ring + s * kA * L * 32, src, stride, tile(s), a.T, c0, a.D);
    copies_commit();
  }
  if (kPacked && threadIdx.x < L) code[0][threadIdx.x] = code_of(cu, a.N, a.T, tile(0) + threadIdx.x);
  copies_wait<kStages - 1>();
  __syncthreads();
  for (int j = 0; j < nt; ++j) {
    const uint32_t* stage = ring + (j % kStages) * kA * L * 32;
    const int t0 = tile(j) + w * kBwdRun;
    uint32_t first = 0, dead = 0;
    if (kPacked) {
      const int cd = lane < kBwdRun ? code[j % 3][w * kBwdRun + lane] : 0;
      dead = __ballot_sync(0xffffffffu, cd < 0);
      first = __ballot_sync(0xffffffffu, cd < 0 || (cd & kFirst));
    }
    float h[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      h[k] = c + k < a.D ? marks[((size_t)axis * nt + (nt - 1 - j)) * a.D + c + k] : 0.f;
    // per step and channel: a, the state's increment b, g, a^2 u g / m, dx / dh, di / dh, 1 - s(r), dy
    float av[kBwdRun][CPT], bv[kBwdRun][CPT], gv[kBwdRun][CPT], kv[kBwdRun][CPT], mi[kBwdRun][CPT], di1[kBwdRun][CPT],
        r1[kBwdRun][CPT], up[kBwdRun][CPT];
    float A[CPT], B[CPT], R[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) A[k] = 1.f, B[k] = R[k] = 0.f;
#pragma unroll
    for (int s = 0; s < kBwdRun; ++s) {
      float xv[CPT], rv[CPT], iv[CPT];
      const uint32_t* p = stage + (w * kBwdRun + s) * 32 + lane;
      unpack(p[0], xv);
      unpack(p[L * 32], rv);
      unpack(p[2 * L * 32], iv);
      unpack(p[3 * L * 32], up[s]);
      const bool start = kPacked && (first >> s & 1), none = kPacked ? (dead >> s & 1) : t0 + s >= a.T;
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float er = exp_neg<T>(rv[k]), ei = exp_neg<T>(iv[k]), sr = inv(1.f + er), si = inv(1.f + ei);
        gv[s][k] = ksp[k] * sr;
        r1[s][k] = er * sr;
        const float e1 = expm1_neg<T>(gv[s][k]), m2 = -e1 * (2.f + e1), rm = m2 == 0.f ? 0.f : rsqrtf(m2);
        av[s][k] = 1.f + e1;
        mi[s][k] = m2 * rm * si;
        bv[s][k] = mi[s][k] * xv[k];
        di1[s][k] = bv[s][k] * (ei * si);
        kv[s][k] = av[s][k] * av[s][k] * (si * xv[k]) * (gv[s][k] * rm);
        if (none) av[s][k] = 1.f, bv[s][k] = up[s][k] = 0.f;
      }
      if (kPacked) {
        const int cd = code[j % 3][w * kBwdRun + s];
        if (dh_final && cd >= 0 && (cd & kLast)) {
          const float* from = dh_final + (size_t)(cd & kSeq) * a.D + c;
#pragma unroll
          for (int k = 0; k < CPT; ++k)
            if (c + k < a.D) up[s][k] += from[k];
        }
        if (start && h0 && !none) {
          const float* from = h0 + (size_t)(cd & kSeq) * a.D + c;
#pragma unroll
          for (int k = 0; k < CPT; ++k)
            if (c + k < a.D) bv[s][k] = fmaf(av[s][k], from[k], bv[s][k]);
        }
      }
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        B[k] = kPacked && start ? bv[s][k] : fmaf(av[s][k], B[k], bv[s][k]);
        A[k] = kPacked && start ? -0.f : signbit(A[k]) ? A[k] : A[k] * av[s][k];
      }
    }
#pragma unroll
    for (int s = kBwdRun - 1; s >= 0; --s)
#pragma unroll
      for (int k = 0; k < CPT; ++k)  // (what a first step hands on goes to dh0, not to the step before it)
        R[k] = kPacked && (first >> s & 1) ? 0.f : av[s][k] * (up[s][k] + R[k]);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      agg[j & 1][w][3 * k][lane] = A[k];
      agg[j & 1][w][3 * k + 1][lane] = B[k];
      agg[j & 1][w][3 * k + 2][lane] = R[k];
    }
    if (kPacked && threadIdx.x < L && j + 1 < nt)
      code[(j + 1) % 3][threadIdx.x] = code_of(cu, a.N, a.T, tile(j + 1) + threadIdx.x);
    copies_wait<kStages - 2>();
    __syncthreads();
    if (j + kStages < nt)
      fetch<T, kVec, kBwdRun, kA>(ring + (j % kStages) * kA * L * 32, src, stride, tile(j + kStages), a.T, c0, a.D);
    copies_commit();
    float d[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) d[k] = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps - 1; ++v)
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (v < w) {
          const float Av = agg[j & 1][v][3 * k][lane], Bv = agg[j & 1][v][3 * k + 1][lane];
          h[k] = kPacked ? apply(Av, Bv, h[k]) : fmaf(Av, h[k], Bv);
        }
#pragma unroll
    for (int v = kWarps - 1; v >= 0; --v)
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        if (v == w) d[k] = back[k];
        const float Av = agg[j & 1][v][3 * k][lane], Rv = agg[j & 1][v][3 * k + 2][lane];
        back[k] = kPacked ? apply(Av, Rv, back[k]) : fmaf(Av, back[k], Rv);
      }
    // the states before each step, and with them a h_{t-1} g - a^2 u g / m
#pragma unroll
    for (int s = 0; s < kBwdRun; ++s) {
      const bool start = kPacked && (first >> s & 1);
      if (start) {
        const int cd = code[j % 3][w * kBwdRun + s];
#pragma unroll
        for (int k = 0; k < CPT; ++k)
          h[k] = h0 && cd >= 0 && c + k < a.D ? h0[(size_t)(cd & kSeq) * a.D + c + k] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        kv[s][k] = fmaf(av[s][k] * gv[s][k], h[k], -kv[s][k]);
        h[k] = start ? bv[s][k] : fmaf(av[s][k], h[k], bv[s][k]);
      }
    }
#pragma unroll
    for (int s = kBwdRun - 1; s >= 0; --s) {
      const int t = t0 + s;
      const bool none = kPacked ? (dead >> s & 1) : t >= a.T;
      float vx[CPT], vr[CPT], vi[CPT], out[CPT];
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float dh = up[s][k] + d[k], q = dh * kv[s][k];
        d[k] = av[s][k] * dh;
        out[k] = d[k];
        vx[k] = none ? 0.f : dh * mi[s][k];
        vi[k] = none ? 0.f : dh * di1[s][k];
        vr[k] = none ? 0.f : q * r1[s][k];
        qsum[k] += none ? 0.f : q;
      }
      if (kPacked && (first >> s & 1)) {
        const int cd = code[j % 3][w * kBwdRun + s];
        if (dh0 && cd >= 0) {
#pragma unroll
          for (int k = 0; k < CPT; ++k)
            if (c + k < a.D) dh0[(size_t)(cd & kSeq) * a.D + c + k] = out[k];
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) d[k] = 0.f;
      }
      if (t >= a.T) continue;
      if (!kPacked && dh0 && t == 0) {
#pragma unroll
        for (int k = 0; k < CPT; ++k)
          if (c + k < a.D) dh0[(size_t)axis * a.D + c + k] = out[k];
      }
      const size_t at = (row0 + t) * a.D;
      store<T>(dx + at, c, a.D, pair, vx);
      store<T>(dr + at, c, a.D, pair, vr);
      store<T>(di + at, c, a.D, pair, vi);
    }
  }
  copies_wait<0>();
  // the warps' sums of q, in order
  __syncthreads();
#pragma unroll
  for (int k = 0; k < CPT; ++k) agg[0][w][k][lane] = qsum[k];
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) s += agg[0][v][k][lane];
      if (c + k < a.D) part[(size_t)axis * a.D + c + k] = s;
    }
  }
}

// dlam = s(lam) / softplus(lam) sum of n rows of part; the factor goes to 1 where both vanish.
__global__ void __launch_bounds__(1024) k_glr_lam(const float* __restrict__ part, int n, int D, const float* lam, float* dlam) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < n; i += 32) v += part[(size_t)i * D + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < D) {
    const float l = lam[col];
    dlam[col] = v * (l < -60.f ? 1.f : sigmoid_f(l) / softplus_f(l));
  }
}

struct Call {
  Args a;
  const void *dy, *x, *r, *i;
  const float *lam, *h0, *dh_final;
  const int* cu;
  void *y, *dx, *dr, *di;
  float *h_final, *marks, *dh0, *dlam, *part;
};

int axes(const Args& a) { return a.packed ? 1 : a.N; }
long long mark_count(const Args& a) { return (long long)axes(a) * ((a.T + kMark - 1) / kMark) * a.D; }

template <typename T, bool kVec, bool kPacked>
cudaError_t forward_of(const Call& c, cudaStream_t st) {
  constexpr int smem = kStages * 3 * kFwdRun * kWarps * 128;
  const auto kernel = k_glr_forward<T, kVec, kPacked>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int W = 128 / (int)sizeof(T);
  const dim3 grid((c.a.D + W - 1) / W, axes(c.a));
  SSD_LAUNCH("k_glr_forward", st,
             kernel<<<grid, kThreads, smem, st>>>(c.a, (const T*)c.x, (const T*)c.r, (const T*)c.i, c.lam, c.h0, c.cu, (T*)c.y,
                                                  c.h_final, c.marks));
  return cudaGetLastError();
}
template <typename T, bool kVec, bool kPacked>
cudaError_t backward_of(const Call& c, cudaStream_t st) {
  constexpr int smem = kStages * 4 * kBwdRun * kWarps * 128;
  const auto kernel = k_glr_backward<T, kVec, kPacked>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int W = 128 / (int)sizeof(T);
  const dim3 grid((c.a.D + W - 1) / W, axes(c.a));
  SSD_LAUNCH("k_glr_backward", st,
             kernel<<<grid, kThreads, smem, st>>>(c.a, (const T*)c.dy, c.dh_final, (const T*)c.x, (const T*)c.r, (const T*)c.i,
                                                  c.lam, c.h0, c.cu, c.marks, (T*)c.dx, (T*)c.dr, (T*)c.di, c.dh0, c.part));
  return cudaGetLastError();
}
// Whole 16-byte pieces of every row: x, r, i (and dy) are copied by them.
bool whole(const Call& c, bool back) {
  const int w = c.a.f32 ? 4 : 8;
  return !(c.a.D % w || c.a.xs % w || c.a.rs % w || c.a.is % w || off(c.x, 16) || off(c.r, 16) || off(c.i, 16) ||
           (back && off(c.dy, 16)));
}
template <typename T>
cudaError_t forward(const Call& c, cudaStream_t st) {
  if (whole(c, false)) return c.a.packed ? forward_of<T, true, true>(c, st) : forward_of<T, true, false>(c, st);
  return c.a.packed ? forward_of<T, false, true>(c, st) : forward_of<T, false, false>(c, st);
}
template <typename T>
cudaError_t backward(const Call& c, cudaStream_t st) {
  if (whole(c, true)) return c.a.packed ? backward_of<T, true, true>(c, st) : backward_of<T, true, false>(c, st);
  return c.a.packed ? backward_of<T, false, true>(c, st) : backward_of<T, false, false>(c, st);
}

// The workspace of a call: the backward's partial sums, and the marks where no stash is given.
size_t workspace(Call* c, bool stashed, void* ws) {
  Carver cv(ws);
  c->part = cv.take<float>((size_t)axes(c->a) * c->a.D);
  if (!stashed) c->marks = cv.take<float>((size_t)mark_count(c->a));
  return cv.off;
}

ssd_status check_inputs(const Call& c) {
  const uintptr_t elem = c.a.f32 ? 4 : 2;
  if (!c.x || !c.r || !c.i || !c.lam || (c.a.packed != (c.cu != nullptr))) return SSD_ERR_INVALID_ARG;
  if (!(c.a.scale >= 0.f) || c.a.scale > 3e38f) return SSD_ERR_INVALID_ARG;
  if (off(c.x, elem) || off(c.r, elem) || off(c.i, elem) || off(c.lam, 4) || off(c.h0, 4) || off(c.cu, 4))
    return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}

}  // namespace

ssd_status make_args(const ssd_glr_problem* p, Args* a) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if ((p->io_dtype != SSD_F32 && p->io_dtype != SSD_BF16) || (p->packed != 0 && p->packed != 1)) return SSD_ERR_INVALID_ARG;
  if (p->batch < 1 || p->seqlen < 1 || p->dim < 1 || p->x_stride < 0 || p->r_stride < 0 || p->i_stride < 0)
    return SSD_ERR_INVALID_ARG;
  if (p->seqlen > 0x7ffff000ll || p->batch >= kLast || p->dim > 0x7ffff000ll) return SSD_ERR_SHAPE;
  if (!p->packed && (p->batch > 65535 || p->batch * p->seqlen > 0x7fffffffll)) return SSD_ERR_SHAPE;
  for (const int64_t s : {p->x_stride, p->r_stride, p->i_stride})
    if (s && s < p->dim) return SSD_ERR_SHAPE;
  *a = Args{};
  a->N = (int)p->batch;
  a->T = (int)p->seqlen;
  a->D = (int)p->dim;
  a->packed = p->packed == 1;
  a->f32 = p->io_dtype == SSD_F32;
  a->xs = p->x_stride ? p->x_stride : p->dim;
  a->rs = p->r_stride ? p->r_stride : p->dim;
  a->is = p->i_stride ? p->i_stride : p->dim;
  return SSD_OK;
}

}  // namespace glr
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_glr_stash_size(const ssd_glr_problem* prob, size_t* bytes) {
  glr::Args a;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = glr::make_args(prob, &a);
  if (s != SSD_OK) return s;
  *bytes = (size_t)glr::mark_count(a) * 4;
  return SSD_OK;
}

ssd_status ssd_glr_workspace_size(const ssd_glr_problem* prob, int stashed, size_t* bytes) {
  glr::Call c = {};
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = glr::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  *bytes = glr::workspace(&c, stashed != 0, nullptr);
  return SSD_OK;
}

ssd_status ssd_glr_forward(const ssd_glr_problem* prob, const void* x, const void* r, const void* i, const float* lam,
                           const float* h0, const int32_t* cu_seqlens, float scale, void* y, float* h_final, void* stash,
                           size_t stash_bytes, void* cuda_stream) {
  glr::Call c = {};
  ssd_status s = glr::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.a.scale = scale;
  c.x = x, c.r = r, c.i = i, c.lam = lam, c.h0 = h0, c.cu = cu_seqlens;
  if ((s = glr::check_inputs(c)) != SSD_OK) return s;
  if (!y) return SSD_ERR_INVALID_ARG;
  if (off(y, 16) || off(h_final, 4) || off(stash, 16)) return SSD_ERR_ALIGNMENT;
  if (stash && stash_bytes < (size_t)glr::mark_count(c.a) * 4) return SSD_ERR_WORKSPACE;
  c.y = y, c.h_final = h_final, c.marks = static_cast<float*>(stash);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = c.a.f32 ? glr::forward<float>(c, st) : glr::forward<bf16>(c, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_glr_backward(const ssd_glr_problem* prob, const void* dy, const float* dh_final, const void* x, const void* r,
                            const void* i, const float* lam, const float* h0, const int32_t* cu_seqlens, float scale,
                            void* dx, void* dr, void* di, float* dlam, float* dh0, const void* stash, size_t stash_bytes,
                            void* ws, size_t ws_bytes, void* cuda_stream) {
  glr::Call c = {};
  ssd_status s = glr::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.a.scale = scale;
  c.x = x, c.r = r, c.i = i, c.lam = lam, c.h0 = h0, c.cu = cu_seqlens;
  if ((s = glr::check_inputs(c)) != SSD_OK) return s;
  if (!dy || !dx || !dr || !di || !dlam || !ws) return SSD_ERR_INVALID_ARG;
  if (off(dy, c.a.f32 ? 4 : 2) || off(dh_final, 4) || off(dx, 16) || off(dr, 16) || off(di, 16) ||
      off(dlam, 4) || off(dh0, 4) || off(stash, 16) || off(ws, 16))
    return SSD_ERR_ALIGNMENT;
  if (stash && stash_bytes < (size_t)glr::mark_count(c.a) * 4) return SSD_ERR_WORKSPACE;
  if (ws_bytes < glr::workspace(&c, stash != nullptr, nullptr)) return SSD_ERR_WORKSPACE;
  glr::workspace(&c, stash != nullptr, ws);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (stash)
    c.marks = const_cast<float*>(static_cast<const float*>(stash));
  else
    e = c.a.f32 ? glr::forward<float>(c, st) : glr::forward<bf16>(c, st);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  c.dy = dy, c.dh_final = dh_final, c.dx = dx, c.dr = dr, c.di = di, c.dh0 = dh0;
  e = c.a.f32 ? glr::backward<float>(c, st) : glr::backward<bf16>(c, st);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  SSD_LAUNCH("k_glr_lam", st,
             glr::k_glr_lam<<<(c.a.D + 31) / 32, dim3(32, 32), 0, st>>>(c.part, glr::axes(c.a), c.a.D, lam, dlam));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
