// Layer norm over the last dimension, forward and backward, with the reductions of the weight's and the bias's
// gradient.  Per row x of D values:
//     mean = sum x / D,   var = sum (x - mean)^2 / D,   rstd = (var + eps)^-1/2,   h = (x - mean) rstd,   y = h w + b
//     dx = rstd (w dy - mean(w dy) - h mean(w dy h)),   dw = sum over rows of dy h,   db = sum over rows of dy
// Both passes are bound by memory: a row is read once and held in registers (the variance is summed from the
// differences to the mean, in a second pass over the registers), sums are fp32.  The backward's blocks each take every
// n-th row and keep their columns' dw and db in registers; one row of partial sums a block goes to the workspace and
// k_norm_columns adds those in block order, so the result does not depend on timing.  Measured: 16384 rows of 2560 bf16
// values with fp32 weights 45 us forward and 59 us backward (3.7 and 4.3 TB/s), 8 us for k_norm_columns; 262144 rows of
// 128 30 us (4.5 TB/s).  Weight and bias are read again for every row, through L1: four bytes for each byte of such a row.
// Rows that are not whole 16-byte pieces are read element by element: 16384 rows of 2559 take 60 us forward and 131 us
// backward.  Where a row is long or so read, the backward's registers do not suffice: at 40 elements a thread element by
// element 272 to 708 bytes are spilled, at 512 threads a row (from 10241 bf16 or 8193 fp32 values on) 48 to 1036.
#pragma once

#include <type_traits>

#include "norm_common.cuh"

namespace ssd {
namespace norm {
namespace {

__device__ __forceinline__ float lo_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(bf16* p, float x) { *p = __float2bfloat16_rn(x); }
template <typename T>
struct Width;  // elements of a 16-byte piece
template <>
struct Width<float> {
  static constexpr int n = 4;
};
template <>
struct Width<bf16> {
  static constexpr int n = 8;
};
__device__ __forceinline__ void as_floats(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void as_floats(const uint4& v, float (&x)[8]) {
  x[0] = lo_f(v.x);
  x[1] = hi_f(v.x);
  x[2] = lo_f(v.y);
  x[3] = hi_f(v.y);
  x[4] = lo_f(v.z);
  x[5] = hi_f(v.z);
  x[6] = lo_f(v.w);
  x[7] = hi_f(v.w);
}
template <typename T, int N>
__device__ __forceinline__ void ld16(const T* p, float (&x)[N]) {
  as_floats(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void st16(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void st16(bf16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
}

// A thread's E elements of a row held by TPR threads.  kVec: pieces of 16 bytes, piece i of thread t at column
// (i TPR + t) W; otherwise single elements, element i at column i TPR + t.
template <typename T, int TPR, int E, bool kVec>
struct Row {
  static constexpr int W = kVec ? Width<T>::n : 1;
  static constexpr int NP = E / W;
  static __device__ __forceinline__ int col(int i, int t) { return (i * TPR + t) * W; }
  template <typename U>
  static __device__ __forceinline__ void load(const U* p, int D, int t, float (&x)[E], float fill) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = col(i, t);
      if constexpr (kVec && W >= Width<U>::n) {
#pragma unroll
        for (int k = 0; k < W; k += Width<U>::n) {
          float y[Width<U>::n];
#pragma unroll
          for (int j = 0; j < Width<U>::n; ++j) y[j] = fill;
          if (c < D) ld16(p + c + k, y);
#pragma unroll
          for (int j = 0; j < Width<U>::n; ++j) x[i * W + k + j] = y[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) x[i * W + j] = c + j < D ? ld1(p + c + j) : fill;
      }
    }
  }
  // The elements as they lie in memory, for a row that is wanted later.
  using Piece = typename std::conditional<kVec, uint4, T>::type;
  static __device__ __forceinline__ void fetch(const T* p, int D, int t, Piece (&r)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = col(i, t);
      r[i] = Piece{};
      if (c < D) r[i] = *reinterpret_cast<const Piece*>(p + c);
    }
  }
  static __device__ __forceinline__ void unpack(const Piece (&r)[NP], float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (kVec) {
        float y[Width<T>::n];
        as_floats(r[i], y);
#pragma unroll
        for (int j = 0; j < W; ++j) x[i * W + j] = y[j];
      } else {
        x[i] = ld1(&r[i]);
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, int D, int t, const float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = col(i, t);
      if (c >= D) continue;
      if constexpr (kVec) {
        float y[Width<T>::n];
#pragma unroll
        for (int j = 0; j < W; ++j) y[j] = x[i * W + j];
        st16(p + c, y);
      } else {
        st1(p + c, x[i]);
      }
    }
  }
  static __device__ __forceinline__ void weights(const void* w, bool wbf16, int D, int t, float (&x)[E], float fill) {
    if (!w) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = fill;
    } else if (wbf16) {
      load(static_cast<const bf16*>(w), D, t, x, fill);
    } else {
      load(static_cast<const float*>(w), D, t, x, fill);
    }
  }
  static __device__ __forceinline__ bool in(int i, int D, int t) { return col(i, t) < D; }  // piece i: all of it or none
};

// Sums over the TPR threads of a row, in every one of them.  TPR > 32: `red` holds NV floats per warp of the row; two
// barriers of the whole block, which every thread takes part in.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&x)[NV], float* red, int t) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1)
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], o);
  if (TPR > 32) {
    __syncthreads();
    if ((t & 31) == 0)
#pragma unroll
      for (int j = 0; j < NV; ++j) red[(t >> 5) * NV + j] = x[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = 0.f;
#pragma unroll
      for (int i = 0; i < (TPR + 31) / 32; ++i) x[j] += red[i * NV + j];
    }
  }
}

template <int TPR>
constexpr int block_threads() {
  return TPR < 128 ? 128 : TPR;
}
// Blocks an SM, by their registers: an element backward takes four values (h, the gradient, dw, db) and its two as
// they lie in memory, two or four bytes each; forward three in all, the next row's among them.
template <typename T, int TPR, int E, bool kVec, bool kBack>
constexpr int blocks_per_sm() {
  const int regs = kBack ? (kVec && sizeof(T) == 2 ? 5 : 6) * E + 48 : 3 * E + 40;
  const int n = 65536 / (block_threads<TPR>() * (regs < 255 ? regs : 255));
  return n < 1 ? 1 : n;
}

// Backward, rows of x and dy that are on their way to shared memory at a time: as many as 40 KB a block take, four at most (0:
// one row, in registers).  A thread copies the 16-byte pieces that it reads itself, so no barrier stands between.  16384
// rows of 2560: 59 us, with the next row in registers 64; forward the same took 49 us in place of 45, so there the next
// row stays in registers.
template <typename T, int TPR, int E, bool kVec>
constexpr int ring_stages() {
  const int n = 40960 / (block_threads<TPR>() * E * (int)sizeof(T) * 2);
  return !kVec ? 0 : n < 4 ? n : 4;
}
__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: zeros, and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void copies_wait() {  // all but the last kN groups have arrived
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}
template <typename R, int kT, typename T>
__device__ __forceinline__ void copy_row(uint4* slot, const T* p, bool live, int D, int t) {
#pragma unroll
  for (int i = 0; i < R::NP; ++i) {
    const bool ok = live && R::in(i, D, t);
    copy16(slot + i * kT, ok ? p + R::col(i, t) : p, ok);
  }
}

// The groups of a block take every n-th row each; a group's next row is on its way while it sums the one before.
template <typename T, int TPR, int E, bool kVec>
__global__ void __launch_bounds__(block_threads<TPR>(), blocks_per_sm<T, TPR, E, kVec, false>())
    k_norm_forward(Args a, const T* __restrict__ x, const void* w, const void* b, T* y, float* mean, float* rstd) {
  using R = Row<T, TPR, E, kVec>;
  constexpr int kGroups = block_threads<TPR>() / TPR;
  __shared__ float red[kGroups][(TPR + 31) / 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const long long step = (long long)gridDim.x * kGroups;
  const float inv = 1.f / (float)a.D;
  typename R::Piece next[R::NP];
  const auto fetch = [&](long long row) { R::fetch(x + (row < a.rows ? row : 0) * a.xs, row < a.rows ? a.D : 0, t, next); };
  long long row = (long long)blockIdx.x * kGroups + grp;
  fetch(row);
  for (long long first = (long long)blockIdx.x * kGroups; first < a.rows; first += step, row += step) {
    const bool live = row < a.rows;
    float v[E];
    R::unpack(next, v);
    fetch(row + step);
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) s[0] += v[e];
    row_sum<TPR, 1>(s, red[grp], t);
    const float m = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < R::NP; ++i)
      if (R::in(i, a.D, t))
#pragma unroll
        for (int e = i * R::W; e < (i + 1) * R::W; ++e) {
          v[e] -= m;
          s[0] = fmaf(v[e], v[e], s[0]);
        }
    row_sum<TPR, 1>(s, red[grp], t);
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    if (!live) continue;
    float wt[E];
    R::weights(w, a.wbf16, a.D, t, wt, 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = v[e] * r * wt[e];
    R::weights(b, a.wbf16, a.D, t, wt, 0.f);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += wt[e];
    R::store(y + (size_t)row * a.D, a.D, t, v);
    if (t == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = r;
    }
  }
}

template <typename T, int TPR, int E, bool kVec>
__global__ void __launch_bounds__(block_threads<TPR>(), blocks_per_sm<T, TPR, E, kVec, true>())
    k_norm_backward(Args a, const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const void* w, T* dx, float* part) {
  using R = Row<T, TPR, E, kVec>;
  constexpr int kGroups = block_threads<TPR>() / TPR;
  __shared__ float red[kGroups][2 * ((TPR + 31) / 32)];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float dw[E], db[E];
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.f;
  const float inv = 1.f / (float)a.D;
  const long long step = (long long)gridDim.x * kGroups;
  constexpr int kS = ring_stages<T, TPR, E, kVec>(), kT = block_threads<TPR>();
  __shared__ uint4 ring[kS ? 2 * kS * R::NP * kT : kGroups > 1 ? TPR * E / 4 : 1];
  typename R::Piece nx[R::NP], ng[R::NP];
  float nm = 0.f, nr = 0.f;
  int slot = 0;
  const auto fetch = [&](long long row) {
    const bool live = row < a.rows;
    const T *px = x + (live ? row : 0) * a.xs, *pg = dy + (live ? row : 0) * (long long)a.D;
    if constexpr (kS > 0) {
      uint4* to = ring + 2 * slot * R::NP * kT + threadIdx.x;
      copy_row<R, kT>(to, px, live, a.D, t);
      copy_row<R, kT>(to + R::NP * kT, pg, live, a.D, t);
      copies_commit();
      slot = slot + 1 == kS ? 0 : slot + 1;
    } else {
      R::fetch(px, live ? a.D : 0, t, nx);
      R::fetch(pg, live ? a.D : 0, t, ng);
    }
  };
  const auto stats = [&](long long row) {
    nm = row < a.rows ? mean[row] : 0.f;
    nr = row < a.rows ? rstd[row] : 0.f;
  };
  long long row = (long long)blockIdx.x * kGroups + grp;
  for (int i = 0; i < (kS ? kS : 1); ++i) fetch(row + i * step);
  stats(row);
  for (long long first = (long long)blockIdx.x * kGroups; first < a.rows; first += step, row += step) {
    float h[E], g[E];
    if constexpr (kS > 0) {
      copies_wait<(kS ? kS - 1 : 0)>();
      const uint4* from = ring + 2 * slot * R::NP * kT + threadIdx.x;
#pragma unroll
      for (int i = 0; i < R::NP; ++i) {
        nx[i] = from[i * kT];
        ng[i] = from[(R::NP + i) * kT];
      }
    }
    R::unpack(nx, h);
    R::unpack(ng, g);
    const float m = nm, r = nr;
    stats(row + step);
    if (kS == 0) fetch(row + step);
    float s[2] = {0.f, 0.f};
    float wt[E];
    R::weights(w, a.wbf16, a.D, t, wt, 1.f);
    // (past the row's end the upstream gradient is zero: nothing is added there, and nothing stored)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h[e] = (h[e] - m) * r;
      db[e] += g[e];
      dw[e] = fmaf(g[e], h[e], dw[e]);
      g[e] *= wt[e];
      s[0] += g[e];
      s[1] = fmaf(g[e], h[e], s[1]);
    }
    row_sum<TPR, 2>(s, red[grp], t);
    if (kS > 0) fetch(row + kS * step);  // (what the slot held has been summed)
    const float s0 = s[0] * inv, s1 = s[1] * inv;
    const float a0 = -r * s0, a1 = -r * s1;
#pragma unroll
    for (int e = 0; e < E; ++e) g[e] = fmaf(r, g[e], fmaf(a1, h[e], a0));
    if (row < a.rows) R::store(dx + (size_t)row * a.D, a.D, t, g);
  }
  if constexpr (kS > 0) copies_wait<0>();
  if (!part) return;
  // this block's sums: its groups in order, over the ring
  float* s_part = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float(&acc)[E] = which ? db : dw;
    if (kGroups > 1) {
      for (int k = 1; k < kGroups; ++k) {
        __syncthreads();
        if (grp == k)
#pragma unroll
          for (int e = 0; e < E; ++e) s_part[e * TPR + t] = acc[e];
        __syncthreads();
        if (grp == 0)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += s_part[e * TPR + t];
      }
    }
    if (grp == 0) {
      float* p = part + ((size_t)which * gridDim.x + blockIdx.x) * a.D;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = R::col(e / R::W, t) + e % R::W;
        if (c < a.D) p[c] = acc[e];
      }
    }
  }
}

template <typename T, int TPR, int E, bool kVec>
void launch(const Call& c, cudaStream_t st) {
  constexpr int kT = block_threads<TPR>(), kGroups = kT / TPR;
  if (!c.backward) {
    constexpr long long kMost = 152 * blocks_per_sm<T, TPR, E, kVec, false>();  // as many as this GPU's 152 SMs hold at once
    const long long want = (c.a.rows + kGroups - 1) / kGroups;
    const unsigned grid = (unsigned)(want < kMost ? want : kMost);
    SSD_LAUNCH("k_norm_forward", st,
               k_norm_forward<T, TPR, E, kVec><<<grid, kT, 0, st>>>(c.a, (const T*)c.x, c.w, c.b, (T*)c.y, c.mean, c.rstd));
    return;
  }
  const int nb = backward_blocks(c.a.rows, c.a.D, sizeof(T) == 4);
  SSD_LAUNCH("k_norm_backward", st,
             k_norm_backward<T, TPR, E, kVec>
             <<<nb, kT, 0, st>>>(c.a, (const T*)c.dy, (const T*)c.x, c.mean, c.rstd, c.w, (T*)c.dx, c.part));
}

// The elements a thread that shape_of gives for TPR threads a row, and no others: 8 and 16 only at the fewest threads (16
// in fp32 at any), 32 in bf16 or at the most threads, 40 in bf16 below those.
template <typename T, int TPR, bool kVec>
void by_elements(const Call& c, int e, cudaStream_t st) {
  if constexpr (TPR == 8)
    if (e == 8) return launch<T, TPR, 8, kVec>(c, st);
  if constexpr (TPR == 8 || sizeof(T) == 4)
    if (e == 16) return launch<T, TPR, 16, kVec>(c, st);
  if constexpr (TPR == 512 || sizeof(T) == 2)
    if (e == 32) return launch<T, TPR, 32, kVec>(c, st);
  if constexpr (sizeof(T) == 2 && TPR < 512)
    if (e == 40) return launch<T, TPR, 40, kVec>(c, st);
  launch<T, TPR, 24, kVec>(c, st);
}
template <typename T, bool kVec>
void by_width(const Call& c, cudaStream_t st) {
  const Shape s = shape_of(c.a.D, sizeof(T) == 4);
  switch (s.tpr) {
    case 8: return by_elements<T, 8, kVec>(c, s.e, st);
    case 16: return by_elements<T, 16, kVec>(c, s.e, st);
    case 32: return by_elements<T, 32, kVec>(c, s.e, st);
    case 64: return by_elements<T, 64, kVec>(c, s.e, st);
    case 128: return by_elements<T, 128, kVec>(c, s.e, st);
    case 256: return by_elements<T, 256, kVec>(c, s.e, st);
    default: return by_elements<T, 512, kVec>(c, s.e, st);
  }
}
template <typename T>
void by_type(const Call& c, cudaStream_t st) {
  constexpr int w = 16 / sizeof(T);
  if (c.a.D % w == 0 && c.a.xs % w == 0 && (reinterpret_cast<uintptr_t>(c.x) & 15u) == 0)
    by_width<T, true>(c, st);
  else
    by_width<T, false>(c, st);
}

}  // namespace
}  // namespace norm
}  // namespace ssd
