// The gradients of the gated linear recurrence (the split: glr_common.cuh).  With dh_t = dy_t + D_{t+1}, D_t = a_t dh_t:
//     dx = dh m s(i),   di = dh m u (1 - s(i)),   q = dL/dn n = dh (a n) (a u / m - h_{t-1}),   dr = q (1 - s(r)),
//     dlam = s(lam) / softplus(lam) sum of q,   dh0 = D_0
// n / m goes to 0 with n, so a gate that is shut has finite gradients.
#include <type_traits>

#include "glr_common.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kStages = 2;  // tiles in shared memory or on their way there

// Tile by tile from the end.  The stash holds the state that enters each thread's run, so a run's states and all factors of
// its gradients come without a word from other warps; only the upstream gradients' maps D -> a D + a dy are joined as the
// states are forward, in the other direction.  The factors of a run's first steps wait for that in shared memory (eight
// numbers a step and lane, written and read by the same thread), those of its last four in registers: runs of eight steps
// halve the barriers that runs of four would take.  part [axes share, D]: the sums of q.
template <typename T, bool kVec, bool kPacked, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == kFewWarps ? 2 : 1)
    k_glr_backward(Args a, const T* __restrict__ dy, const float* __restrict__ dh_final, const T* __restrict__ x,
                   const T* __restrict__ r, const T* __restrict__ i, const float* __restrict__ lam,
                   const float* __restrict__ h0, const int* __restrict__ cu, const float* __restrict__ marks, T* dx, T* dr,
                   T* di, float* dh0, float* part) {
  constexpr int kThreads = 32 * kWarps, kRun = mark_of(sizeof(T) == 4), L = kRun * kWarps, kAside = kRun - 4;
  using Tile = Tiles<T, kVec, kWarps, kRun, 4>;
  using Word = typename Words<T>::Word;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ Map rev[2][kWarps][32];
  __shared__ Map xchg[2][kMostShare][32];
  __shared__ int code[2][kPacked ? L : 1];
  Map* aside = reinterpret_cast<Map*>(ring + kStages * Tile::kBytes) + threadIdx.x;  // [kAside][2][kThreads]
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int share = a.share, rank = blockIdx.x % share;
  const int c0 = (int)(blockIdx.x / share) * kWidth, c = c0 + lane * 2, axis = blockIdx.y;
  const size_t row0 = (size_t)axis * a.T;
  const T* const from[4] = {x + row0 * a.xs, r + row0 * a.rs, i + row0 * a.is, dy + row0 * a.D};
  const uint32_t step[4] = {(uint32_t)a.xs, (uint32_t)a.rs, (uint32_t)a.is, (uint32_t)a.D};
  const int nt = (a.T + L - 1) / L, rounds = (nt + share - 1) / share, nm = (a.T + kRun - 1) / kRun;
  Tile tiles(from, step, c0, a.D, a.T, (nt - 1 - rank) * L, -share);
  const auto bring = [&](int stage) {
    tiles.bring(ring + stage * Tile::kBytes);
    copies_commit();
  };
  int near = 0;
  // (below 0: there is no such tile)
  const auto codes = [&](int j) {
    if (!kPacked || threadIdx.x >= L) return;
    const int found = code_of(cu, a, (nt - 1 - (j * share + rank)) * L + (int)threadIdx.x, near);
    code[j & 1][threadIdx.x] = found;
    if (h0 && found >= 0 && (found & kFirst)) prefetch_state(h0, found, c0, a.D);
    if (dh_final && found >= 0 && (found & kLast)) prefetch_state(dh_final, found, c0, a.D);
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) bring(s);
  codes(0);
  const P rate = load_rate(lam, c, a.D, a.scale);
  const bool far = any_far(rate), second = c + 1 < a.D;
  P back = !kPacked && dh_final ? load_two(dh_final + (size_t)axis * a.D, c, a.D) : both(0.f);  // D behind the round
  P qsum = both(0.f);
  if (kPacked && dh0 && rank == 0) empty_sequences(cu, a, c0, dh_final, dh0);
  // The state that enters this thread's run of the j-th tile, on its way one tile ahead.
  const auto mark = [&](int j) {
    const int t = (nt - 1 - (j * share + rank)) * L + w * kRun;
    return j < rounds && t >= 0 && t < a.T ? load_two(marks + ((size_t)axis * nm + t / kRun) * a.D, c, a.D) : both(0.f);
  };
  P next = mark(0);
  copies_wait<kStages - 1>();
  __syncthreads();
  if (share > 1) {  // (the other blocks of the cluster have begun before anything is written to them)
    cluster_arrive_relaxed();
    cluster_wait();
  }
  const uint32_t o0 = (uint32_t)(w * kRun) * a.D + c;  // from a tile's first step
  Ring<kStages> sg;
  for (int j = 0; j < rounds; ++j, sg.next()) {
    const int tile = nt - 1 - (j * share + rank), t0 = tile < 0 ? a.T : tile * L + w * kRun;
    const Word* stage = reinterpret_cast<const Word*>(ring + sg.at * Tile::kBytes) + w * kRun * 32 + lane;
    const Bits bits = bits_of<kPacked, kRun>(&code[j & 1][kPacked ? w * kRun : 0], t0, a.T, lane);
    const bool odd = (bits.first | bits.none | (kPacked ? bits.last : 0)) != 0;
    // per step: a, dy; of the last four: dx / dh, di / dh, q / dh, 1 - s(r)
    P av[kRun], up[kRun], mi[4], ki[4], kq[4], r1[4];
    P h = next;
    const auto factors = [&](auto is_far, auto is_odd) {
#pragma unroll
      for (int s = 0; s < kRun; ++s) {
        const auto most = [](float v) { return min_nan(v, 1e30f); };
        const P xv = Words<T>::open(stage[s * 32]);
        const P er = each(exp_neg(Words<T>::open(stage[(L + s) * 32])), most), sr = inv_one_more(er);
        const P ei = each(exp_neg(Words<T>::open(stage[(2 * L + s) * 32])), most), si = inv_one_more(ei);
        up[s] = Words<T>::open(stage[(3 * L + s) * 32]);
        const P n = rate * sr, o = one_minus_exp<decltype(is_far)::value>(n);
        av[s] = one_less(o);
        const P m2 = o * one_more(av[s]);
        const P rm = each(m2, [](float v) { return rsqrt_f(fmaxf(v, 1e-37f)); });  // (m2 = 0: n is 0 too)
        const P sm = si * rm, fx = m2 * sm, b = fx * xv, fi = b * (ei * si), fr = er * sr;
        if (decltype(is_odd)::value) {
          if (bits.none >> s & 1) {
            av[s] = both(1.f), up[s] = both(0.f);
          } else if (kPacked) {
            const size_t at = (size_t)bits.seq(s) * a.D;
            if ((bits.first >> s & 1)) h = h0 ? load_two(h0 + at, c, a.D) : both(0.f);
            if ((bits.last >> s & 1) && dh_final) up[s] = up[s] + load_two(dh_final + at, c, a.D);
          }
        }
        const P fq = av[s] * n * less(av[s] * (sm * xv), h);
        h = fma(av[s], h, b);
        if (s < kAside) {
          aside[(2 * s) * kThreads] = Map{fx, fi};
          aside[(2 * s + 1) * kThreads] = Map{fq, fr};
        } else {
          mi[s - kAside] = fx, ki[s - kAside] = fi, kq[s - kAside] = fq, r1[s - kAside] = fr;
        }
      }
    };
    if (far || odd)  // (one copy of the rare forms)
      factors(std::true_type(), std::true_type());
    else
      factors(std::false_type(), std::false_type());
    Map b = {both(1.f), both(0.f)};
    if (kPacked && bits.first) {
#pragma unroll
      for (int s = kRun - 1; s >= 0; --s)  // (what a first step hands on goes to dh0, not to the step before it)
        b = bits.first >> s & 1 ? Map{anew(), both(0.f)} : after<true>(b, Map{av[s], av[s] * up[s]});
    } else {
      b = Map{av[kRun - 1], av[kRun - 1] * up[kRun - 1]};
#pragma unroll
      for (int s = kRun - 2; s >= 0; --s) b = Map{av[s] * b.a, av[s] * (up[s] + b.b)};
    }
    rev[j & 1][w][lane] = b;
    codes(j + 1);
    // the runs' maps are there, the next tile has come, and this one's stage is free
    copies_wait<kStages - 2>();
    const bool resets = kPacked && __syncthreads_or(bits.first != 0);
    if (!kPacked) __syncthreads();
    if (share > 1) {
      if (w == kWarps - 1) {
        b = rev[j & 1][kWarps - 1][lane];
        if (kPacked && resets) {
#pragma unroll 1
          for (int v = kWarps - 2; v >= 0; --v) b = after<true>(b, rev[j & 1][v][lane]);
        } else {
#pragma unroll
          for (int v = kWarps - 2; v >= 0; --v) b = after<false>(b, rev[j & 1][v][lane]);
        }
        for (int k = 0; k < share; ++k) store_to(&xchg[j & 1][rank][lane], k, b);
        cluster_arrive();
      } else {
        cluster_arrive_relaxed();
      }
    }
    bring(sg.at);
    next = mark(j + 1);
    P d = back;  // D of the step behind this thread's
    if (share > 1) {
      cluster_wait();
#pragma unroll
      for (int v = 0; v < kMostShare; ++v) {
        if (v == share) break;
        if (v == rank) d = back;
        back = through<kPacked>(xchg[j & 1][v][lane], back);
      }
    }
    const auto join_back = [&](auto anew_too) {
      constexpr bool kAnew = decltype(anew_too)::value;
#pragma unroll
      for (int v = kWarps - 1; v > 0; --v)
        if (v > w) d = through<kAnew>(rev[j & 1][v][lane], d);
      if (share == 1) {
        back = d;
#pragma unroll
        for (int v = kWarps - 1; v >= 0; --v)
          if (v <= w) back = through<kAnew>(rev[j & 1][v][lane], back);
      }
    };
    if (kPacked && resets)
      join_back(std::true_type());
    else
      join_back(std::false_type());
    if (t0 >= a.T) continue;
    const size_t at = (row0 + (size_t)tile * L) * a.D;
    T *px = dx + at, *pr = dr + at, *pi = di + at;
    const bool plain = !(bits.first | bits.none) && (kPacked || t0 > 0), live = c < a.D;
#pragma unroll
    for (int s = kRun - 1; s >= 0; --s) {
      Map f, g;
      if (s < kAside) {
        f = aside[(2 * s) * kThreads];
        g = aside[(2 * s + 1) * kThreads];
      } else {
        f = Map{mi[s - kAside], ki[s - kAside]};
        g = Map{kq[s - kAside], r1[s - kAside]};
      }
      const P dh = up[s] + d;
      d = av[s] * dh;
      P q = dh * g.a, vx = dh * f.a, vi = dh * f.b, vr = q * g.b;
      if (!plain) {
        if (bits.none >> s & 1) q = vx = vi = vr = both(0.f);
        if (dh0 && (kPacked ? (bits.first & ~bits.none) >> s & 1 : t0 + s == 0))
          store_two(dh0 + (size_t)(kPacked ? bits.seq(s) : axis) * a.D, c, a.D, d);
        if (kPacked && (bits.first >> s & 1)) d = both(0.f);
      }
      qsum = qsum + q;
      if (live && (plain || t0 + s < a.T)) {
        const uint32_t o = o0 + s * (uint32_t)a.D;
        store_row<T, kVec>(px + o, second, vx);
        store_row<T, kVec>(pr + o, second, vr);
        store_row<T, kVec>(pi + o, second, vi);
      }
    }
  }
  copies_wait<0>();
  // the warps' sums of q, in order
  __syncthreads();
  rev[0][w][lane].a = qsum;
  __syncthreads();
  if (w == 0) {
    P s = rev[0][0][lane].a;
#pragma unroll
    for (int v = 1; v < kWarps; ++v) s = s + rev[0][v][lane].a;
    store_two(part + ((size_t)axis * share + rank) * a.D, c, a.D, s);
  }
}

template <typename T, bool kVec, bool kPacked, int kWarps>
struct Shape {
  static constexpr auto kernel = &k_glr_backward<T, kVec, kPacked, kWarps>;
  static constexpr int warps = kWarps, run = mark_of(sizeof(T) == 4);
  static constexpr int aside = (run - 4) * 2 * 32 * kWarps * (int)sizeof(Map);
  static constexpr int smem = kStages * Tiles<T, kVec, kWarps, run, 4>::kBytes + aside;
};
template <typename T, bool kVec, bool kPacked>
cudaError_t run(Call& c, cudaStream_t st) {
  return launch_cluster<Shape<T, kVec, kPacked, kFewWarps>, Shape<T, kVec, kPacked, kManyWarps>>(
      "k_glr_backward", c.a, st, (const T*)c.dy, c.dh_final, (const T*)c.x, (const T*)c.r, (const T*)c.i, c.lam, c.h0, c.cu,
      (const float*)c.marks, (T*)c.dx, (T*)c.dr, (T*)c.di, c.dh0, c.part);
}
template <typename T>
cudaError_t by_type(Call& c, cudaStream_t st) {
  if (whole(c, true)) return c.a.packed ? run<T, true, true>(c, st) : run<T, true, false>(c, st);
  return c.a.packed ? run<T, false, true>(c, st) : run<T, false, false>(c, st);
}

}  // namespace

cudaError_t backward(const Call& call, cudaStream_t st, int* rows) {
  Call c = call;
  c.a = flattened(c.a);
  const cudaError_t e = c.a.f32 ? by_type<float>(c, st) : by_type<bf16>(c, st);
  *rows = axes(c.a) * c.a.share;
  return e;
}

}  // namespace glr
}  // namespace ssd
