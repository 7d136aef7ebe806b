// The gated linear recurrence over whole sequences, forward (formulas and the split: glr_common.cuh).
#include <type_traits>

#include "glr_common.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kStages = 2;  // tiles in shared memory or on their way there
// Steps a thread has of a tile, and blocks an SM.  Long runs share the joining of their maps and the cluster's barriers: one
// sequence of 16384 steps of 2560 channels takes 91 us in runs of 16 (two blocks an SM), 106 us in runs of 8 (three); packed,
// 24 sequences of 20011 steps take 149 us and 182 us.  fp32 words are twice as wide.
template <typename T>
constexpr int run_of() {
  return sizeof(T) == 4 ? 4 : 16;
}
template <typename T>
constexpr int blocks_of() {
  return sizeof(T) == 4 ? 3 : 2;
}

// 1 / sqrt(m2 e1^2): with e1 = 1 + e^-i, m2 times it is m s(i), by one root in place of a root and a reciprocal (16384 steps
// of 2560 channels: 90 us, 93 with both).  0 where m2 is, and where e1^2 is infinite (a gate below 2^-64).
__device__ __forceinline__ P inv_root(P m2, P e1) {
  return each(each(m2, [](float v) { return fmaxf(v, 1e-37f); }) * (e1 * e1), [](float v) { return rsqrt_f(v); });
}

// y, the final states and the marks (the states that enter the backward's runs).  Grid: (64-channel slabs x a.share,
// sequences; one for a packed batch).  Tile j share + k of a sequence is block k's of its cluster.  One warp joins the
// runs' maps of each tile to one that goes to all blocks of the cluster; one barrier of the cluster later each of them has
// the state that enters its tile.
template <typename T, bool kVec, bool kPacked, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == kFewWarps ? blocks_of<T>() : 1)
    k_glr_forward(Args a, const T* __restrict__ x, const T* __restrict__ r, const T* __restrict__ i,
                  const float* __restrict__ lam, const float* __restrict__ h0, const int* __restrict__ cu, T* y,
                  float* h_final, float* marks) {
  constexpr int kRun = run_of<T>(), L = kRun * kWarps;
  constexpr int kMark = mark_of(sizeof(T) == 4);
  static_assert(kRun % kMark == 0, "runs begin where states are kept");
  using Tile = Tiles<T, kVec, kWarps, kRun, 3>;
  using Word = typename Words<T>::Word;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ Map maps[2][kWarps][32];
  __shared__ Map xchg[2][kMostShare][32];
  __shared__ int code[2][kPacked ? L : 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int share = a.share, rank = blockIdx.x % share;
  const int c0 = (int)(blockIdx.x / share) * kWidth, c = c0 + lane * 2, axis = blockIdx.y;
  const size_t row0 = (size_t)axis * a.T;
  const T* const from[3] = {x + row0 * a.xs, r + row0 * a.rs, i + row0 * a.is};
  const uint32_t step[3] = {(uint32_t)a.xs, (uint32_t)a.rs, (uint32_t)a.is};
  Tile tiles(from, step, c0, a.D, a.T, rank * L, share);
  const int nt = (a.T + L - 1) / L, rounds = (nt + share - 1) / share, nm = (a.T + kMark - 1) / kMark;
  const auto bring = [&](int stage) {
    tiles.bring(ring + stage * Tile::kBytes);
    copies_commit();
  };
  int near = 0;
  const auto codes = [&](int j) {
    if (!kPacked || threadIdx.x >= L) return;
    const int found = code_of(cu, a, (j * share + rank) * L + threadIdx.x, near);
    code[j & 1][threadIdx.x] = found;
    if (h0 && found >= 0 && (found & kFirst)) prefetch_state(h0, found, c0, a.D);
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) bring(s);
  codes(0);
  const P rate = load_rate(lam, c, a.D, a.scale);
  const bool far = any_far(rate), second = c + 1 < a.D;
  P carry = !kPacked && h0 ? load_two(h0 + (size_t)axis * a.D, c, a.D) : both(0.f);  // the state that enters the round
  if (kPacked && h_final && rank == 0) empty_sequences(cu, a, c0, h0, h_final);
  copies_wait<kStages - 1>();
  __syncthreads();
  if (share > 1) {  // (the other blocks of the cluster have begun before anything is written to them)
    cluster_arrive_relaxed();
    cluster_wait();
  }
  int t0 = rank * L + w * kRun;
  T* ty = y + (row0 + rank * L) * a.D;  // the tile's first step
  const uint32_t oy = (uint32_t)(w * kRun) * a.D + c;
  Ring<kStages> sg;
  for (int j = 0; j < rounds; ++j, t0 += share * L, ty += (long long)(share * L) * a.D, sg.next()) {
    const Word* stage = reinterpret_cast<const Word*>(ring + sg.at * Tile::kBytes) + w * kRun * 32 + lane;
    P av[kRun], bv[kRun];
    const auto maps_of_steps = [&](auto is_far) {
#pragma unroll
      for (int s = 0; s < kRun; ++s) {
        const P o = one_minus_exp<decltype(is_far)::value>(rate * sigmoid(Words<T>::open(stage[(L + s) * 32])));
        av[s] = one_less(o);
        const P m2 = o * one_more(av[s]), e1 = one_more(exp_neg(Words<T>::open(stage[(2 * L + s) * 32])));
        bv[s] = m2 * inv_root(m2, e1) * Words<T>::open(stage[s * 32]);
      }
    };
    if (far)
      maps_of_steps(std::true_type());
    else
      maps_of_steps(std::false_type());
    const Bits bits = bits_of<kPacked, kRun>(&code[j & 1][kPacked ? w * kRun : 0], t0, a.T, lane);
    if (bits.first | bits.none) {
      // (one step at a time in one copy of the code; the steps' registers are chosen by comparisons)
      if (kPacked && h0)
        for (uint32_t left = bits.first & ~bits.none; left; left &= left - 1) {
          const int at = __ffs(left) - 1;
          const P from = load_two(h0 + (size_t)bits.seq(at) * a.D, c, a.D);
#pragma unroll
          for (int s = 0; s < kRun; ++s)
            if (s == at) bv[s] = fma(av[s], from, bv[s]);
        }
#pragma unroll
      for (int s = 0; s < kRun; ++s) {
        if (bits.none >> s & 1) av[s] = both(1.f), bv[s] = both(0.f);
      }
    }
    // (a packed batch's first steps are told by their bits, in the one copy of the code: a second one for runs that have any
    // would be fetched anew each time)
    const auto starts = [&](int s) { return kPacked && (bits.first >> s & 1); };
    Map m = {av[0], bv[0]};
#pragma unroll
    for (int s = 1; s < kRun; ++s) {
      m.a = m.a * av[s];
      const P n = fma(av[s], m.b, bv[s]);
      m.b = starts(s) ? bv[s] : n;
    }
    if (kPacked && bits.first) m.a = anew();
    maps[j & 1][w][lane] = m;
    codes(j + 1);
    // the runs' maps are there, the next tile has come, and this one's stage is free
    copies_wait<kStages - 2>();
    const bool resets = kPacked && __syncthreads_or(bits.first != 0);
    if (!kPacked) __syncthreads();
    if (share > 1) {
      if (w == kWarps - 1) {
        m = maps[j & 1][0][lane];
        if (kPacked && resets) {
#pragma unroll 1
          for (int v = 1; v < kWarps; ++v) m = after<true>(m, maps[j & 1][v][lane]);
        } else {
#pragma unroll
          for (int v = 1; v < kWarps; ++v) m = after<false>(m, maps[j & 1][v][lane]);
        }
        for (int k = 0; k < share; ++k) store_to(&xchg[j & 1][rank][lane], k, m);
        cluster_arrive();
      } else {
        cluster_arrive_relaxed();
      }
    }
    bring(sg.at);
    P h = carry;
    if (share > 1) {
      cluster_wait();
#pragma unroll
      for (int v = 0; v < kMostShare; ++v) {
        if (v == share) break;
        if (v == rank) h = carry;
        carry = through<kPacked>(xchg[j & 1][v][lane], carry);
      }
    }
    const auto join = [&](auto anew_too) {
      constexpr bool kAnew = decltype(anew_too)::value;
#pragma unroll
      for (int v = 0; v < kWarps - 1; ++v)
        if (v < w) h = through<kAnew>(maps[j & 1][v][lane], h);
      if (share == 1) {
        carry = h;
#pragma unroll
        for (int v = 0; v < kWarps; ++v)
          if (v >= w) carry = through<kAnew>(maps[j & 1][v][lane], carry);
      }
    };
    if (kPacked && resets)
      join(std::true_type());
    else
      join(std::false_type());
    if (t0 >= a.T) continue;
    float* kept = marks ? marks + ((size_t)axis * nm + t0 / kMark) * a.D : nullptr;
    if (h_final)
      for (uint32_t left = bits.last; left; left &= left - 1) {  // the state after each last step, walked to once more
        const int at = __ffs(left) - 1, n = kPacked ? bits.seq(at) : axis;
        P g = h;
#pragma unroll
        for (int s = 0; s < kRun; ++s)
          if (s <= at) g = starts(s) ? bv[s] : fma(av[s], g, bv[s]);
        store_two(h_final + (size_t)n * a.D, c, a.D, g);
      }
    const auto outputs = [&](auto is_short) {
#pragma unroll
      for (int s = 0; s < kRun; ++s) {
        const bool there = !decltype(is_short)::value || t0 + s < a.T;
        if (kept && s % kMark == 0 && there) store_row<float, kVec>(kept + (size_t)(s / kMark) * a.D + c, second, h);
        const P n = fma(av[s], h, bv[s]);
        h = starts(s) ? bv[s] : n;
        if (y && there) store_row<T, kVec>(ty + (oy + s * (uint32_t)a.D), second, h);
      }
    };
    if (c < a.D) {
      if (t0 + kRun > a.T)
        outputs(std::true_type());
      else
        outputs(std::false_type());
    }
  }
  copies_wait<0>();
}

template <typename T, bool kVec, bool kPacked, int kWarps>
struct Shape {
  static constexpr auto kernel = &k_glr_forward<T, kVec, kPacked, kWarps>;
  static constexpr int warps = kWarps, run = run_of<T>(), smem = kStages * Tiles<T, kVec, kWarps, run, 3>::kBytes;
};
template <typename T, bool kVec, bool kPacked>
cudaError_t run(Call& c, cudaStream_t st) {
  return launch_cluster<Shape<T, kVec, kPacked, kFewWarps>, Shape<T, kVec, kPacked, kManyWarps>>(
      "k_glr_forward", c.a, st, (const T*)c.x, (const T*)c.r, (const T*)c.i, c.lam, c.h0, c.cu, (T*)c.y, c.h_final, c.marks);
}
template <typename T>
cudaError_t by_type(Call c, cudaStream_t st) {
  c.a = flattened(c.a);
  if (whole(c, false)) return c.a.packed ? run<T, true, true>(c, st) : run<T, true, false>(c, st);
  return c.a.packed ? run<T, false, true>(c, st) : run<T, false, false>(c, st);
}

}  // namespace

cudaError_t forward(const Call& c, cudaStream_t st) { return c.a.f32 ? by_type<float>(c, st) : by_type<bf16>(c, st); }

}  // namespace glr
}  // namespace ssd
