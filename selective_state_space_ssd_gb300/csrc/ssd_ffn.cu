// The gated feed-forward: h = act(G) U with G = x Wg^T and U = x Wu^T, and its gradients
//     dU = dh act(G),  dG = dh U act'(G),  dx = dG Wg + dU Wu,  dWg = dG^T x,  dWu = dU^T x
// in three kernels: forward (both projections, the activation and the product), the elementwise dG and dU, and dx with both
// weights' gradients.  The products run on the tensor cores: bf16 operands by TMA into 128-byte swizzled tiles, fp32
// accumulators in tensor memory.
//
// One kernel for all of them, k_ffn_product: pairs of blocks, one block an SM, that walk over pairs of output tiles of 128 x
// 256; a warp issues the copies, one the products, four turn an accumulator into results while the next tile is under way (two
// accumulators of 256 columns, four warps each: with four for both, tiles of four steps waited for them).  In the forward's
// tile the 256 columns are 128 of G and the same 128 of U, so that a thread meets both.
// A pair's product is one of 256 rows: each block brings its own rows and half of the columns' operand, which the tensor cores
// of both read, so that a third less comes out of L2 than with whole operands in every block and six stages fit in place of
// four.  Per launch, us, pairs and single blocks: 8192 rows of 2560 and 7680 forward 371 and 401, gradients 688 and 725; 1501
// of 776 and 2056 25 and 27, 35 and 41; 4000 of 1536 and 4608 83 and 92, 131 and 141; 125 of 288 and 8816, with few steps a
// tile, gradients 25 and 24.  (One copy of the operand that goes to both blocks would do the same; it is not for memory of
// other GPUs, and these calls take any.)  Tiles of 128 x 128 where they end sooner (sooner()).
//
// dx sums over 2 F numbers; with few rows its sums are taken in pieces, fp32, that another launch joins (grads_plan()).
//
// The training forward keeps G and U for the backward.  dG and dU are rounded to bf16, as operands of the tensor cores have
// to be: the one rounding of the backward before its results'.
#include <initializer_list>
#include <type_traits>

#include "ssd.h"
#include "ssd_device.cuh"
#include "ssd_internal.h"
#include "pair.cuh"
#include "tc_common.cuh"
#include "vec_io.cuh"

namespace ssd {
namespace ffn {
namespace {

using namespace tc;

constexpr int BM = 128, BK = 64;
constexpr int kThreads = 384, kSMs = 152;  // a warp for copies, one for products, four for the results of every other tile
constexpr int kBytesA = BM * BK * 2;
constexpr int kBytesPiece = BM * 64 * 2, kBytesOut = 2 * kBytesPiece;  // 64 columns on their way out, of two tiles
constexpr int kMostSmem = 232448;

// Stages of a result's tile of BN columns: as many as shared memory holds.
template <int BN>
struct Stages {
  static constexpr int kBytesB = BN / 2 * BK * 2, kBytes = kBytesA + kBytesB;  // of a block
  static constexpr int kN = BN == 256 ? 6 : 8;
  static constexpr int kSmem = kN * kBytes + kBytesOut + 1024 + 256;
  static_assert(kSmem <= kMostSmem, "");
};

enum Kind { kForward, kGrads };
// Pairs of row tiles that are walked over together, column by column, so that their operands stay in L2.  8192 rows of 2560
// and 7680, us: forward 393 with 4, 375 with 8, 368 with 16, 384 with 32; gradients 687 with 1, 683 with 2, 692 with 4 and
// with 8, 699 with 16.
constexpr int group_of(Kind kind) { return kind == kForward ? 16 : 2; }

struct Args {
  int M, D, F;
  bool gelu;
  long long xs;
};

// Operands a (rows of the result), b (its columns), results o; of the forward's product (or dx) and of the weights'
// gradients, two of each where there are two matrices.
struct Maps {
  CUtensorMap a[2], b[2], o, wa[2], wb, wo[2];
};
struct Plan {
  int m_tiles, n_tiles, steps, half;      // tiles and steps of BK; dx: half of the steps are of the first pair of matrices
  int w_m_tiles, w_n_tiles, w_steps, w_half;  // the weights' gradients; half of the row tiles are of the first matrix
  int both;                                   // of those, pairs of tiles that every pair of blocks has
  int pieces;                                 // of each sum of dx, taken as tiles of their own and joined by k_ffn_join
};
// Two blocks, a cluster, work on two row tiles of the same columns.  The n-th of such pairs of tiles of a pair of blocks: the
// forward's go round.  dx's (piece by piece) do too, and the first of them leave some with one more; the weights' gradients'
// follow, `both` for every pair of blocks and the others for those with fewer of dx's, as many as end the two kinds about
// together (balance()).
struct Item {
  bool weights;
  int t, from, to, piece;  // pair of tiles, steps of its sum
};
__host__ __device__ __forceinline__ int pairs_of(int m_tiles, int n_tiles) { return (m_tiles + 1) / 2 * n_tiles; }
template <Kind kKind>
__device__ __forceinline__ bool item_of(const Plan& p, int n, Item& it) {
  const int blocks = gridDim.x / 2, i = blockIdx.x / 2, whole = pairs_of(p.m_tiles, p.n_tiles), tiles = whole * p.pieces;
  it = Item{false, n * blocks + i, 0, p.steps, 0};
  if (it.t < tiles) {
    if (kKind == kGrads && p.pieces > 1) {
      it.piece = it.t / whole;
      it.t -= it.piece * whole;
      it.from = (int)((long long)p.steps * it.piece / p.pieces);
      it.to = (int)((long long)p.steps * (it.piece + 1) / p.pieces);
    }
    return true;
  }
  if (kKind == kForward) return false;
  it.to = p.w_steps;
  const int more = tiles % blocks, k = n - (tiles / blocks + (i < more));  // those that have one more of dx's: 0 .. more - 1
  it.weights = true;
  it.t = k < p.both ? k * blocks + i : p.both * blocks + (k - p.both) * (blocks - more) + i - more;
  return (k < p.both || i >= more) && it.t < pairs_of(p.w_m_tiles, p.w_n_tiles);
}

// The activation and its slope at g, right for every finite g and NaN of a NaN: q = s(z) is 0 or 1 where e^-z is beyond fp32,
// and 1 - q is taken of q, so that no infinity meets a zero.
__device__ __forceinline__ void act_and_slope(float g, bool gelu, float& a, float& s) {
  if (gelu) {
    // tanh form: g s(z) with z = 2 sqrt(2 / pi) (g + 0.044715 g^3).  From |g| = 16 on, where |z| is 317, q no longer changes
    // and the term of 1 - q is 0, so powers of g stay below.
    const float c = 1.5957691216057308f, v = max_nan(min_nan(g, 16.f), -16.f), v2 = v * v;
    const float q = __fdividef(1.f, 1.f + __expf(-c * fmaf(0.044715f * v2, v, v)));
    a = g * q;
    s = fmaf(v * q * (1.f - q), c * fmaf(3.f * 0.044715f, v2, 1.f), q);
  } else {
    const float q = __fdividef(1.f, 1.f + __expf(-g));
    a = g * q;
    s = q * fmaf(g, 1.f - q, 1.f);
  }
}

// The stash: G and U with 24 bits of each number, rounded to nearest (2^-16 of a value at most, where bf16 would leave 2^-8
// in every factor of dG and dU), as the upper 16 and the next 8 bits in planes of their own.  A piece is eight columns of a
// row; pieces of 128 rows follow one another, as the forward's threads write them.
struct Kept {
  uint4* hi;
  uint2* lo;
};
__host__ __device__ __forceinline__ size_t kept_pieces(const Args& a) { return (size_t)((a.M + BM - 1) / BM) * BM * (a.F / 8); }
__device__ __forceinline__ Kept kept(uint8_t* stash, const Args& a, int row, int f, int which) {
  const size_t n = kept_pieces(a), at = ((size_t)(row / BM) * (a.F / 8) + f / 8) * BM + row % BM;
  return Kept{reinterpret_cast<uint4*>(stash) + which * n + at, reinterpret_cast<uint2*>(stash + 2 * n * 16) + which * n + at};
}
// (numbers that would become infinite are cut off, as are infinities and NaN, whose upper bits stay as they are)
__device__ __forceinline__ uint32_t nearest24(uint32_t v) { return (v & 0x7fffffffu) < 0x7f7fff80u ? v + 0x80u : v; }
__device__ __forceinline__ void keep_one(const Kept& k, const uint32_t* full) {
  uint32_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = nearest24(full[e]);
  const auto hi = [](uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x7632); };
  const auto lo = [](const uint32_t* x) {
    return __byte_perm(__byte_perm(x[0], x[1], 0x0051), __byte_perm(x[2], x[3], 0x0051), 0x5410);
  };
  *k.hi = make_uint4(hi(v[0], v[1]), hi(v[2], v[3]), hi(v[4], v[5]), hi(v[6], v[7]));
  *k.lo = make_uint2(lo(v), lo(v + 4));
}
__device__ __forceinline__ void keep(uint8_t* stash, const Args& a, int row, int f, const uint32_t* g, const uint32_t* u) {
  keep_one(kept(stash, a, row, f, 0), g);
  keep_one(kept(stash, a, row, f, 1), u);
}
__device__ __forceinline__ void kept_values(const Kept& k, float (&v)[8]) {
  const uint4 h = *k.hi;
  const uint2 l = *k.lo;
  const uint32_t hi[4] = {h.x, h.y, h.z, h.w}, lo[2] = {l.x, l.y};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t low = lo[e / 4] >> (8 * (e % 4)) & 0xffu;
    v[e] = __uint_as_float((e % 2 ? hi[e / 2] & 0xffff0000u : hi[e / 2] << 16) | low << 8);
  }
}

// This block's row tile (m_tiles: there is none) and column tile of an item.
template <Kind kKind>
__device__ __forceinline__ void tile_of(const Plan& p, const Item& it, int& m, int& n) {
  constexpr int kGroup = group_of(kKind);
  const int m_pairs = ((it.weights ? p.w_m_tiles : p.m_tiles) + 1) / 2, n_tiles = it.weights ? p.w_n_tiles : p.n_tiles;
  const int per = kGroup * n_tiles, g = it.t / per, m0 = g * kGroup, gm = min(kGroup, m_pairs - m0), r = it.t - g * per;
  m = 2 * (m0 + r % gm) + (blockIdx.x & 1);
  n = r / gm;
}

// ------------------------------------------------------------ two blocks on one product
// A product of 256 rows: each block has 128 of them, in its own shared memory and as its own lanes of tensor memory, and half
// of the columns' operand, which the tensor cores of both read from where it lies.  The first block of the pair issues it.
__device__ __forceinline__ uint32_t in_first_block(const void* p) {  // the same place in the first block's shared memory
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(p)));
  return at;
}
// Into this block's shared memory; the bytes are counted by the first block's barrier.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t first_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(first_bar)
      : "memory");
}
__device__ __forceinline__ void pair_mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrives at both blocks' barriers once the products so far have ended.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}
__device__ __forceinline__ void arrive_in_first_block(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// (all of it: the accumulators then lie at the same place in both)
constexpr int kTmemAll = 512;
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

// Registers of a tcgen05.ld after its wait: nothing that reads them may be moved in front of this.
__device__ __forceinline__ void settled(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

template <Kind kKind, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_ffn_product(const __grid_constant__ Maps maps, Plan plan, Args args, uint8_t* stash, float4* part, int* status) {
  constexpr int kStages = Stages<BN>::kN, kBytesStage = Stages<BN>::kBytes;
  constexpr int kOwn = BN / 2;  // the forward: columns of G, and of U
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  uint8_t* out = smem + kStages * kBytesStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out + kBytesOut);
  uint64_t *full = bars, *empty = bars + kStages, *tfull = bars + 2 * kStages, *tempty = tfull + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int s = 0; s < 2; ++s) mbar_init(tfull + s, 1), mbar_init(tempty + s, 8);
    mbar_init_fence();
    if (kKind == kForward && blockIdx.x == 0) *status = 0;
  }
  if (warp == 2) pair_tmem_alloc(slot, kTmemAll);
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // (both blocks' barriers are there before anything arrives at them)
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int rank = blockIdx.x & 1;

  if (warp == 0) {  // copies: the block's own rows, and its half of the columns (the forward's: G's or U's)
    const auto load = [&](int s, bool weights, int m, int n, int k) {
      uint8_t *a = smem + s * kBytesStage, *b = a + kBytesA;
      const uint32_t bar = in_first_block(full + s);
      if (rank == 0) mbar_expect_tx(full + s, 2 * kBytesStage);
      if (kKind == kForward) {
        pair_load_2d(a, &maps.a[0], k * BK, m * BM, bar);
        pair_load_2d(b, &maps.b[rank], k * BK, n * kOwn, bar);
      } else if (!weights) {
        const int which = k >= plan.half, kk = (k - (which ? plan.half : 0)) * BK;
        pair_load_2d(a, &maps.a[which], kk, m * BM, bar);
#pragma unroll
        for (int j = 0; j < BN / 128; ++j)
          pair_load_2d(b + j * 8192, &maps.b[which], n * BN + (rank * (BN / 128) + j) * 64, kk, bar);
      } else {
        const int which = m >= plan.w_half, row = (m - (which ? plan.w_half : 0)) * BM;
#pragma unroll
        for (int j = 0; j < BM / 64; ++j) pair_load_2d(a + j * 8192, &maps.wa[which], row + j * 64, k * BK, bar);
#pragma unroll
        for (int j = 0; j < BN / 128; ++j)
          pair_load_2d(b + j * 8192, &maps.wb, n * BN + (rank * (BN / 128) + j) * 64, k * BK, bar);
      }
    };
    int it = 0;
    bool ok = true;
    Item tile;
    for (int i = 0; ok && item_of<kKind>(plan, i, tile); ++i) {
      int m, n;
      tile_of<kKind>(plan, tile, m, n);
      for (int k = tile.from; k < tile.to; ++k, ++it) {
        const int s = it % kStages;
        if (it >= kStages && !(ok = mbar_wait(empty + s, (it / kStages - 1) & 1, status, 1))) break;
        if (elect_one()) load(s, tile.weights, m, n, k);
        __syncwarp();
      }
    }
    // the last stages have to be done with before the block may end
    for (int j = max(0, it - kStages); j < it; ++j) mbar_wait(empty + j % kStages, (j / kStages) & 1, status, 2);
  } else if (warp == 1 && rank == 0) {  // products of both blocks
    int it = 0, done = 0;
    bool ok = true;
    Item tile;
    for (int i = 0; ok && item_of<kKind>(plan, i, tile); ++i, ++done) {
      // the forward's operands lie along the sum; dx's right one across it, the weights' gradients' both
      const bool a_mn = kKind == kGrads && tile.weights;
      constexpr bool kBmn = kKind == kGrads;
      const uint32_t idesc = idesc_bf16(2 * BM, BN, a_mn, kBmn);
      const int acc = done & 1;
      const uint64_t step_a = a_mn ? mdesc_step(16) : kdesc_step(BM, 16);
      if (done >= 2 && !(ok = mbar_wait(tempty + acc, (done / 2 - 1) & 1, status, 3))) break;
      fence_cluster();
      tc_fence_after();
      for (int k = tile.from; k < tile.to; ++k, ++it) {
        const int s = it % kStages;
        if (!(ok = mbar_wait(full + s, (it / kStages) & 1, status, 4))) break;
        tc_fence_after();
        uint8_t *a = smem + s * kBytesStage, *b = a + kBytesA;
        const uint64_t da = a_mn ? mdesc(a, BK, 0) : kdesc(a, BM, 0), db = kBmn ? mdesc(b, BK, 0) : kdesc(b, BN / 2, 0);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK; kk += 16)
            pair_mma_bf16(tmem + acc * BN, da + (kk / 16) * step_a, db + (kBmn ? mdesc_step(kk) : kdesc_step(BN / 2, kk)),
                          idesc, k > tile.from || kk > 0);
          pair_commit(empty + s);
        }
        __syncwarp();
      }
      if (elect_one()) pair_commit(tfull + acc);
      __syncwarp();
    }
    // the last products have to end before the tensor memory is given back
    for (int d = max(0, done - 2); d < done; ++d) mbar_wait(tfull + (d & 1), (d / 2) & 1, status, 5);
  } else if (warp >= 4) {  // results
    const int q = warp & 3, row = q * 32 + lane, acc = (warp >> 2) - 1, bar = 1 + acc;
    const bool leader = q == 0 && lane == 0;
    out += acc * kBytesPiece;
    const uint32_t drained = in_first_block(tempty + acc);
    Item tile;
    for (int done = acc; item_of<kKind>(plan, done, tile); done += 2) {
      int m, n;
      tile_of<kKind>(plan, tile, m, n);
      const bool there = m < (tile.weights ? plan.w_m_tiles : plan.m_tiles);  // (an odd last row tile has no neighbour)
      const bool ok = mbar_wait(tfull + acc, (done / 2) & 1, status, 6);
      if (named_bar_or(bar, 128, !ok)) break;
      tc_fence_after();
      const uint32_t base = taddr(tmem, q * 32, acc * BN);
      if (kKind == kForward) {
#pragma unroll
        for (int c = 0; c < kOwn / 32; ++c) {
          uint32_t g[32], u[32];
          tmem_ld32_nowait(base + c * 32, g);
          tmem_ld32_nowait(base + kOwn + c * 32, u);
          tmem_wait_ld();
          settled(g), settled(u);
          float h[32];
          const auto products = [&](auto gelu) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float a, s;
              act_and_slope(__uint_as_float(g[e]), decltype(gelu)::value, a, s);
              h[e] = a * __uint_as_float(u[e]);
            }
          };
          if (args.gelu)
            products(std::true_type());
          else
            products(std::false_type());
          if (c % 2 == 0) {
            if (leader) tma_store_wait_read0();
            named_bar(bar, 128);
          }
          store_row_bf16(out, row, (c & 1) * 4, h, 4);
          if (c % 2) {
            fence_proxy_async();
            named_bar(bar, 128);
            const int col = n * kOwn + (c - 1) * 32;
            if (leader && there && col < args.F) {
              tma_store_2d(&maps.o, out, col, m * BM);
              tma_store_commit();
            }
          }
          if (stash && there) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n * kOwn + c * 32 + j * 8 < args.F)
                keep(stash, args, m * BM + row, n * kOwn + c * 32 + j * 8, g + 8 * j, u + 8 * j);
          }
        }
        tc_fence_before();
        if (lane == 0) arrive_in_first_block(drained);
      } else if (!tile.weights && plan.pieces > 1) {
        float4* to = part + (((size_t)tile.piece * plan.m_tiles + m) * (args.D / 4) + n * (BN / 4)) * BM + row;
#pragma unroll 1
        for (int c = 0; there && c < BN / 32 && n * BN + c * 32 < args.D; ++c, to += 8 * BM) {
          uint32_t v[32];
          tmem_ld32_nowait(base + c * 32, v);
          tmem_wait_ld();
          settled(v);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n * BN + c * 32 + e * 4 < args.D)
              to[e * BM] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                       __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
        }
        tc_fence_before();
        if (lane == 0) arrive_in_first_block(drained);
      } else {
        const int which = tile.weights && m >= plan.w_half, row0 = (m - (which ? plan.w_half : 0)) * BM;
        const CUtensorMap* to_map = tile.weights ? &maps.wo[which] : &maps.o;
#pragma unroll 1
        for (int p = 0; p < BN / 64; ++p) {
          uint32_t v[2][32];
          tmem_ld32_nowait(base + p * 64, v[0]);
          tmem_ld32_nowait(base + p * 64 + 32, v[1]);
          if (leader) tma_store_wait_read0();
          tmem_wait_ld();
          settled(v[0]), settled(v[1]);
          named_bar(bar, 128);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[c][e]);
            store_row_bf16(out, row, c * 4, f, 4);
          }
          fence_proxy_async();
          named_bar(bar, 128);
          if (leader && there && n * BN + p * 64 < args.D) {
            tma_store_2d(to_map, out, n * BN + p * 64, row0);
            tma_store_commit();
          }
        }
        tc_fence_before();
        if (lane == 0) arrive_in_first_block(drained);
      }
    }
    if (leader) tma_store_wait0();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // (nothing of the other block's is on its way here any more)
  if (warp == 2) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, kTmemAll);
  }
}

// dG and dU of the stashed G and U: a warp has eight rows of four pieces of eight columns.  status: cleared, where this is
// a call's first kernel (the forward's product clears it where that is).
__global__ void __launch_bounds__(256)
    k_ffn_gates(Args a, uint8_t* stash, const bf16* __restrict__ dh, bf16* dg, bf16* du, int* status) {
  if (status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int f = (blockIdx.y * 32 + warp * 4 + (lane & 3)) * 8;
  const int row = blockIdx.x * 8 + (lane >> 2);
  if (row >= a.M || f >= a.F) return;
  float g[8], u[8];
  const uint4 d4 = *reinterpret_cast<const uint4*>(dh + (size_t)row * a.F + f);
  kept_values(kept(stash, a, row, f, 0), g);
  kept_values(kept(stash, a, row, f, 1), u);
  const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
  uint32_t og[4], ou[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float dv[2], x[2], y[2];
    unpack(d[e], dv);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float act, slope;
      act_and_slope(g[2 * e + k], a.gelu, act, slope);
      x[k] = dv[k] * u[2 * e + k] * slope;
      y[k] = dv[k] * act;
    }
    og[e] = pack2(x[0], x[1]);
    ou[e] = pack2(y[0], y[1]);
  }
  *reinterpret_cast<uint4*>(dg + (size_t)row * a.F + f) = make_uint4(og[0], og[1], og[2], og[3]);
  *reinterpret_cast<uint4*>(du + (size_t)row * a.F + f) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
}

// dx of its sums' pieces [pieces, row tiles, D / 4, 128] of four columns, in order: a warp has eight rows of four pieces of
// eight columns.
__global__ void __launch_bounds__(256)
    k_ffn_join(Args a, const float4* __restrict__ part, int m_tiles, int pieces, bf16* dx) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.y * 32 + warp * 4 + (lane & 3)) * 8, row = blockIdx.x * 8 + (lane >> 2);
  if (row >= a.M || c >= a.D) return;
  const float4* from = part + ((size_t)(row / BM) * (a.D / 4) + c / 4) * BM + row % BM;
  float s[8] = {};
#pragma unroll 4
  for (int p = 0; p < pieces; ++p, from += (size_t)m_tiles * (a.D / 4) * BM) {
    const float4 x = from[0], y = from[BM];
    s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
  }
  *reinterpret_cast<uint4*>(dx + (size_t)row * a.D + c) = make_uint4(pack2(s[0], s[1]), pack2(s[2], s[3]), pack2(s[4], s[5]),
                                                                     pack2(s[6], s[7]));
}

// The forward with few rows, where all that counts is how fast the weights come in: one tile a block, of up to 128 rows and
// as many features (`wide`, of G and of U) as give every SM a block; stages of just the rows that there are.  (The products
// take 128 rows of what lies there; results of those behind the last row go nowhere.)
struct Few {
  int rows, wide, stages, m_tiles;  // rows and wide: multiples of 8
};
constexpr int kFewThreads = 192, kFewStages = 16;
__global__ void __launch_bounds__(kFewThreads, 1)
    k_ffn_few(const __grid_constant__ Maps maps, Few few, Args args, bf16* h, uint8_t* stash, int* status) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ uint64_t full[kFewStages], empty[kFewStages], done;
  __shared__ uint32_t slot;
  uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m = blockIdx.x % few.m_tiles, n = blockIdx.x / few.m_tiles, steps = (args.D + BK - 1) / BK;
  const int bytes_a = few.rows * 128, bytes_b = few.wide * 128, bytes = bytes_a + 2 * bytes_b;
  const auto load = [&](int k, int s) {
    uint8_t *a = smem + s * bytes, *b = a + bytes_a;
    mbar_expect_tx(full + s, bytes);
    tma_load_2d(b, &maps.b[0], k * BK, n * few.wide, full + s);
    tma_load_2d(b + bytes_b, &maps.b[1], k * BK, n * few.wide, full + s);
    tma_load_2d(a, &maps.a[0], k * BK, m * few.rows, full + s);
  };
  const int ahead = steps < few.stages ? steps : few.stages;
  if (warp == 0) {  // the first stages' copies set out before the block is ready for them
    if (elect_one()) {
      for (int s = 0; s < few.stages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
      mbar_init(&done, 1);
      mbar_init_fence();
      if (blockIdx.x == 0) *status = 0;
      for (int k = 0; k < ahead; ++k) load(k, k);
    }
    __syncwarp();
  }
  if (warp == 1) tmem_alloc(&slot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = slot;
  if (warp == 0) {  // copies
    int k = ahead;
    for (int s = 0, turn = 0; k < steps; ++k) {
      if (!mbar_wait(empty + s, turn & 1, status, 1)) break;
      if (elect_one()) load(k, s);
      __syncwarp();
      if (++s == few.stages) s = 0, ++turn;
    }
    // what is still on its way has to arrive before the block may end
    for (int j = max(0, k - few.stages); j < k; ++j) mbar_wait(full + j % few.stages, (j / few.stages) & 1, status, 2);
  } else if (warp == 1) {  // products
    const uint32_t idesc = idesc_bf16(BM, 2 * few.wide, false, false);
    for (int k = 0, s = 0, turn = 0; k < steps; ++k) {
      if (!mbar_wait(full + s, turn & 1, status, 3)) break;
      tc_fence_after();
      const uint64_t da = kdesc(smem + s * bytes, BM, 0), db = kdesc(smem + s * bytes + bytes_a, 2 * few.wide, 0);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK; kk += 16)
          mma_bf16(tmem, da + kdesc_step(BM, kk), db + kdesc_step(BM, kk), idesc, k > 0 || kk > 0);
        mma_commit(empty + s);
      }
      __syncwarp();
      if (++s == few.stages) s = 0, ++turn;
    }
    if (elect_one()) mma_commit(&done);
    __syncwarp();
  } else {  // results
    const int q = warp & 3, r = q * 32 + lane, row = m * few.rows + r;
    const bool live = r < few.rows && row < args.M;
    // (every thread waits: the products end before the tensor memory is given back)
    if (mbar_wait(&done, 0, status, 4) && q * 32 < few.rows) {
      tc_fence_after();
      for (int j = 0; j < few.wide; j += 8) {
        uint32_t g[8], u[8];
        tmem_ld8_nowait(taddr(tmem, q * 32, j), g);
        tmem_ld8_nowait(taddr(tmem, q * 32, few.wide + j), u);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) asm volatile("" : "+r"(g[e]), "+r"(u[e]));
        const int f = n * few.wide + j;
        if (!live || f >= args.F) continue;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float act, slope;
          act_and_slope(__uint_as_float(g[e]), args.gelu, act, slope);
          o[e] = act * __uint_as_float(u[e]);
        }
        *reinterpret_cast<uint4*>(h + (size_t)row * args.F + f) =
            make_uint4(pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
        if (stash) keep(stash, args, row, f, g, u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

struct Call {
  Args a;
  const void *x, *wg, *wu, *dh;
  void *h, *dx, *dwg, *dwu;
  uint8_t* stash;
  bf16 *dg, *du;
  float4* part;  // room for dx's sums' pieces
  int* status;
  Plan plan;     // the gradients'
  bool narrow;
};

cudaError_t map(CUtensorMap* m, const void* p, int cols, int rows, long long stride, int box_cols, int box_rows) {
  return make_tmap_rows_bf16(m, p, cols, rows, stride, box_cols, box_rows);
}

template <Kind kKind, int BN>
cudaError_t launch(const char* name, const Maps& maps, const Plan& plan, const Call& c, cudaStream_t st) {
  const auto kernel = k_ffn_product<kKind, BN>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Stages<BN>::kSmem, allowed);
  if (e != cudaSuccess) return e;
  const int pairs = pairs_of(plan.m_tiles, plan.n_tiles) * plan.pieces +
                    (kKind == kGrads ? pairs_of(plan.w_m_tiles, plan.w_n_tiles) : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs < kSMs / 2 ? 2 * pairs : kSMs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Stages<BN>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t launched = cudaSuccess;
  SSD_LAUNCH(name, st,
             launched = cudaLaunchKernelEx(&cfg, kernel, maps, plan, c.a, kKind == kForward ? c.stash : (uint8_t*)nullptr,
                                           c.part, c.status));
  return launched;
}
int up(long long a, int b) { return (int)((a + b - 1) / b); }

// Steps that a tile's results take: a tile of fewer ends no sooner.  Gradients with 10 and with 4, us: 256 rows of 2560 and
// 7680 53 and 63; 512 of 2560 and 7680 69 and 76; 453 of 712 and 11912 51 and 55; 128 of 1024 and 4096 26 with either.
constexpr int kLeast = 10;
// dx and the weights' gradients in one launch: how many of the latter's pairs of tiles every pair of blocks takes, so
// that the last ends soonest (steps of those with one more of dx's, and of the others).  Returns the steps until then.  8192
// rows of 2560 and 7680: 320 pairs of tiles of 240 steps and 600 of 128 on 76 pairs of blocks end after 2112 steps, one kind
// after the other they would after 2224.
long long balance(Plan* p) {
  const int tiles = pairs_of(p->m_tiles, p->n_tiles) * p->pieces, w_tiles = pairs_of(p->w_m_tiles, p->w_n_tiles);
  const int steps = up(p->steps, p->pieces), w_steps = p->w_steps > kLeast ? p->w_steps : kLeast;
  const int blocks = tiles + w_tiles < kSMs / 2 ? tiles + w_tiles : kSMs / 2;
  const int more = tiles % blocks, each = tiles / blocks, others = blocks - more;
  long long best = -1;
  const int least = w_tiles / blocks - steps / w_steps - 2;  // (with fewer, the others would end later than the first)
  for (int both = least > 0 ? least : 0; both <= (w_tiles + blocks - 1) / blocks; ++both) {
    const int left = w_tiles - both * blocks > 0 ? w_tiles - both * blocks : 0;
    const long long first = more ? (each + 1ll) * steps + (long long)both * w_steps : 0;
    const long long second = (long long)each * steps + (both + (left + others - 1) / others) * (long long)w_steps;
    const long long end = first > second ? first : second;
    if (best < 0 || end < best) best = end, p->both = both;
  }
  return best;
}

// Whether tiles of half the columns end sooner: their step takes about 5/8 of a whole one's, and they are dealt out more
// evenly.  Forward, us: 2088 rows of 568 and 2096 in narrow ones 25.3, in wide ones 26.9; 2048 of 1024 and 4096 43.6 and
// 39.4; 8192 of 2560 and 7680 449 and 368.  Gradients: 131 rows of 632 and 832 14.2 and 20.2; 6800 of 272 and 2000 44 and 61;
// 2048 of 1024 and 4096 55 and 48; 8192 of 2560 and 7680 830 and 681.
constexpr int kWideStep = 8, kNarrowStep = 5;
bool sooner(long long narrow_steps, long long wide_steps) { return narrow_steps * kNarrowStep < wide_steps * kWideStep; }

// The gradients' tiles: wide or narrow, and dx's sums in as many pieces as end soonest, the launch that joins them (12 steps)
// and the bytes it reads counted in.  With few rows dx is a few tiles of long sums (the gradients and the joining
// launch, us, in pieces and in one: 125 rows of 288 and 8816 25 and 59; 453 of 712 and 11912 51 and 111; 256 of 2560 and 7680
// 53 and 56; 1501 of 776 and 2056 stay in one, 35 and 41 in two).
constexpr int kMostPieces = 16, kLeastSteps = 8, kJoinSteps = 12;  // pieces, steps of one
Plan grads_plan(const Args& a, bool* narrow) {
  Plan best = {};
  long long least = -1;
  for (const int cols : {256, 128}) {
    Plan p = {up(a.M, BM),     up(a.D, cols), 2 * up(a.F, BK), up(a.F, BK),
              2 * up(a.F, BM), up(a.D, cols), up(a.M, BK),     up(a.F, BM)};
    const auto fits = [&](int pieces) {
      return pieces <= kMostPieces && p.steps >= kLeastSteps * pieces &&
             (long long)pairs_of(p.m_tiles, p.n_tiles) * pieces <= 4 * kSMs;
    };
    for (p.pieces = 1; p.pieces == 1 || fits(p.pieces); ++p.pieces) {
      long long end = balance(&p) * (cols == 256 ? kWideStep : kNarrowStep);
      if (p.pieces > 1) end += kWideStep * (kJoinSteps + (long long)p.pieces * a.M * a.D / (1 << 18));  // (2 MB a step)
      if (least < 0 || end < least) least = end, best = p, *narrow = cols == 128;
    }
  }
  return best;
}

// Few rows: where tiles of 128 rows and 128 features leave SMs without one.
bool few_rows(const Args& a, Few* few) {
  const int mt = up(a.M, BM);
  if ((long long)mt * up(a.F, 128) > kSMs) return false;
  few->m_tiles = mt;
  few->rows = up(up(a.M, mt), 8) * 8;
  few->wide = up(up(a.F, kSMs / mt), 8) * 8;
  const int stage = (few->rows + 2 * few->wide) * 128, room = kMostSmem - 2048 - kBytesA;
  few->stages = room / stage < kFewStages ? room / stage : kFewStages;
  return true;
}

cudaError_t forward(const Call& c, cudaStream_t st) {
  Maps maps;
  Few few;
  const bool is_few = few_rows(c.a, &few);
  const auto rounds = [&](int cols) { return up(pairs_of(up(c.a.M, BM), up(c.a.F, cols)), kSMs / 2); };
  const bool narrow = sooner(rounds(64), rounds(128));
  const int wide = is_few ? few.wide : narrow ? 64 : 128;
  cudaError_t e = map(&maps.a[0], c.x, c.a.D, c.a.M, c.a.xs, BK, is_few ? few.rows : BM);
  if (e == cudaSuccess) e = map(&maps.b[0], c.wg, c.a.D, c.a.F, c.a.D, BK, wide);
  if (e == cudaSuccess) e = map(&maps.b[1], c.wu, c.a.D, c.a.F, c.a.D, BK, wide);
  if (e == cudaSuccess && !is_few) e = map(&maps.o, c.h, c.a.F, c.a.M, c.a.F, 64, BM);
  if (e != cudaSuccess) return e;
  maps.a[1] = maps.a[0];
  if (!is_few) {
    maps.wa[0] = maps.wa[1] = maps.wb = maps.wo[0] = maps.wo[1] = maps.a[0];
    const Plan p = {up(c.a.M, BM), up(c.a.F, wide), up(c.a.D, BK), 0, 0, 0, 0, 0, 0, 1};
    return narrow ? launch<kForward, 128>("k_ffn_forward", maps, p, c, st)
                  : launch<kForward, 256>("k_ffn_forward", maps, p, c, st);
  }
  maps.o = maps.wa[0] = maps.wa[1] = maps.wb = maps.wo[0] = maps.wo[1] = maps.a[0];
  // (behind the last stage's rows the products still read what 128 rows would take)
  const int smem = few.stages * (few.rows + 2 * few.wide) * 128 + kBytesA + 1024;
  static std::atomic<unsigned long long> allowed{0};
  if ((e = allow_smem(reinterpret_cast<const void*>(k_ffn_few), kMostSmem - 1024, allowed)) != cudaSuccess) return e;
  SSD_LAUNCH("k_ffn_few", st,
             k_ffn_few<<<few.m_tiles * up(c.a.F, few.wide), kFewThreads, smem, st>>>(maps, few, c.a, (bf16*)c.h, c.stash,
                                                                                     c.status));
  return cudaGetLastError();
}

cudaError_t backward(const Call& c, bool first, cudaStream_t st) {
  const Args& a = c.a;
  SSD_LAUNCH("k_ffn_gates", st,
             k_ffn_gates<<<dim3(up(a.M, 8), up(a.F, 256)), 256, 0, st>>>(a, c.stash, (const bf16*)c.dh, c.dg, c.du,
                                                                     first ? c.status : nullptr));
  cudaError_t e = cudaGetLastError();
  Maps maps;
  if (e == cudaSuccess) e = map(&maps.a[0], c.dg, a.F, a.M, a.F, BK, BM);
  if (e == cudaSuccess) e = map(&maps.a[1], c.du, a.F, a.M, a.F, BK, BM);
  if (e == cudaSuccess) e = map(&maps.b[0], c.wg, a.D, a.F, a.D, 64, BK);
  if (e == cudaSuccess) e = map(&maps.b[1], c.wu, a.D, a.F, a.D, 64, BK);
  if (e == cudaSuccess) e = map(&maps.o, c.dx, a.D, a.M, a.D, 64, BM);
  if (e == cudaSuccess) e = map(&maps.wa[0], c.dg, a.F, a.M, a.F, 64, BK);
  if (e == cudaSuccess) e = map(&maps.wa[1], c.du, a.F, a.M, a.F, 64, BK);
  if (e == cudaSuccess) e = map(&maps.wb, c.x, a.D, a.M, a.xs, 64, BK);
  if (e == cudaSuccess) e = map(&maps.wo[0], c.dwg, a.D, a.F, a.D, 64, BM);
  if (e == cudaSuccess) e = map(&maps.wo[1], c.dwu, a.D, a.F, a.D, 64, BM);
  if (e != cudaSuccess) return e;
  const Plan& p = c.plan;
  e = c.narrow ? launch<kGrads, 128>("k_ffn_grads", maps, p, c, st) : launch<kGrads, 256>("k_ffn_grads", maps, p, c, st);
  if (e != cudaSuccess || p.pieces == 1) return e;
  SSD_LAUNCH("k_ffn_join", st,
             k_ffn_join<<<dim3(up(a.M, 8), up(a.D, 256)), 256, 0, st>>>(a, c.part, p.m_tiles, p.pieces, (bf16*)c.dx));
  return cudaGetLastError();
}

ssd_status make_args(const ssd_ffn_problem* p, Args* a) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->io_dtype != SSD_F32 && p->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (p->activation != SSD_ACT_SILU && p->activation != SSD_ACT_GELU) return SSD_ERR_INVALID_ARG;
  if (p->rows < 1 || p->dim < 1 || p->hidden < 1 || p->x_stride < 0) return SSD_ERR_INVALID_ARG;
  if (p->io_dtype != SSD_BF16) return SSD_ERR_DTYPE;
  const int64_t most = 1 << 20;
  if (p->dim > most || p->hidden > most || p->rows > (1 << 24) || p->dim % 8 || p->hidden % 8 || p->x_stride % 8 ||
      (p->x_stride && p->x_stride < p->dim) || p->x_stride >= (1ll << 38))
    return SSD_ERR_SHAPE;
  *a = Args{(int)p->rows, (int)p->dim, (int)p->hidden, p->activation == SSD_ACT_GELU, p->x_stride ? p->x_stride : p->dim};
  return SSD_OK;
}

size_t stash_bytes_of(const Args& a) { return kept_pieces(a) * 2 * 24; }

size_t workspace(Call* c, bool back, bool stashed, void* ws) {
  Carver cv(ws);
  c->status = static_cast<int*>(ws);
  if (back) {
    c->dg = cv.take<bf16>((size_t)c->a.M * c->a.F);
    c->du = cv.take<bf16>((size_t)c->a.M * c->a.F);
    c->plan = grads_plan(c->a, &c->narrow);
    if (c->plan.pieces > 1) c->part = cv.take<float4>((size_t)c->plan.pieces * c->plan.m_tiles * BM * (c->a.D / 4));
    if (!stashed) {
      c->stash = cv.take<uint8_t>(stash_bytes_of(c->a));
      c->h = cv.take<bf16>((size_t)c->a.M * c->a.F);  // of the forward that is made again
    }
  }
  return cv.off;
}

ssd_status check(std::initializer_list<const void*> req, const void* stash) {
  for (const void* p : req)
    if (!p) return SSD_ERR_INVALID_ARG;
  for (const void* p : req)
    if (off(p, 16)) return SSD_ERR_ALIGNMENT;
  return off(stash, 16) ? SSD_ERR_ALIGNMENT : SSD_OK;
}

}  // namespace
}  // namespace ffn
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_ffn_stash_size(const ssd_ffn_problem* prob, size_t* bytes) {
  ffn::Args a;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = ffn::make_args(prob, &a);
  if (s != SSD_OK) return s;
  *bytes = ffn::stash_bytes_of(a);
  return SSD_OK;
}

ssd_status ssd_ffn_workspace_size(const ssd_ffn_problem* prob, int backward, int stashed, size_t* bytes) {
  ffn::Call c = {};
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = ffn::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  *bytes = ffn::workspace(&c, backward != 0, stashed != 0, nullptr);
  return SSD_OK;
}

ssd_status ssd_ffn_forward(const ssd_ffn_problem* prob, const void* x, const void* w_gate, const void* w_up, void* h,
                           void* stash, size_t stash_bytes, void* ws, size_t ws_bytes, void* cuda_stream) {
  ffn::Call c = {};
  ssd_status s = ffn::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  if ((s = ffn::check({x, w_gate, w_up, h, ws}, stash)) != SSD_OK) return s;
  if (stash && stash_bytes < ffn::stash_bytes_of(c.a)) return SSD_ERR_WORKSPACE;
  if (ws_bytes < ffn::workspace(&c, false, stash != nullptr, nullptr)) return SSD_ERR_WORKSPACE;
  ffn::workspace(&c, false, stash != nullptr, ws);
  c.x = x, c.wg = w_gate, c.wu = w_up, c.h = h, c.stash = static_cast<uint8_t*>(stash);
  return ffn::forward(c, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_ffn_backward(const ssd_ffn_problem* prob, const void* dh, const void* x, const void* w_gate, const void* w_up,
                            void* dx, void* dw_gate, void* dw_up, const void* stash, size_t stash_bytes, void* ws,
                            size_t ws_bytes, void* cuda_stream) {
  ffn::Call c = {};
  ssd_status s = ffn::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  if ((s = ffn::check({dh, x, w_gate, w_up, dx, dw_gate, dw_up, ws}, stash)) != SSD_OK) return s;
  if (stash && stash_bytes < ffn::stash_bytes_of(c.a)) return SSD_ERR_WORKSPACE;
  if (ws_bytes < ffn::workspace(&c, true, stash != nullptr, ws)) return SSD_ERR_WORKSPACE;
  c.x = x, c.wg = w_gate, c.wu = w_up, c.dh = dh, c.dx = dx, c.dwg = dw_gate, c.dwu = dw_up;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (stash)
    c.stash = static_cast<uint8_t*>(const_cast<void*>(stash));
  else
    e = ffn::forward(c, st);
  if (e == cudaSuccess) e = ffn::backward(c, stash != nullptr, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
