// The two sequential scans of the chunked delta rule on tcgen05: one block per (sequence, value head) walks its chunks
// of 64 steps in order (k_delta_scan) or in reverse (k_delta_rev).  The formulas are in ssd_delta.cu.
//
// Everything is transposed: a TMEM lane (and the four threads that serve it) is a column v of V, so S^T [128 v][K] is
// the left operand of every product and the results of one product, X^T = S^T K^T, R^T = Y^T T^T, S'^T += R^T K, are
// the left operand of the next after a few elementwise operations.  tcgen05 takes the left operand from tensor memory:
// the chain of a chunk never touches shared memory, which holds only the tiles that are read as right operands as they
// lie in global memory (K and Q by rows for S^T K^T, the same bytes by columns for R^T K).
//
// Twenty-four warps:
//   0-15   the chain: four warps a lane quadrant, each with a quarter of the columns; S stays in their registers (fp32)
//   16-19  beside the chain: o forward; dV and the scaled dO^T operand in reverse
//   20     issues every MMA
//   21-22  copy the next chunk's tiles (two stages; TMA where rows are whole 16-byte pieces)
//   23     sends off what is kept: the chain's warps leave S and R (dS' and dY) as tiles of shared memory while they wait
//          for MMAs, one bulk copy each
// Between two chunks lie three round trips through tensor memory (X, R, S'), which is what bounds the kernel: about
// 105 cycles of latency for each group of MMAs, 32 cycles for each 128 x 64 x 16 one (A in TMEM; 57 with A in shared
// memory), and the elementwise work of 128 x 64 and 128 x K values between them.  So the chain goes in two halves, warps
// 0-7 with the steps 0-31 and the first half of the keys and warps 8-15 with the others: while one half is at its
// elementwise work the MMAs run that need only the other's (X's first keys, R's first steps, the state's first half).
// Measured at K = V = 128, 128 heads of 64 chunks at once: 205 us forward with the stash, 3.2 us a chunk (1.08 GB moved,
// 5.2 TB/s: four fifths of a plain copy's rate), 201 us in reverse.
#include "delta_tc.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kChainWarps = 16, kSideWarps = 4;
constexpr int kMmaWarp = kChainWarps + kSideWarps;
constexpr int kLoadWarp0 = kMmaWarp + 1, kSendWarp = kLoadWarp0 + kLoadWarps;
constexpr int kThreads = 32 * (kSendWarp + 1);
constexpr uint32_t kTmemCols = 512;
constexpr int kSideBar = 1;  // named barrier of the side warps
constexpr uint32_t kKeep = 32768, kOut = 16384;

// A stage: [K; Q] rows as one 128-row K-major tile, V (or dO) [64][128], the chunk's record.  Beside the two stages the
// tiles through which results leave: the kept state, and after it in the same place R or dY, as the images that the
// gradient kernel reads; o or dV.
template <int KP>
struct Tiles {
  static constexpr uint32_t kKQ = 128 * KP * 2, kV = kC * 128 * 2;
  static constexpr uint32_t kRec = kKQ + kV;
  static constexpr uint32_t kBytes = (kRec + kRecordBytes + 1023) / 1024 * 1024;
};
template <int KP>
constexpr uint32_t scan_smem() {
  return 2 * Tiles<KP>::kBytes + kKeep + kOut + 1024;  // 1024: the tiles' alignment
}

struct Bars {
  uint64_t full[2], empty[2], tail, s[2], x[2], y[2], r[2], rp[2], ro, d[2], o, e2, f, kept, sent, dv, dv_sent,
      done;  // [2]: stages, halves
};
struct Maps {
  CUtensorMap k, q, v;  // v: V forward, dO in reverse
};

// 16 values as the bf16 operand columns [8] and what the rounding left [8], the two side by side in tensor memory.
__device__ __forceinline__ void put_split(uint32_t addr, const float (&x)[16]) {
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split(x[2 * i], x[2 * i + 1], h[i], l[i]);
  st8u(addr, h);
  st8u(addr + 8, l);
}
// What the copy warps do for one chunk: its tiles into a stage and an arrival on the stage's barrier.  TMA copies and
// the record arrive by themselves, but for a chunk of fewer than 64 steps: what a box brings in past its end belongs to
// the next sequence and is overwritten with zeros first.
template <int KP>
struct Loader {
  const Dims& d;
  const In& in;
  const Maps& maps;
  const bf16* v;  // null: zeros
  long long vstride;
  bool vvec, with_q;
  int hk, hv;
  uint64_t* tail;  // (completes once a block: a run has one cut chunk at most, so no warp can miss a phase)
  uint32_t tails;  // chunks of fewer steps so far

  __device__ bool operator()(uint8_t* st, uint64_t* full, const uint8_t* record, int first, int rows, int tid,
                             int* status) {
    const bool kt = d.kvec, qt = with_q && d.qvec, vt = vvec && v, cut = rows < kC;
    uint8_t* vtile = st + Tiles<KP>::kKQ;
    if (tid == 0) {
      uint64_t* bar = cut ? tail : full;
      const uint32_t rowsb = kC * 128;
      mbar_expect_tx(bar, kRecordBytes + rowsb * ((kt ? KP / 64 : 0) + (qt ? KP / 64 : 0) + (vt ? 2 : 0)));
      bulk_load(smem_u32(st + Tiles<KP>::kRec), record, kRecordBytes, bar);
#pragma unroll
      for (int a = 0; a < KP / 64; ++a) {
        if (kt) tma_load_3d(st + a * 128 * 128, &maps.k, 64 * a, hk, first, bar);
        if (qt) tma_load_3d(st + a * 128 * 128 + kC * 128, &maps.q, 64 * a, hk, first, bar);
      }
      if (vt)
        for (int a = 0; a < 2; ++a) tma_load_3d(vtile + a * kC * 128, &maps.v, 64 * a, hv, first, bar);
    }
    if (!kt) load_elements(st, 128, KP, in.k + (long long)first * d.ks + (long long)hk * d.K, d.ks, rows, d.K, tid);
    if (with_q && !qt)
      load_elements(st + kC * 128, 128, KP, in.q + (long long)first * d.qs + (long long)hk * d.K, d.qs, rows, d.K, tid);
    if (!v)
      zero_rows(vtile, kC, 2, 0, tid);
    else if (!vt)
      load_elements(vtile, kC, 128, v + (long long)first * vstride + (long long)hv * d.V, vstride, rows, d.V, tid);
    bool ok = true;
    if (cut) {
      ok = wait_warp(tail, tails & 1, status, 43);
      ++tails;
      if (kt) zero_rows(st, 128, KP / 64, rows, tid);
      if (qt) zero_rows(st + kC * 128, 128, KP / 64, rows, tid);
      if (vt) zero_rows(vtile, kC, 2, rows, tid);
    }
    fence_proxy_async();  // the MMAs read these tiles
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(full);
    if (cut && tid == 0) mbar_arrive(full);  // in the place of the arrival that announced the bytes, on the other barrier
    return ok;
  }
};

// s [K, V] fp32 to and from a thread's keys k0 .. k0 + NK - 1 of lane v: neighbouring lanes are neighbouring columns.
template <int NK>
__device__ __forceinline__ void read_state(float (&S)[NK], const float* s, int K, int V, int k0, int v) {
#pragma unroll
  for (int i = 0; i < NK; ++i) S[i] = s && k0 + i < K && v < V ? s[(size_t)(k0 + i) * V + v] : 0.f;
}
template <int NK>
__device__ __forceinline__ void write_state(float* s, const float (&S)[NK], int K, int V, int k0, int v) {
#pragma unroll
  for (int i = 0; i < NK; ++i)
    if (k0 + i < K && v < V) s[(size_t)(k0 + i) * V + v] = S[i];
}

// Columns of tensor memory.  fp32 results: X (then Y high, low in place), QS (forward: (Q S)^T; reverse: U), R (then R' high, low in place), O2 (forward: (P R)^T) or F (reverse: the scaled dO^T, high and low), D (the state's
// update); the state's operand, high and low.  R's operand for o lies over X.
template <int KP>
struct Cols {
  static constexpr int X = 0, QS = 64, R = 128, O2 = 192, D = 256, Sh = 384, Sl = Sh + KP / 2, Ro = X;
};
// Operand columns of the 16-value block kb: 8 high, 8 low, where its 16 fp32 values were.
__device__ __forceinline__ constexpr int pair_col(int base, int kb, bool low) { return base + 16 * kb + (low ? 8 : 0); }

struct Block {
  int hv, hk;
  Seq sq;
  size_t unit, su;  // sequence and value head; its state's offset
};
// The (sequence, value head) of a place in the grid.  Packed: the longest sequences first, so that what runs last is
// short: 24 sequences of 20011 steps and 32 heads of 128 x 96 take 222 us, in their own order 253.
__device__ __forceinline__ int unit_of(const Dims& d, const Table& tb, int place) {
  if (!d.packed || d.N > kRanked) return place;
  const int n = place / d.HV;
  return tb.order[n] * d.HV + (place - n * d.HV);
}
__device__ __forceinline__ Block block_of(const Dims& d, const Table& tb, int unit) {
  Block b;
  const int n = unit / d.HV;
  b.hv = unit - n * d.HV;
  b.hk = b.hv / d.G;
  b.sq = sequence(d, tb, n);
  b.unit = (size_t)unit;
  b.su = b.unit * d.K * d.V;
  return b;
}
// The chunks c0 .. c1 - 1 of a block's sequence that it walks, from where to where its state goes, and whether it is a
// map (an identity to start from, no V).
struct Run {
  int c0, c1;
  const float* from;
  float* to;
  int rows, columns;  // of the state at `to`
  bool map;
};
// part: in the order of the walk, `back`: from the last chunk on.
__device__ __forceinline__ Run run_of(const Dims& d, const Split& sp, const Block& b, int part, bool back, bool map,
                                      bool first_pass, const float* s0, float* s_final) {
  Run r;
  const int nc = b.sq.nc, per = (nc + sp.parts - 1) / sp.parts;
  r.c0 = min(nc, (back ? sp.parts - 1 - part : part) * per);
  r.c1 = min(nc, r.c0 + per);
  float* states = sp.states + (b.unit * (sp.parts - 1) + part) * d.K * d.V;
  r.map = map;
  r.rows = map ? d.KP : d.K;
  r.columns = map ? d.KP : d.V;
  if (first_pass) {
    r.from = part == 0 && s0 ? s0 + b.su : nullptr;
    r.to = map ? sp.maps + (b.unit * (sp.parts - 2) + part - 1) * d.KP * d.KP : states;
  } else {
    r.from = part > 0 ? states - d.K * d.V : s0 ? s0 + b.su : nullptr;
    r.to = part == sp.parts - 1 && s_final ? s_final + b.su : nullptr;
  }
  return r;
}

__device__ __forceinline__ void init_bars(Bars* b) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&b->full[i], kLoadWarps + 1);
    mbar_init(&b->empty[i], 1 + kChainWarps + kSideWarps);
  }
  mbar_init(&b->tail, 1);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&b->s[i], kChainWarps / 2);
    mbar_init(&b->x[i], 1);
    mbar_init(&b->y[i], kChainWarps / 2);
    mbar_init(&b->r[i], 1);
    mbar_init(&b->rp[i], kChainWarps / 2);
    mbar_init(&b->d[i], 1);
  }
  mbar_init(&b->ro, kChainWarps);
  mbar_init(&b->o, 1);
  mbar_init(&b->e2, kSideWarps);
  mbar_init(&b->f, kSideWarps);
  mbar_init(&b->kept, kChainWarps);
  mbar_init(&b->sent, 1);
  mbar_init(&b->dv, kChainWarps);
  mbar_init(&b->dv_sent, kSideWarps);
  mbar_init(&b->done, 1);
  mbar_init_fence();
}

// A chain thread's keys as operand columns: high parts into Sh, low parts into Sl.
template <int KP>
__device__ __forceinline__ void put_state(uint32_t tm, int lane0, int wg, const float (&S)[KP / 4]) {
#pragma unroll
  for (int b = 0; b < KP / 64; ++b) {
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split(S[16 * b + 2 * i], S[16 * b + 2 * i + 1], h[i], l[i]);
    st8u(taddr(tm, lane0, Cols<KP>::Sh + wg * (KP / 8) + 8 * b), h);
    st8u(taddr(tm, lane0, Cols<KP>::Sl + wg * (KP / 8) + 8 * b), l);
  }
}
// Values b .. b + 7 (b = 0, 8) of the same layout as put_split's.
__device__ __forceinline__ void put_split8(uint32_t addr, int b, const float (&x)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(x[2 * i], x[2 * i + 1], h[i], l[i]);
  st4u(addr + b / 2, h);
  st4u(addr + b / 2 + 8, l);
}
// The high parts as their pieces of row v of the state's image.
template <int KP>
__device__ __forceinline__ void keep_state(uint8_t* tile, int VP, int v, int k0, const float (&S)[KP / 4]) {
  if (v < VP)
#pragma unroll
    for (int j = 0; j < KP / 32; ++j)
      *reinterpret_cast<uint4*>(tile + (k0 >> 6) * VP * 128 + sw128_chunk(v, ((k0 & 63) >> 3) + j)) =
          make_uint4(pack(S[8 * j], S[8 * j + 1]), pack(S[8 * j + 2], S[8 * j + 3]), pack(S[8 * j + 4], S[8 * j + 5]),
                     pack(S[8 * j + 6], S[8 * j + 7]));
}
// The warp's part of a tile that is sent off has been written.
__device__ __forceinline__ void signal_tile(uint64_t* bar, int lane) {
  fence_proxy_async();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// S = keep S + D
template <int KP>
__device__ __forceinline__ void update_state(uint32_t tm, int lane0, int k0, float keep, float (&S)[KP / 4]) {
#pragma unroll
  for (int b = 0; b < KP / 64; ++b) {
    float x[16];
    ld16(taddr(tm, lane0, Cols<KP>::D + k0 + 16 * b), x);
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      fma2(S[16 * b + i], S[16 * b + i + 1], keep, keep, S[16 * b + i], S[16 * b + i + 1], x[i], x[i + 1]);
  }
  tc_fence_before();
}

// The sending warp: two tiles a chunk out of one place, each free again once its copy has read it.
__device__ __forceinline__ void send_kept(Bars& bars, const uint8_t* tile, uint8_t* first, size_t step1, uint32_t bytes1,
                                          uint8_t* second, size_t step2, uint32_t bytes2, long long stride, int n, int lane,
                                          int* status) {
  for (int i = 0; i < 2 * n; ++i) {
    if (!wait_warp(&bars.kept, i & 1, status, 91)) break;
    if (lane == 0) {
      uint8_t* dst = i & 1 ? second + (long long)step2 * stride * (i >> 1) : first + (long long)step1 * stride * (i >> 1);
      bulk_store(dst, tile, i & 1 ? bytes2 : bytes1);
      tma_store_commit();
      tma_store_wait_read0();
      mbar_arrive(&bars.sent);
    }
    __syncwarp();
  }
  if (lane == 0) tma_store_wait0();
}

// The [64][128] bf16 tile of the side warps to rows of a tensor, first step at dst.
__device__ __forceinline__ void store_tile(const uint8_t* tile, bf16* dst, long long stride, int rows, int V, bool vec,
                                           int tid) {
  const bf16* t = reinterpret_cast<const bf16*>(tile);
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (tid >> 4) + 8 * i, c = 8 * (tid & 15);
      if (r < rows && c < V)
        *reinterpret_cast<uint4*>(dst + (long long)r * stride + c) = *reinterpret_cast<const uint4*>(t + r * 128 + c);
    }
  } else {
    for (int r = 0; r < rows; ++r)
      if (tid < V) dst[(long long)r * stride + tid] = t[r * 128 + tid];
  }
}

// ---------------------------------------------------------------- forward
template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    k_delta_scan(Dims d, Table tb, In in, const __grid_constant__ Maps maps, const uint8_t* records, Split sp,
                 bool first_pass, bf16* o, float* s_final, bf16* Sout, bf16* Rout, int* status) {
  using C = Cols<KP>;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tslot;
  __shared__ Block s_blk;  // (kept here: the chain has no registers to spare)
  __shared__ Run s_run;
  __shared__ __align__(16) float s_eg[2][kC];
  uint8_t* smem = aligned_smem(raw);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    init_bars(&bars);
    const int per_unit = first_pass ? 2 * sp.parts - 3 : sp.parts, place = blockIdx.x / per_unit, r = blockIdx.x - place * per_unit;
    s_blk = block_of(d, tb, unit_of(d, tb, place));
    s_run = run_of(d, sp, s_blk, first_pass ? (r + 1) >> 1 : r, false, first_pass && r > 0 && !(r & 1), first_pass,
                           in.s0, s_final);
  }
  if (w == kMmaWarp) tmem_alloc(&tslot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tslot;
  // blocks of a sequence and value head: its runs; of the first pass: run 0, then the runs 1 .. and their maps in turn
  const Block& blk = s_blk;
  const Run& run = s_run;
  const int nc = run.c1 - run.c0, chunk0 = blk.sq.chunk + run.c0, step0 = blk.sq.start + run.c0 * kC,
            steps = blk.sq.len - run.c0 * kC;
  const bool stash = Sout != nullptr;
  uint8_t* keep_tile = smem + 2 * Tiles<KP>::kBytes;

  if (w < kChainWarps) {
    const int wg = w >> 2, half = wg >> 1, lane0 = 32 * (w & 3), v = lane0 + lane, k0 = wg * (KP / 4);
    float S[KP / 4];
    read_state(S, run.from, d.K, d.V, k0, v);
    if (run.map)
#pragma unroll
      for (int j = 0; j < KP / 4; ++j) S[j] = k0 + j == v && v < d.K ? 1.f : 0.f;
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const uint8_t* st = smem + (c & 1) * Tiles<KP>::kBytes;
      const float* gates = reinterpret_cast<const float*>(st + Tiles<KP>::kRec + kRecordGates);
      put_state<KP>(tm, lane0, wg, S);
      signal_tmem(&bars.s[half], lane);
      if (stash) {
        if (c > 0 && !wait_warp(&bars.sent, 1, status, 11)) break;
        keep_state<KP>(keep_tile, d.VP, fresh(v), k0, S);
        signal_tile(&bars.kept, lane);
      }
      if (!wait_warp(&bars.full[c & 1], (c >> 1) & 1, status, 13)) break;
      if (!wait_warp(&bars.x[half], ph, status, 14)) break;
      tc_fence_after();
      float x[16];
      ld16(taddr(tm, lane0, C::X + 16 * wg), x);
      {
        const uint8_t* vt = st + Tiles<KP>::kKQ + 16 * wg * 128;
        const int vf = fresh(v);
#pragma unroll
        for (int b = 0; b < 16; b += 8) {  // Y = beta (V - e^G X)
          float e[8], be[8];
          lds8(gates + 16 * wg + b, e);
          lds8(gates + 2 * kC + 16 * wg + b, be);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float a0, a1;
            fma2(a0, a1, -e[i], -e[i + 1], x[b + i], x[b + i + 1],
                 __bfloat162float(*reinterpret_cast<const bf16*>(vt + v_off(b + i, vf))),
                 __bfloat162float(*reinterpret_cast<const bf16*>(vt + v_off(b + i + 1, vf))));
            mul2(x[b + i], x[b + i + 1], be[i], be[i + 1], a0, a1);
          }
        }
      }
      put_split(taddr(tm, lane0, C::X + 16 * wg), x);
      signal_tmem(&bars.y[half], lane);
      if (!wait_warp(&bars.r[half], ph, status, 15)) break;
      tc_fence_after();
      ld16(taddr(tm, lane0, C::R + 16 * wg), x);
#pragma unroll
      for (int b = 0; b < 16; b += 8) {  // R' = e^{G_end - G} R
        float a[8];
        lds8(gates + kC + 16 * wg + b, a);
#pragma unroll
        for (int i = 0; i < 8; i += 2) mul2(a[i], a[i + 1], a[i], a[i + 1], x[b + i], x[b + i + 1]);
        put_split8(taddr(tm, lane0, C::R + 16 * wg), b, a);
      }
      signal_tmem(&bars.rp[half], lane);
      const float keep = gates[kC - 1];
      if (o) {
        put_split(taddr(tm, lane0, C::Ro + 16 * wg), x);  // R itself
        signal_tmem(&bars.ro, lane);
      }
      if (stash) {
        if (!wait_warp(&bars.sent, 0, status, 18)) break;
        const int vf = fresh(v);
        if (vf < d.VP) {
          *reinterpret_cast<uint4*>(keep_tile + sw128_chunk(vf, 2 * wg)) =
              make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
          *reinterpret_cast<uint4*>(keep_tile + sw128_chunk(vf, 2 * wg + 1)) =
              make_uint4(pack(x[8], x[9]), pack(x[10], x[11]), pack(x[12], x[13]), pack(x[14], x[15]));
        }
        signal_tile(&bars.kept, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[c & 1]);
      if (!wait_warp(&bars.d[half], ph, status, 16)) break;
      tc_fence_after();
      update_state<KP>(tm, lane0, k0, keep, S);
    }
    if (run.to) write_state(run.to, S, run.rows, run.columns, k0, v);
  } else if (w < kMmaWarp) {
    const int lane0 = 32 * (w & 3), v = lane0 + lane, tid = threadIdx.x - 32 * kChainWarps;
    const long long os = (long long)d.HV * d.V;
    unsigned short* tile = reinterpret_cast<unsigned short*>(keep_tile + kKeep);
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const float* gates =
          reinterpret_cast<const float*>(smem + (c & 1) * Tiles<KP>::kBytes + Tiles<KP>::kRec + kRecordGates);
      // the decays that o needs, so that the stage is not held until o is there (and a wait for the stage in any case, so
      // that no warp is a phase ahead)
      bool ok = wait_warp(&bars.full[c & 1], (c >> 1) & 1, status, 23);
      if (lane < 16) s_eg[ph][16 * (w & 3) + lane] = gates[4 * kC + 16 * (w & 3) + lane];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[c & 1]);
      if (!o) {
        if (!ok) break;
        continue;
      }
      ok = ok && wait_warp(&bars.o, ph, status, 24);
      // the tile's last rows have been stored; all side warps go on together or not at all
      if (named_bar_or(kSideBar, 32 * kSideWarps, !ok)) break;
      tc_fence_after();
#pragma unroll 2
      for (int b = 0; b < 8; ++b) {
        uint32_t q[8], r[8];
        tmem_ld8_nowait(taddr(tm, lane0, C::QS + 8 * b), q);
        tmem_ld8_nowait(taddr(tm, lane0, C::O2 + 8 * b), r);
        float e[8];
        lds8(s_eg[ph] + 8 * b, e);
        tmem_wait_ld();
        if (b == 7) signal_read(&bars.e2, lane);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float a0, a1;
          fma2(a0, a1, e[i], e[i + 1], __uint_as_float(q[i]), __uint_as_float(q[i + 1]), __uint_as_float(r[i]),
               __uint_as_float(r[i + 1]));
          const uint32_t y = pack(a0, a1);
          tile[(8 * b + i) * 128 + v] = (unsigned short)y;
          tile[(8 * b + i + 1) * 128 + v] = (unsigned short)(y >> 16);
        }
      }
      named_bar(kSideBar, 32 * kSideWarps);
      store_tile(reinterpret_cast<const uint8_t*>(tile), o + ((long long)(step0 + c * kC) * d.HV + blk.hv) * d.V, os,
                 min(kC, steps - c * kC), d.V, d.ovec, tid);
    }
  } else if (w == kMmaWarp) {
    constexpr uint32_t n64 = idesc_bf16(128, 64, false, false), n32 = idesc_bf16(128, 32, false, false),
                       nk = idesc_bf16(128, KP, false, true), n64k = idesc_bf16(128, 64, false, true);
    constexpr int kH = KP / 32;  // 16-key blocks of a half of the state
    for (int c = 0; c < nc; ++c) {
      const uint32_t ph = c & 1;
      const uint8_t* st = smem + (c & 1) * Tiles<KP>::kBytes;
      const uint8_t* rc = st + Tiles<KP>::kRec;
      const uint64_t kd = kdesc(st, 128, 0), qd = kdesc(st + kC * 128, 128, 0), kd1 = kdesc(st + 32 * 128, 128, 0);
      // the same K rows as [step][key], all keys and the second half of them
      const uint64_t km = sdesc_sw128(smem_u32(st), 128 * 128, 1024);
      const uint64_t km1 = sdesc_sw128(smem_u32(st) + 128 * 128, 128 * 128, 1024);
      if (o && c > 0 && !wait_warp(&bars.o, ph ^ 1, status, 30)) break;  // (what X is written over)
      if (!wait_warp(&bars.full[c & 1], (c >> 1) & 1, status, 31)) break;
      if (!wait_warp(&bars.s[0], ph, status, 32)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kb = 0; kb < kH; ++kb) {
          mma_ts(tm + C::X, tm + C::Sh + 8 * kb, kd + kdesc_step(128, 16 * kb), n64, kb > 0);
          mma_ts(tm + C::X, tm + C::Sl + 8 * kb, kd + kdesc_step(128, 16 * kb), n64, true);
        }
      }
      __syncwarp();
      if (!wait_warp(&bars.s[1], ph, status, 38)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int kb = kH; kb < 2 * kH; ++kb) {
            mma_ts(tm + C::X + 32 * h, tm + C::Sh + 8 * kb, (h ? kd1 : kd) + kdesc_step(128, 16 * kb), n32, true);
            mma_ts(tm + C::X + 32 * h, tm + C::Sl + 8 * kb, (h ? kd1 : kd) + kdesc_step(128, 16 * kb), n32, true);
          }
          mma_commit(&bars.x[h]);
        }
      }
      __syncwarp();
      // (Q S)^T, of no hurry, while Y is made
      if (o) {
        if (c > 0 && !wait_warp(&bars.e2, ph ^ 1, status, 33)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kb = 0; kb < KP / 16; ++kb) {
            mma_ts(tm + C::QS, tm + C::Sh + 8 * kb, qd + kdesc_step(128, 16 * kb), n64, kb > 0);
            mma_ts(tm + C::QS, tm + C::Sl + 8 * kb, qd + kdesc_step(128, 16 * kb), n64, true);
          }
        }
        __syncwarp();
      }
      // R^T = Y^T T^T: the steps of 16-block kb reach the steps i >= 16 kb
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait_warp(&bars.y[h], ph, status, 34)) goto end;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kb = 2 * h; kb < 2 * h + 2; ++kb) {
            const uint32_t id = idesc_bf16(128, kC - 16 * kb, false, false);
            const uint32_t yh = tm + pair_col(C::X, kb, false), yl = tm + pair_col(C::X, kb, true);
            const uint64_t th = kdesc(rc + 16 * kb * 128, kC, 16 * kb), tl = kdesc(rc + 8192 + 16 * kb * 128, kC, 16 * kb);
            mma_ts(tm + C::R + 16 * kb, yh, th, id, kb > 0);
            mma_ts(tm + C::R + 16 * kb, yl, th, id, true);
            mma_ts(tm + C::R + 16 * kb, yh, tl, id, true);
          }
          mma_commit(&bars.r[h]);
        }
        __syncwarp();
      }
      if (!wait_warp(&bars.rp[0], ph, status, 35)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          mma_ts(tm + C::D, tm + pair_col(C::R, kb, false), km + mdesc_step(16 * kb), nk, kb > 0);
          mma_ts(tm + C::D, tm + pair_col(C::R, kb, true), km + mdesc_step(16 * kb), nk, true);
        }
      }
      __syncwarp();
      if (!wait_warp(&bars.rp[1], ph, status, 39)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (64 keys are one atom of the tile, which is not cut: all of it before the first half's signal)
          if (KP == 128 || h == 0)
#pragma unroll
            for (int kb = 2; kb < 4; ++kb) {
              mma_ts(tm + C::D + 64 * h, tm + pair_col(C::R, kb, false), (h ? km1 : km) + mdesc_step(16 * kb), n64k, true);
              mma_ts(tm + C::D + 64 * h, tm + pair_col(C::R, kb, true), (h ? km1 : km) + mdesc_step(16 * kb), n64k, true);
            }
          mma_commit(&bars.d[h]);
        }
      }
      __syncwarp();
      if (o) {
        if (!wait_warp(&bars.ro, ph, status, 36)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) {
            const uint32_t id = idesc_bf16(128, kC - 16 * kb, false, false);
            const uint32_t rh = tm + pair_col(C::Ro, kb, false), rl = tm + pair_col(C::Ro, kb, true);
            const uint64_t p0 = kdesc(rc + 2 * 8192 + 16 * kb * 128, kC, 16 * kb), p1 = kdesc(rc + 3 * 8192 + 16 * kb * 128, kC, 16 * kb);
            mma_ts(tm + C::O2 + 16 * kb, rh, p0, id, kb > 0);
            mma_ts(tm + C::O2 + 16 * kb, rl, p0, id, true);
            mma_ts(tm + C::O2 + 16 * kb, rh, p1, id, true);
          }
          mma_commit(&bars.o);
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit(&bars.empty[c & 1]);
      __syncwarp();
    }
  end:
    if (elect_one()) mma_commit(&bars.done);  // every MMA has finished before the tensor memory is given back
    __syncwarp();
    wait_warp(&bars.done, 0, status, 37);
  } else if (w == kSendWarp) {
    if (stash) {
      const size_t item = (size_t)chunk0 * d.HV + blk.hv;
      send_kept(bars, keep_tile, reinterpret_cast<uint8_t*>(Sout + item * d.VP * KP), (size_t)d.VP * KP * 2,
                (uint32_t)(d.VP * KP * 2), reinterpret_cast<uint8_t*>(Rout + item * d.VP * kC), (size_t)d.VP * kC * 2,
                (uint32_t)(d.VP * kC * 2), d.HV, nc, lane, status);
    }
  } else {
    const int tid = threadIdx.x - 32 * kLoadWarp0;
    Loader<KP> ld{d, in, maps, run.map ? nullptr : in.v, d.vs, d.vvec, o != nullptr, blk.hk, blk.hv, &bars.tail, 0};
    int loaded = -1;
    for (int c = 0; c < nc; ++c) {
      if (c >= 2 && !wait_warp(&bars.empty[c & 1], ((c >> 1) & 1) ^ 1, status, 41)) break;
      const bool ok = ld(smem + (c & 1) * Tiles<KP>::kBytes, &bars.full[c & 1],
                         records + ((size_t)(chunk0 + c) * d.HV + blk.hv) * kRecordBytes, step0 + c * kC,
                         min(kC, steps - c * kC), tid, status);
      loaded = c;
      if (!ok) break;
    }
    // no copy is in flight when the block ends, also where a wait above ran out
    for (int c = max(loaded - 1, 0); c <= loaded; ++c) wait_warp(&bars.full[c & 1], (c >> 1) & 1, status, 42);
  }
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tm, kTmemCols);
  }
}

// ---------------------------------------------------------------- reverse
template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
    k_delta_rev(Dims d, Table tb, In in, const __grid_constant__ Maps maps, const uint8_t* records, Split sp,
                bool first_pass, const bf16* dout, const float* ds_final, bf16* dv, float* ds0, bf16* dSout, bf16* dYout, int* status) {
  using C = Cols<KP>;
  constexpr int U = C::QS, F = C::O2;
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tslot;
  __shared__ Block s_blk;  // (kept here: the chain has no registers to spare)
  __shared__ Run s_run;
  uint8_t* smem = aligned_smem(raw);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    init_bars(&bars);
    const int per_unit = first_pass ? 2 * sp.parts - 3 : sp.parts, place = blockIdx.x / per_unit, r = blockIdx.x - place * per_unit;
    s_blk = block_of(d, tb, unit_of(d, tb, place));
    s_run = run_of(d, sp, s_blk, first_pass ? (r + 1) >> 1 : r, true, first_pass && r > 0 && !(r & 1), first_pass,
                           ds_final, ds0);
  }
  if (w == kMmaWarp) tmem_alloc(&tslot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tslot;
  const Block& blk = s_blk;
  const Run& run = s_run;
  const int nc = run.c1 - run.c0, chunk0 = blk.sq.chunk + run.c0, step0 = blk.sq.start + run.c0 * kC,
            steps = blk.sq.len - run.c0 * kC;
  const long long os = (long long)d.HV * d.V;
  uint8_t* keep_tile = smem + 2 * Tiles<KP>::kBytes;
  const int dyw = (d.VP + 63) / 64 * 64;  // columns of dY's image

  // i counts the chunks in the order they are walked; chunk nc - 1 - i
  if (w < kChainWarps) {
    const int wg = w >> 2, half = wg >> 1, lane0 = 32 * (w & 3), v = lane0 + lane, k0 = wg * (KP / 4);
    float S[KP / 4];
    read_state(S, run.from, d.K, d.V, k0, v);
    if (run.map)
#pragma unroll
      for (int j = 0; j < KP / 4; ++j) S[j] = k0 + j == v && v < d.K ? 1.f : 0.f;
    for (int i = 0; i < nc; ++i) {
      const uint32_t ph = i & 1;
      const uint8_t* st = smem + (i & 1) * Tiles<KP>::kBytes;
      const float* gates = reinterpret_cast<const float*>(st + Tiles<KP>::kRec + kRecordGates);
      put_state<KP>(tm, lane0, wg, S);
      signal_tmem(&bars.s[half], lane);
      if (!first_pass) {
        if (i > 0 && !wait_warp(&bars.sent, 1, status, 51)) break;
        keep_state<KP>(keep_tile, d.VP, fresh(v), k0, S);
        signal_tile(&bars.kept, lane);
      }
      if (!wait_warp(&bars.full[i & 1], (i >> 1) & 1, status, 52)) break;
      if (!wait_warp(&bars.x[half], ph, status, 53)) break;
      tc_fence_after();
      float x[16];
#pragma unroll
      for (int b = 0; b < 16; b += 8) {  // dR = e^{G_end - G} X + U (the scores hold the scale)
        uint32_t p[8], q[8];
        float e[8];
        tmem_ld8_nowait(taddr(tm, lane0, C::X + 16 * wg + b), p);
        tmem_ld8_nowait(taddr(tm, lane0, U + 16 * wg + b), q);
        lds8(gates + kC + 16 * wg + b, e);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          fma2(x[b + j], x[b + j + 1], e[j], e[j + 1], __uint_as_float(p[j]), __uint_as_float(p[j + 1]),
               __uint_as_float(q[j]), __uint_as_float(q[j + 1]));
      }
      put_split(taddr(tm, lane0, C::X + 16 * wg), x);
      signal_tmem(&bars.y[half], lane);
      if (!wait_warp(&bars.r[half], ph, status, 54)) break;
      tc_fence_after();
      ld16(taddr(tm, lane0, C::R + 16 * wg), x);  // dY
      {
#pragma unroll
        for (int b = 0; b < 16; b += 8) {  // dX = -beta e^G dY
          float e[8], be[8];
          lds8(gates + 16 * wg + b, e);
          lds8(gates + 2 * kC + 16 * wg + b, be);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            mul2(e[j], e[j + 1], e[j], e[j + 1], -be[j], -be[j + 1]);
            mul2(e[j], e[j + 1], e[j], e[j + 1], x[b + j], x[b + j + 1]);
          }
          put_split8(taddr(tm, lane0, C::R + 16 * wg), b, e);
        }
      }
      signal_tmem(&bars.rp[half], lane);
      const float keep = gates[kC - 1];
      if (!first_pass) {  // dY and dV = beta dY on their way out
        if (!wait_warp(&bars.sent, 0, status, 56)) break;
        if (i > 0 && !wait_warp(&bars.dv_sent, ph ^ 1, status, 57)) break;
        const int vf = fresh(v);
        uint8_t* yt = keep_tile + 16 * wg * 128;
        unsigned short* tile = reinterpret_cast<unsigned short*>(keep_tile + kKeep) + 16 * wg * 128 + vf;
#pragma unroll
        for (int b = 0; b < 16; b += 8) {
          float be[8];
          lds8(gates + 2 * kC + 16 * wg + b, be);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const uint32_t y = pack(x[b + j], x[b + j + 1]);
            if (vf < dyw) {
              *reinterpret_cast<unsigned short*>(yt + v_off(b + j, vf)) = (unsigned short)y;
              *reinterpret_cast<unsigned short*>(yt + v_off(b + j + 1, vf)) = (unsigned short)(y >> 16);
            }
            float a0, a1;
            mul2(a0, a1, be[j], be[j + 1], x[b + j], x[b + j + 1]);
            const uint32_t z = pack(a0, a1);
            tile[(b + j) * 128] = (unsigned short)z;
            tile[(b + j + 1) * 128] = (unsigned short)(z >> 16);
          }
        }
        signal_tile(&bars.kept, lane);
        if (lane == 0) mbar_arrive(&bars.dv);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty[i & 1]);
      if (!wait_warp(&bars.d[half], ph, status, 55)) break;
      tc_fence_after();
      update_state<KP>(tm, lane0, k0, keep, S);
    }
    if (run.to) write_state(run.to, S, run.rows, run.columns, k0, v);
  } else if (w < kMmaWarp) {
    const int lane0 = 32 * (w & 3), v = lane0 + lane, tid = threadIdx.x - 32 * kChainWarps;
    for (int i = 0; i < nc; ++i) {
      const uint32_t ph = i & 1;
      const int c = nc - 1 - i;
      const uint8_t* st = smem + (i & 1) * Tiles<KP>::kBytes;
      const float* gates = reinterpret_cast<const float*>(st + Tiles<KP>::kRec + kRecordGates);
      if (!wait_warp(&bars.full[i & 1], (i >> 1) & 1, status, 61)) break;
      if (i > 0 && !wait_warp(&bars.d[0], ph ^ 1, status, 62)) break;  // F of the chunk before has been read
      tc_fence_after();
#pragma unroll 2
      for (int b = 0; b < 8; ++b) {  // F = scale e^G dO^T
        float x[8];
        lds8(gates + 4 * kC + 8 * b, x);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] *= __bfloat162float(*reinterpret_cast<const bf16*>(st + Tiles<KP>::kKQ + v_off(8 * b + j, v)));
        put_split8(taddr(tm, lane0, F + 16 * (b >> 1)), 8 * (b & 1), x);
      }
      signal_tmem(&bars.f, lane);
      if (lane == 0) mbar_arrive(&bars.empty[i & 1]);
      if (first_pass) continue;
      if (!wait_warp(&bars.dv, ph, status, 64)) break;
      store_tile(keep_tile + kKeep, dv + ((long long)(step0 + c * kC) * d.HV + blk.hv) * d.V, os,
                 min(kC, steps - c * kC), d.V, d.ovec, tid);
      signal_read(&bars.dv_sent, lane);
    }
  } else if (w == kMmaWarp) {
    constexpr uint32_t n64 = idesc_bf16(128, 64, false, false), n32 = idesc_bf16(128, 32, false, false),
                       nk = idesc_bf16(128, KP, false, true), n64k = idesc_bf16(128, 64, false, true);
    constexpr int kH = KP / 32;
    for (int i = 0; i < nc; ++i) {
      const uint32_t ph = i & 1;
      const uint8_t* st = smem + (i & 1) * Tiles<KP>::kBytes;
      const uint8_t* rc = st + Tiles<KP>::kRec;
      const uint64_t kd = kdesc(st, 128, 0), kd1 = kdesc(st + 32 * 128, 128, 0);
      const uint64_t km = sdesc_sw128(smem_u32(st), 128 * 128, 1024), qm = sdesc_sw128(smem_u32(st) + kC * 128, 128 * 128, 1024),
                     km1 = sdesc_sw128(smem_u32(st) + 128 * 128, 128 * 128, 1024);
      const uint64_t od = sdesc_sw128(smem_u32(st) + Tiles<KP>::kKQ, kC * 128, 1024);  // dO^T: [step][v]
      if (!wait_warp(&bars.full[i & 1], (i >> 1) & 1, status, 71)) break;
      tc_fence_after();
      if (elect_one()) {  // U^T = dO^T P: the steps of 16-block kb reach the steps t <= 16 kb + 15
#pragma unroll
        for (int kb = 3; kb >= 0; --kb) {
          const uint32_t id = idesc_bf16(128, 16 * (kb + 1), true, true);
          mma_bf16(tm + U, od + mdesc_step(16 * kb), mdesc(rc + 2 * 8192, kC, 16 * kb), id, kb < 3);
          mma_bf16(tm + U, od + mdesc_step(16 * kb), mdesc(rc + 3 * 8192, kC, 16 * kb), id, true);
        }
      }
      __syncwarp();
      // the second half leads: dY goes from the last step back
      if (!wait_warp(&bars.s[1], ph, status, 72)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kb = kH; kb < 2 * kH; ++kb) {
          mma_ts(tm + C::X, tm + C::Sh + 8 * kb, kd + kdesc_step(128, 16 * kb), n64, kb > kH);
          mma_ts(tm + C::X, tm + C::Sl + 8 * kb, kd + kdesc_step(128, 16 * kb), n64, true);
        }
      }
      __syncwarp();
      if (!wait_warp(&bars.s[0], ph, status, 78)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int h = 1; h >= 0; --h) {
#pragma unroll
          for (int kb = 0; kb < kH; ++kb) {
            mma_ts(tm + C::X + 32 * h, tm + C::Sh + 8 * kb, (h ? kd1 : kd) + kdesc_step(128, 16 * kb), n32, true);
            mma_ts(tm + C::X + 32 * h, tm + C::Sl + 8 * kb, (h ? kd1 : kd) + kdesc_step(128, 16 * kb), n32, true);
          }
          mma_commit(&bars.x[h]);
        }
      }
      __syncwarp();
      // dY^T = dR^T T: the steps of 16-block kb reach the steps t <= 16 kb + 15
#pragma unroll
      for (int h = 1; h >= 0; --h) {
        if (!wait_warp(&bars.y[h], ph, status, 74)) goto end;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kb = 2 * h + 1; kb >= 2 * h; --kb) {
            const uint32_t id = idesc_bf16(128, 16 * (kb + 1), false, true);
            const uint32_t yh = tm + pair_col(C::X, kb, false), yl = tm + pair_col(C::X, kb, true);
            const uint64_t th = mdesc(rc, kC, 16 * kb), tl = mdesc(rc + 8192, kC, 16 * kb);
            mma_ts(tm + C::R, yh, th, id, kb < 3);
            mma_ts(tm + C::R, yl, th, id, true);
            mma_ts(tm + C::R, yh, tl, id, true);
          }
          mma_commit(&bars.r[h]);
        }
        __syncwarp();
      }
      if (!wait_warp(&bars.f, ph, status, 73)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          mma_ts(tm + C::D, tm + pair_col(F, kb, false), qm + mdesc_step(16 * kb), nk, kb > 0);
          mma_ts(tm + C::D, tm + pair_col(F, kb, true), qm + mdesc_step(16 * kb), nk, true);
        }
      }
      __syncwarp();
      if (!wait_warp(&bars.rp[1], ph, status, 75)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kb = 2; kb < 4; ++kb) {
          mma_ts(tm + C::D, tm + pair_col(C::R, kb, false), km + mdesc_step(16 * kb), nk, true);
          mma_ts(tm + C::D, tm + pair_col(C::R, kb, true), km + mdesc_step(16 * kb), nk, true);
        }
      }
      __syncwarp();
      if (!wait_warp(&bars.rp[0], ph, status, 79)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          // (64 keys are one atom of the tile, which is not cut: all of it before the first half's signal)
          if (KP == 128 || h == 1) {
            const int at = KP == 128 ? h : 0;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              mma_ts(tm + C::D + 64 * at, tm + pair_col(C::R, kb, false), (at ? km1 : km) + mdesc_step(16 * kb), n64k, true);
              mma_ts(tm + C::D + 64 * at, tm + pair_col(C::R, kb, true), (at ? km1 : km) + mdesc_step(16 * kb), n64k, true);
            }
          }
          mma_commit(&bars.d[h]);
        }
        mma_commit(&bars.empty[i & 1]);
      }
      __syncwarp();
    }
  end:
    if (elect_one()) mma_commit(&bars.done);
    __syncwarp();
    wait_warp(&bars.done, 0, status, 76);
  } else if (w == kSendWarp) {
    if (!first_pass && nc > 0) {
      const size_t item = (size_t)(chunk0 + nc - 1) * d.HV + blk.hv;
      send_kept(bars, keep_tile, reinterpret_cast<uint8_t*>(dSout + item * d.VP * KP), (size_t)d.VP * KP * 2,
                (uint32_t)(d.VP * KP * 2), reinterpret_cast<uint8_t*>(dYout + item * dyw * kC), (size_t)dyw * kC * 2,
                (uint32_t)(dyw * kC * 2), -(long long)d.HV, nc, lane, status);
    }
  } else {
    const int tid = threadIdx.x - 32 * kLoadWarp0;
    Loader<KP> ld{d, in, maps, run.map ? nullptr : dout, os, d.ovec, true, blk.hk, blk.hv, &bars.tail, 0};
    int loaded = -1;
    for (int i = 0; i < nc; ++i) {
      const int c = nc - 1 - i;
      if (i >= 2 && !wait_warp(&bars.empty[i & 1], ((i >> 1) & 1) ^ 1, status, 81)) break;
      const bool ok = ld(smem + (i & 1) * Tiles<KP>::kBytes, &bars.full[i & 1],
                         records + ((size_t)(chunk0 + c) * d.HV + blk.hv) * kRecordBytes, step0 + c * kC,
                         min(kC, steps - c * kC), tid, status);
      loaded = i;
      if (!ok) break;
    }
    for (int i = max(loaded - 1, 0); i <= loaded; ++i) wait_warp(&bars.full[i & 1], (i >> 1) & 1, status, 82);
  }
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tm, kTmemCols);
  }
}

template <typename F>
cudaError_t allow_smem(F* f, uint32_t bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

cudaError_t make_maps(const Dims& d, const In& in, const bf16* v, long long vstride, bool vvec, Maps* m) {
  const uint64_t steps = d.packed ? (uint64_t)d.T : (uint64_t)d.N * d.T;
  cudaError_t e = cudaSuccess;
  if (d.kvec) e = make_tmap_heads_bf16(&m->k, in.k, d.K, d.H, steps, d.ks);
  if (e == cudaSuccess && d.qvec) e = make_tmap_heads_bf16(&m->q, in.q, d.K, d.H, steps, d.qs);
  if (e == cudaSuccess && vvec) e = make_tmap_heads_bf16(&m->v, v, d.V, d.HV, steps, vstride);
  return e;
}

// S_in of the runs of a split scan: S_in of run 1 is there (the first run's result), S_in of run i + 1 is M_i S_in_i + B_i
// in the place of B_i.  A block per (sequence, value head) and 16 columns; a thread two columns of every 32nd row.  fp32; the
// next map's copy is in flight while a product is computed.  16 heads of 128 x 128 at 16384 steps: 28.5 us, bound by the
// latency of its steps (33 us with four neighbouring rows a thread, whose reads meet half of the banks; 31 us with the keys
// summed by two halves of twice the threads).
constexpr int kMapPitch = 132, kJoinThreads = 256;
template <int KP>
__global__ void __launch_bounds__(kJoinThreads) k_delta_join(Split sp, int K, int V) {
  extern __shared__ __align__(16) float sm[];  // two maps [KP][kMapPitch], the state's columns [KP][16]
  float* cols = sm + 2 * KP * kMapPitch;
  const int tid = threadIdx.x, r0 = tid >> 3, c0 = 2 * (tid & 7), v0 = blockIdx.y * 16 + c0;
  float* st = sp.states + (size_t)blockIdx.x * (sp.parts - 1) * K * V;
  const float* maps = sp.maps + (size_t)blockIdx.x * (sp.parts - 2) * KP * KP;
  const auto fetch = [&](int i) {
    const float* m = maps + (size_t)(i - 1) * KP * KP;
    const uint32_t dst = su32(sm + (i & 1) * KP * kMapPitch);
    for (int j = tid; j < KP * KP / 4; j += kJoinThreads) {
      const int r = j / (KP / 4), c = 4 * (j - r * (KP / 4));
      cp16(dst + 4u * (uint32_t)(r * kMapPitch + c), m + r * KP + c, true);
    }
    cp_commit();
  };
  const auto mine = [&](const float* p, float (&x)[4][2]) {  // this thread's part of a state
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) x[a][b] = r0 + 32 * a < K && v0 + b < V ? p[(size_t)(r0 + 32 * a) * V + v0 + b] : 0.f;
  };
  float x[4][2];
  fetch(1);
  mine(st, x);
  for (int i = 1; i < sp.parts - 1; ++i) {
    float* out = st + (size_t)i * K * V;
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (32 * a < KP) *reinterpret_cast<float2*>(cols + (r0 + 32 * a) * 16 + c0) = make_float2(x[a][0], x[a][1]);
    mine(out, x);
    if (i + 1 < sp.parts - 1)
      fetch(i + 1);
    else
      cp_commit();
    cp_wait<1>();
    __syncthreads();
    {
      const float* m = sm + (i & 1) * KP * kMapPitch + r0 * kMapPitch;
#pragma unroll 4
      for (int k = 0; k < KP; k += 4) {
        float2 s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = *reinterpret_cast<const float2*>(cols + (k + e) * 16 + c0);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          if (32 * a >= KP) break;
          const float4 y = *reinterpret_cast<const float4*>(m + 32 * a * kMapPitch + k);
          const float ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) fma2(x[a][0], x[a][1], ya[e], ya[e], s[e].x, s[e].y, x[a][0], x[a][1]);
        }
      }
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          if (r0 + 32 * a < K && v0 + b < V) out[(size_t)(r0 + 32 * a) * V + v0 + b] = x[a][b];
    }
    __syncthreads();
  }
}

template <int KP>
cudaError_t join(const Dims& d, const Split& split, cudaStream_t st) {
  if (split.parts <= 2) return cudaSuccess;
  const uint32_t smem = 4 * (uint32_t)(2 * KP * kMapPitch + 16 * KP);
  const cudaError_t e = allow_smem(k_delta_join<KP>, smem);
  if (e != cudaSuccess) return e;
  SSD_LAUNCH("k_delta_join", st,
             k_delta_join<KP><<<dim3((unsigned)(d.N * d.HV), (unsigned)((d.V + 15) / 16)), kJoinThreads, smem, st>>>(split, d.K, d.V));
  return cudaGetLastError();
}

template <int KP>
cudaError_t run_scan(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const Split& split, bf16* o,
                     float* s_final, bf16* S, bf16* R, int* status, cudaStream_t st) {
  Maps maps = {};
  cudaError_t e = make_maps(d, in, in.v, d.vs, d.vvec, &maps);
  if (e == cudaSuccess) e = allow_smem(k_delta_scan<KP>, scan_smem<KP>());
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)(d.N * d.HV);
  if (split.parts > 1) {
    SSD_LAUNCH("k_delta_maps", st,
               k_delta_scan<KP><<<units * (2 * split.parts - 3), kThreads, scan_smem<KP>(), st>>>(
                   d, tb, in, maps, records, split, true, nullptr, nullptr, nullptr, nullptr, status));
    if ((e = join<KP>(d, split, st)) != cudaSuccess) return e;
  }
  SSD_LAUNCH("k_delta_scan", st,
             k_delta_scan<KP><<<units * split.parts, kThreads, scan_smem<KP>(), st>>>(
                 d, tb, in, maps, records, split, false, o, s_final, S, R, status));
  return cudaGetLastError();
}
template <int KP>
cudaError_t run_rev(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const Split& split,
                    const bf16* dout, const float* ds_final, bf16* dv, float* ds0, bf16* dS, bf16* dY, int* status,
                    cudaStream_t st) {
  Maps maps = {};
  cudaError_t e = make_maps(d, in, dout, (long long)d.HV * d.V, d.ovec, &maps);
  if (e == cudaSuccess) e = allow_smem(k_delta_rev<KP>, scan_smem<KP>());
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)(d.N * d.HV);
  if (split.parts > 1) {
    SSD_LAUNCH("k_delta_rev_maps", st,
               k_delta_rev<KP><<<units * (2 * split.parts - 3), kThreads, scan_smem<KP>(), st>>>(
                   d, tb, in, maps, records, split, true, dout, ds_final, nullptr, nullptr, nullptr, nullptr, status));
    if ((e = join<KP>(d, split, st)) != cudaSuccess) return e;
  }
  SSD_LAUNCH("k_delta_rev", st,
             k_delta_rev<KP><<<units * split.parts, kThreads, scan_smem<KP>(), st>>>(
                 d, tb, in, maps, records, split, false, dout, ds_final, dv, ds0, dS, dY, status));
  return cudaGetLastError();
}

}  // namespace

// Runs of a scan, by the number of chunk steps that its launches take one after another: a block an SM, 152 of
// them; a step of the first pass (no o) is about three quarters of one with o, and the two further launches cost about
// eight.  16 heads of 256 chunks: 256 steps in one run, 80 in nine.  A packed batch is taken at its mean length.
int scan_parts(const Dims& d) {
  const long long units = (long long)d.N * d.HV, nc = d.nc / d.N;
  const auto waves = [](long long blocks) { return (blocks + 151) / 152; };
  int best = 1;
  double least = 0.8 * (double)(waves(units) * nc);  // a split has to be worth it
  for (int s = 2; s <= 16 && units * s <= 2 * 152; ++s) {
    const long long per = (nc + s - 1) / s;
    const double t = 0.75 * (double)(waves(units * (2 * s - 3)) * per) + (double)(waves(units * s) * per) + 8.0;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

cudaError_t forward_scan(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const Split& split,
                         bf16* o, float* s_final, bf16* S, bf16* R, int* status, cudaStream_t st) {
  return d.KP == 64 ? run_scan<64>(d, tb, in, records, split, o, s_final, S, R, status, st)
                    : run_scan<128>(d, tb, in, records, split, o, s_final, S, R, status, st);
}
cudaError_t reverse_scan(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const Split& split,
                         const bf16* dout, const float* ds_final, bf16* dv, float* ds0, bf16* dS, bf16* dY, int* status,
                         cudaStream_t st) {
  return d.KP == 64 ? run_rev<64>(d, tb, in, records, split, dout, ds_final, dv, ds0, dS, dY, status, st)
                    : run_rev<128>(d, tb, in, records, split, dout, ds_final, dv, ds0, dS, dY, status, st);
}

}  // namespace delta
}  // namespace ssd
