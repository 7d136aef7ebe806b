// dQ, dK, dbeta and dg of the chunked delta rule, every (chunk, query/key head) by itself, on tcgen05.  With S entering
// the chunk, dS' the gradient of the state leaving it, E_t = e^{G_end - G_t}, D_ij = e^{G_i - G_j} (j <= i):
//     B1_ij = scale D_ij (dO R^T)_ij  (j <= i)          the gradient of q_i . k_j
//     B2_ij = -D_ij (dY R^T)_ij       (j < i)           the gradient of beta_i k_i . k_j, over beta_i
//     dQ    = scale e^G dO S^T + B1 K
//     H     = B2 K - e^G dY S^T,        dK = beta H + dK',    dK' = E R dS'^T + B1^T Q + (beta B2)^T K
//     dbeta = k_t . H_t + dY_t . V_t
// and the gradient of G without any further product: every term of the loss that holds e^{G_i} or D_ij holds q_i, k_i or
// k_j once, so
//     dG_t = q_t . dQ_t + beta_t k_t . H_t - k_t . dK'_t,     dG_end += sum_t E_t k_t . (R dS'^T)_t + e^{G_end} <dS', S>
// and dg is its sum from the right.
//
// Results are transposed (a TMEM lane is a key): six groups of MMAs a value head, the two that read S and the two that
// read [dO; dY] stacked on 128 rows.  The decays never touch an operand but B1, B2: everything else is scaled in fp32
// where it leaves tensor memory.  What a head reads (144 KB for K = V = 128) comes by TMA and bulk copies while the head
// before is in its second half, S and dS' last: the scores do not wait for them.  8192 chunks and heads:
// 268 us, 5.0 TB/s (1.34 GB); the elementwise work between the products bounds it, at 1.3 times the time of the traffic
// alone.
//
// Twenty-four warps: 0-15 the elementwise work, four a lane quadrant (quarters of the columns); 16 the MMAs; 17-18 copies;
// 19-22 the two sums that need no product (dY . V by rows, <dS', S>); 23 dbeta and dg from all sums.  The two sums hold the
// tiles longer than the MMAs do, and the next head's copies with them: fused operations on bf16 pairs took 277 us,
// fp32 ones after a conversion 283, mma.sync (of which the diagonal is wanted) 293, each before the scores stopped waiting
// for S and dS'.
#include "delta_tc.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kWorkWarps = 16, kSumWarps = 4, kMmaWarp = kWorkWarps, kLoadWarp0 = kMmaWarp + 1,
              kSumWarp0 = kLoadWarp0 + kLoadWarps,  // (the sums read no tensor memory: any warps will do)
              kGateWarp = kSumWarp0 + kSumWarps;
constexpr int kThreads = 32 * (kGateWarp + 1);
constexpr int kWorkBar = 1;

// Shared memory.  QK: [Q; K] rows of the head; OY: [dO; dY] rows; R^T, S^T, dS'^T images; B: [B1; B2] rows and beta B2,
// each rounded to bf16, and what that rounding left; Out: dQ rows on their way out (dK's
// leave through B).
constexpr uint32_t kQK = 32768, kOY = 32768, kRt = 16384, kSt = 32768, kB = 16384, kBb = 8192, kOutT = 16384;
constexpr uint32_t oOY = kQK, oR = oOY + kOY, oS = oR + kRt, oD = oS + kSt, oB = oD + kSt, oBl = oB + kB, oBb = oBl + kB,
                   oBbl = oBb + kBb, oOut = oBbl + kBb, oGates = oOut + kOutT, kSmem = oGates + 2 * kGateRows * kC * 4 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of a block");

// Columns of tensor memory: the scores [dO; dY] R^T, and over them, once they have been read, the scores' part of dK';
// dS' 's product; S's two products; [B1; B2] K; dQ and dK summed over the value heads so far.
constexpr int cM = 0, cD = 0, cZ3 = 64, cZ = 128, cW = 256, cSum = 384;
constexpr uint32_t kTmemCols = 512;

struct Bars {
  uint64_t qk, qk_free, full, states, empty, tail, m, z, b, w, dk, free, sums, sums_read, done;
};
struct Maps {
  CUtensorMap k, q, dout;
};

// The value heads of this block's (chunk, query/key head) units, one after another.
struct Work {
  const Dims& d;
  const Table& tb;
  int unit, gi, hk, c;
  Chunk ch;
  int step = 0, qkn = 0;  // value heads and units so far
  __device__ Work(const Dims& dd, const Table& t) : d(dd), tb(t), unit(blockIdx.x), gi(0) { find(); }
  __device__ void find() {  // the next unit that is a chunk of some sequence
    const int units = d.nc * d.H;
    for (; unit < units; unit += gridDim.x) {
      c = unit / d.H;
      hk = unit - c * d.H;
      ch = chunk_of(d, tb, c);
      if (ch.rows > 0) return;
    }
    unit = -1;
  }
  __device__ bool more() const { return unit >= 0; }
  __device__ bool last() const { return gi + 1 == d.G; }
  __device__ int hv() const { return hk * d.G + gi; }
  __device__ size_t item() const { return (size_t)c * d.HV + hv(); }
  __device__ void next() {
    ++step;
    if (++gi == d.G) {
      gi = 0;
      ++qkn;
      unit += gridDim.x;
      find();
    }
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// a . b + x: bf16 pairs multiplied into fp32, without a conversion of their own.
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float x) {
  const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n.reg .b16 a, b, c, d;\nmov.b32 {a, b}, %1;\nmov.b32 {c, d}, %2;\n"
        "fma.rn.f32.bf16 %0, a, c, %0;\nfma.rn.f32.bf16 %0, b, d, %0;\n}"
        : "+f"(x)
        : "r"(p[i]), "r"(q[i]));
  return x;
}

// x[i] summed over the warp's lanes; lane l gets the sum of x[l % 8].
__device__ __forceinline__ float lane_sums(float (&x)[8], int lane) {
#pragma unroll
  for (int o = 4; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  x[0] += __shfl_xor_sync(0xffffffffu, x[0], 8);
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}

__device__ __forceinline__ void put_gate(void* p, size_t i, float x, bool is_bf16) {
  if (is_bf16)
    static_cast<bf16*>(p)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(p)[i] = x;
}

// The [64 steps][128 keys] tile to rows of dq or dk.
__device__ __forceinline__ void store_rows(const bf16* tile, bf16* dst, long long stride, int rows, int K, int tid) {
  if (K % 8 == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 4) + 32 * i, c = 8 * (tid & 15);
      if (r < rows && c < K)
        *reinterpret_cast<uint4*>(dst + (long long)r * stride + c) = *reinterpret_cast<const uint4*>(tile + r * 128 + c);
    }
  } else {
    for (int r = tid >> 7; r < rows; r += 4)
      if ((tid & 127) < K) dst[(long long)r * stride + (tid & 127)] = tile[r * 128 + (tid & 127)];
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    k_delta_grads(Dims d, Table tb, In in, const __grid_constant__ Maps maps, const uint8_t* records, const bf16* dout,
                  const bf16* Sst, const bf16* Rst, const bf16* dSst, const bf16* dYst, GradOut out, int* status) {
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tslot;
  __shared__ float s_yv[2][kC], s_ss[2][kSumWarps], s_a[2][4][kC], s_h[2][4][kC], s_e[2][kWorkWarps];
  uint8_t* smem = aligned_smem(raw);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(&bars.qk, kLoadWarps + 1);
    mbar_init(&bars.qk_free, 1 + kWorkWarps);
    mbar_init(&bars.full, kLoadWarps + 1);
    mbar_init(&bars.states, 1);
    mbar_init(&bars.empty, 1 + kSumWarps + kWorkWarps + 1);
    mbar_init(&bars.tail, kLoadWarps + 1);
    mbar_init(&bars.m, 1);
    mbar_init(&bars.z, 1);
    mbar_init(&bars.b, kWorkWarps);
    mbar_init(&bars.w, 1);
    mbar_init(&bars.dk, 1);
    mbar_init(&bars.free, kWorkWarps);
    mbar_init(&bars.sums, kWorkWarps + kSumWarps);
    mbar_init(&bars.sums_read, 1);
    mbar_init(&bars.done, 1);
    mbar_init_fence();
  }
  if (w == kMmaWarp) tmem_alloc(&tslot, kTmemCols);
  if (d.KP == 64) {  // the key tiles' second atoms, which no copy writes
    for (int i = threadIdx.x; i < 1024; i += kThreads) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(smem + 16384)[i] = z;
      reinterpret_cast<uint4*>(smem + oS + 16384)[i] = z;
      reinterpret_cast<uint4*>(smem + oD + 16384)[i] = z;
    }
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tslot;
  const uint32_t satom = d.KP == 64 ? 16384u : (uint32_t)d.VP * 128u;  // from one 64-key atom of S^T to the next
  Work wk(d, tb);

  if (w < kWorkWarps) {
    const int lane0 = 32 * (w & 3), l = lane0 + lane, wg = w >> 2, tid = threadIdx.x;
    const int i = l & 63;             // the scores' row
    const bool is_y = (w & 3) >= 2;   // lanes 64 .. 127 hold dY's
    bf16 *tq = reinterpret_cast<bf16*>(smem + oOut), *tk = reinterpret_cast<bf16*>(smem + oB);
    for (; wk.more(); wk.next()) {
      const uint32_t ph = wk.step & 1;
      const float* gt = reinterpret_cast<const float*>(smem + oGates) + ph * kGateRows * kC;
      const float *eg = gt, *be = gt + 2 * kC;
      bool ok = wait_warp(&bars.full, ph, status, 101);
      // (an arrival here keeps the copies within one phase of this wait)
      if (lane == 0) mbar_arrive(&bars.empty);
      ok = ok && wait_warp(&bars.m, ph, status, 102);
      tc_fence_after();
      {  // B1, B2, beta B2
        float x[16];
        if (16 * wg <= (lane0 & 63) + 31 && ok) {
          float gj[16];
          lds16(gt + 3 * kC + 16 * wg, gj);
          const float gi = gt[3 * kC + i], f = is_y ? -1.f : in.scale;
          const int top = is_y ? i - 1 : i;  // the last column below the diagonal (dY) or on it (dO)
          ld16(taddr(tm, lane0, cM + 16 * wg), x);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float dec;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(dec) : "f"(gi - gj[e]));
            x[e] = 16 * wg + e <= top ? f * x[e] * dec : 0.f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        const auto put = [&](uint32_t hi, uint32_t lo, int r) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t p[4], q[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) split(x[8 * e + 2 * n], x[8 * e + 2 * n + 1], p[n], q[n]);
            *reinterpret_cast<uint4*>(smem + hi + sw128_chunk(r, 2 * wg + e)) = make_uint4(p[0], p[1], p[2], p[3]);
            *reinterpret_cast<uint4*>(smem + lo + sw128_chunk(r, 2 * wg + e)) = make_uint4(q[0], q[1], q[2], q[3]);
          }
        };
        put(oB, oBl, l);
        if (is_y) {
          const float bi = be[i];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= bi;
          put(oBb, oBbl, i);
        }
        fence_proxy_async();
        signal_read(&bars.b, lane);
      }
      ok = ok && wait_warp(&bars.qk, wk.qkn & 1, status, 106) && wait_warp(&bars.z, ph, status, 103) &&
           wait_warp(&bars.w, ph, status, 104);
      tc_fence_after();
      const uint8_t* qk = smem + (l >> 6) * 16384 + 2 * (l & 7);
      // eight steps of dQ or dK: added to the sum of the value heads before, and kept there or sent out
      const auto emit = [&](bf16* tile, int col, int t0, float(&x)[8]) {
        uint32_t u[8];
        if (wk.gi > 0) {
          tmem_ld8_nowait(taddr(tm, lane0, col), u);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += __uint_as_float(u[e]);
        }
        if (wk.last()) {
#pragma unroll
          for (int e = 0; e < 8; ++e) tile[(t0 + e) * 128 + l] = __float2bfloat16_rn(x[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(x[e]);
          st8u(taddr(tm, lane0, col), u);
          tmem_wait_st();
        }
      };
      float e_all = 0.f;  // this key's share of sum_t E_t k_t.(R dS'^T)_t
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int t0 = 16 * wg + 8 * b;
        float sa[8], sh[8], g[8];  // this key's shares of q.dQ - k.dK' and k.H of eight steps
        uint32_t z[8], s[8];
        tmem_ld8_nowait(taddr(tm, lane0, cZ + t0), z);
        tmem_ld8_nowait(taddr(tm, lane0, cW + t0), s);
        lds8(gt + 4 * kC + t0, g);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sa[e] = __bfloat162float(*reinterpret_cast<const bf16*>(qk + sw128_chunk(t0 + e, (l & 63) >> 3)));
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          fma2(g[e], g[e + 1], g[e], g[e + 1], __uint_as_float(z[e]), __uint_as_float(z[e + 1]), __uint_as_float(s[e]),
               __uint_as_float(s[e + 1]));
          mul2(sa[e], sa[e + 1], sa[e], sa[e + 1], g[e], g[e + 1]);
        }
        emit(tq, cSum + t0, t0, g);
        tmem_ld8_nowait(taddr(tm, lane0, cZ + 64 + t0), z);
        tmem_ld8_nowait(taddr(tm, lane0, cW + 64 + t0), s);
        lds8(eg + t0, g);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e += 2)  // H
          fma2(sh[e], sh[e + 1], -g[e], -g[e + 1], __uint_as_float(z[e]), __uint_as_float(z[e + 1]), __uint_as_float(s[e]),
               __uint_as_float(s[e + 1]));
        if (b == 0) {
          ok = wait_warp(&bars.dk, ph, status, 107) && ok;
          tc_fence_after();
        }
        tmem_ld8_nowait(taddr(tm, lane0, cZ3 + t0), z);
        tmem_ld8_nowait(taddr(tm, lane0, cD + t0), s);
        lds8(gt + kC + t0, g);
        tmem_wait_ld();
        if (b == 1) signal_read(&bars.free, lane);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float k0 = __bfloat162float(*reinterpret_cast<const bf16*>(qk + sw128_chunk(kC + t0 + e, (l & 63) >> 3)));
          const float k1 = __bfloat162float(*reinterpret_cast<const bf16*>(qk + sw128_chunk(kC + t0 + e + 1, (l & 63) >> 3)));
          float r0, r1, m0, m1;
          mul2(r0, r1, g[e], g[e + 1], __uint_as_float(z[e]), __uint_as_float(z[e + 1]));
          fma2(m0, m1, r0, r1, 1.f, 1.f, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          e_all = fmaf(k1, r1, fmaf(k0, r0, e_all));
          fma2(sa[e], sa[e + 1], -k0, -k1, m0, m1, sa[e], sa[e + 1]);
          fma2(g[e], g[e + 1], be[t0 + e], be[t0 + e + 1], sh[e], sh[e + 1], m0, m1);
          mul2(sh[e], sh[e + 1], sh[e], sh[e + 1], k0, k1);
        }
        emit(tk, cSum + 64 + t0, t0, g);
        const float a = lane_sums(sa, lane), h = lane_sums(sh, lane);
        // (the sums of the head before have been read, so that no warp is a phase ahead)
        if (b == 0 && wk.step > 0) ok = wait_warp(&bars.sums_read, ph ^ 1, status, 105) && ok;
        if (lane < 8) {
          s_a[ph][w & 3][t0 + lane] = a;
          s_h[ph][w & 3][t0 + lane] = h;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) e_all += __shfl_xor_sync(0xffffffffu, e_all, o);
      if (lane == 0) s_e[ph][w] = e_all;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.sums);
        if (wk.last()) mbar_arrive(&bars.qk_free);
      }
      if (named_bar_or(kWorkBar, 32 * kWorkWarps, !ok)) break;
      if (wk.last()) {
        const long long stride = (long long)d.H * d.K;
        const size_t at = ((size_t)wk.ch.first * d.H + wk.hk) * d.K;
        store_rows(tq, out.dq + at, stride, wk.ch.rows, d.K, tid);
        store_rows(tk, out.dk + at, stride, wk.ch.rows, d.K, tid);
        named_bar(kWorkBar, 32 * kWorkWarps);  // the tiles have been read: the next head writes B over one
      }
    }
  } else if (w == kMmaWarp) {
    constexpr uint32_t iM = idesc_bf16(128, 64, false, true), iZ = idesc_bf16(128, 128, true, false),
                       iR = idesc_bf16(128, 64, true, true), iW = idesc_bf16(128, 128, true, false);
    const int nv = d.VP / 16;
    for (; wk.more(); wk.next()) {
      const uint32_t ph = wk.step & 1;
      if (!wait_warp(&bars.full, ph, status, 111)) break;
      tc_fence_after();
      const uint64_t oy = kdesc(smem + oOY, 128, 0), rt = mdesc(smem + oR, d.VP, 0);
      const uint64_t sm = sdesc_sw128(smem_u32(smem + oS), satom, 1024), dm = sdesc_sw128(smem_u32(smem + oD), satom, 1024);
      if (wk.step > 0 && !wait_warp(&bars.free, ph ^ 1, status, 112)) break;
      tc_fence_after();
      if (elect_one()) {
        for (int vb = 0; vb < nv; ++vb) mma_bf16(tm + cM, oy + kdesc_step(128, 16 * vb), rt + mdesc_step(16 * vb), iM, vb > 0);
        mma_commit(&bars.m);
      }
      __syncwarp();
      if (!wait_warp(&bars.states, ph, status, 116)) break;
      if (elect_one()) {
        for (int vb = 0; vb < nv; ++vb) mma_bf16(tm + cZ, sm + mdesc_step(16 * vb), oy + kdesc_step(128, 16 * vb), iZ, vb > 0);
        for (int vb = 0; vb < nv; ++vb) mma_bf16(tm + cZ3, dm + mdesc_step(16 * vb), rt + mdesc_step(16 * vb), iR, vb > 0);
        mma_commit(&bars.z);
        mma_commit(&bars.empty);
      }
      __syncwarp();
      if (wk.gi == 0 && !wait_warp(&bars.qk, wk.qkn & 1, status, 113)) break;
      if (!wait_warp(&bars.b, ph, status, 114)) break;
      tc_fence_after();
      const uint64_t qm = sdesc_sw128(smem_u32(smem), 16384, 1024), km = sdesc_sw128(smem_u32(smem) + kC * 128, 16384, 1024);
      const uint64_t bk = kdesc(smem + oB, 128, 0), bkl = kdesc(smem + oBl, 128, 0);
      if (elect_one()) {
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          mma_bf16(tm + cW, km + mdesc_step(16 * jb), bk + kdesc_step(128, 16 * jb), iW, jb > 0);
          mma_bf16(tm + cW, km + mdesc_step(16 * jb), bkl + kdesc_step(128, 16 * jb), iW, true);
        }
        mma_commit(&bars.w);
        // the transposed scores: row block ib has columns j <= 16 ib + 15
#pragma unroll
        for (int ib = 3; ib >= 0; --ib) {
          const uint32_t id = idesc_bf16(128, 16 * (ib + 1), true, true);
          mma_bf16(tm + cD, qm + mdesc_step(16 * ib), mdesc(smem + oB, 128, 16 * ib), id, ib < 3);
          mma_bf16(tm + cD, qm + mdesc_step(16 * ib), mdesc(smem + oBl, 128, 16 * ib), id, true);
          mma_bf16(tm + cD, km + mdesc_step(16 * ib), mdesc(smem + oBb, kC, 16 * ib), id, true);
          mma_bf16(tm + cD, km + mdesc_step(16 * ib), mdesc(smem + oBbl, kC, 16 * ib), id, true);
        }
        mma_commit(&bars.dk);
        if (wk.last()) mma_commit(&bars.qk_free);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&bars.done);
    __syncwarp();
    wait_warp(&bars.done, 0, status, 115);
  } else if (w < kSumWarp0) {
    const int tid = threadIdx.x - 32 * kLoadWarp0;
    uint32_t tails = 0;
    bool ok = true;
    // The copies of a cut chunk have arrived.  Each copy warp arrives here as well, so that a phase cannot end, and the next
    // one neither, before both warps have come to wait for it.
    const auto wait_tail = [&](int code) {
      if (lane == 0) mbar_arrive(&bars.tail);
      return wait_warp(&bars.tail, tails++ & 1, status, code);
    };
    int loaded = -1, units = -1;
    const int na = d.KP / 64, va = (d.VP + 63) / 64;
    for (; wk.more() && ok; wk.next()) {
      const uint32_t ph = wk.step & 1;
      const int first = wk.ch.first, rows = wk.ch.rows;
      const bool cut = rows < kC;
      if (wk.step > 0 && !(ok = wait_warp(&bars.empty, ph ^ 1, status, 123))) break;
      uint64_t* bar = cut ? &bars.tail : &bars.full;
      const size_t item = wk.item();
      if (tid == 0) {
        const uint32_t sb = (uint32_t)d.VP * 128 * na, rb = (uint32_t)d.VP * 128, gb = kGateRows * kC * 4;
        mbar_expect_tx(bar, rb + gb + kC * 128 * va * (1 + (d.ovec ? 1 : 0)));
        if (d.ovec)
          for (int a = 0; a < va; ++a) tma_load_3d(smem + oOY + a * 16384, &maps.dout, 64 * a, wk.hv(), first, bar);
        for (int a = 0; a < va; ++a)
          bulk_load(smem_u32(smem + oOY) + a * 16384 + kC * 128, dYst + item * va * 64 * kC + a * 64 * kC, kC * 128, bar);
        bulk_load(smem_u32(smem + oR), Rst + item * d.VP * kC, rb, bar);
        bulk_load(smem_u32(smem + oGates) + ph * gb, records + item * kRecordBytes + kRecordGates, gb, bar);
        mbar_expect_tx(&bars.states, 2 * sb);
        bulk_load(smem_u32(smem + oS), Sst + item * d.VP * d.KP, sb, &bars.states);
        bulk_load(smem_u32(smem + oD), dSst + item * d.VP * d.KP, sb, &bars.states);
      }
      if (!d.ovec)
        load_elements(smem + oOY, 128, 64 * va, dout + ((long long)first * d.HV + wk.hv()) * d.V, (long long)d.HV * d.V, rows, d.V, tid);
      if (cut) {
        ok = wait_tail(124);
        if (d.ovec) zero_rows(smem + oOY, 128, va, rows, tid);
      }
      fence_proxy_async();
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(&bars.full);
      if (cut && tid == 0) mbar_arrive(&bars.full);
      loaded = wk.step;
      if (wk.gi == 0) {
        if (wk.qkn > 0 && !wait_warp(&bars.qk_free, (wk.qkn & 1) ^ 1, status, 121)) break;
        uint8_t* qt = smem;
        uint64_t* bar = cut ? &bars.tail : &bars.qk;
        if (tid == 0) {
          mbar_expect_tx(bar, kC * 128 * na * ((d.qvec ? 1 : 0) + (d.kvec ? 1 : 0)));
          for (int a = 0; a < na; ++a) {
            if (d.qvec) tma_load_3d(qt + a * 16384, &maps.q, 64 * a, wk.hk, first, bar);
            if (d.kvec) tma_load_3d(qt + a * 16384 + kC * 128, &maps.k, 64 * a, wk.hk, first, bar);
          }
        }
        if (!d.qvec) load_elements(qt, 128, d.KP, in.q + (long long)first * d.qs + (long long)wk.hk * d.K, d.qs, rows, d.K, tid);
        if (!d.kvec) load_elements(qt + kC * 128, 128, d.KP, in.k + (long long)first * d.ks + (long long)wk.hk * d.K, d.ks, rows, d.K, tid);
        if (cut) {
          ok = wait_tail(122) && ok;
          if (d.qvec) zero_rows(qt, 128, na, rows, tid);
          if (d.kvec) zero_rows(qt + kC * 128, 128, na, rows, tid);
        }
        fence_proxy_async();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&bars.qk);
        if (cut && tid == 0) mbar_arrive(&bars.qk);
        units = wk.qkn;
      }
    }
    // no copy is in flight when the block ends
    if (loaded >= 0) {
      wait_warp(&bars.full, loaded & 1, status, 125);
      wait_warp(&bars.states, loaded & 1, status, 127);
    }
    if (units >= 0) wait_warp(&bars.qk, units & 1, status, 126);
  } else if (w < kGateWarp) {
    const int sw = w - kSumWarp0, g = lane >> 2, q4 = lane & 3;
    uint4 v[2][4];  // V, rows 16 sw + g and + 8, pieces of eight columns 4 n + q4: read before the wait
    const auto fetch = [&] {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = 16 * sw + 8 * h + g;
        const bf16* vr = in.v + (long long)(wk.ch.first + t) * d.vs + (long long)wk.hv() * d.V;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int c = 32 * n + 8 * q4;
          v[h][n] = make_uint4(0, 0, 0, 0);
          if (t >= wk.ch.rows || c >= d.V) continue;
          if (d.vvec) {
            v[h][n] = *reinterpret_cast<const uint4*>(vr + c);
          } else {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = pack(c + 2 * e < d.V ? __bfloat162float(vr[c + 2 * e]) : 0.f,
                          c + 2 * e + 1 < d.V ? __bfloat162float(vr[c + 2 * e + 1]) : 0.f);
            v[h][n] = make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
      }
    };
    for (; wk.more(); wk.next()) {
      const uint32_t ph = wk.step & 1;
      fetch();
      bool ok = wait_warp(&bars.full, ph, status, 131);
      const uint32_t oa = smem_u32(smem + oOY) + (kC + 16 * sw + g) * 128;
      float yv[2] = {0.f, 0.f}, ss[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (32 * n >= d.V) break;
        const int j = 4 * n + q4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (8 * j < d.V) yv[h] = dot8(v[h][n], lds128(oa + (n >> 1) * 16384 + h * 1024 + (((j & 7) ^ g) << 4)), yv[h]);
      }
      const uint32_t at = smem_u32(smem) + (uint32_t)(sw * 1024 + lane * 16);
      ok = ok && wait_warp(&bars.states, ph, status, 135);
#pragma unroll 2
      for (int i = sw; i < d.VP * d.KP / 512; i += kSumWarps) {  // a kilobyte of both images
        const uint32_t p = at + (i - sw) * 1024;
#pragma unroll
        for (int h = 0; h < 2; ++h) ss[h] = dot8(lds128(p + 512 * h + oS), lds128(p + 512 * h + oD), ss[h]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.empty);  // (the tiles have been read)
      float y = ss[0] + ss[1];
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) yv[h] += __shfl_xor_sync(0xffffffffu, yv[h], o);
      const float y0 = yv[0], y1 = yv[1];
#pragma unroll
      for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      // (the sums of the head before have been read, so that no warp is a phase ahead)
      if (wk.step > 0) ok = wait_warp(&bars.sums_read, ph ^ 1, status, 132) && ok;
      if (q4 == 0) {
        s_yv[ph][16 * sw + g] = y0;
        s_yv[ph][16 * sw + 8 + g] = y1;
      }
      if (lane == 0) s_ss[ph][sw] = y;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.sums);
      if (!ok) break;
    }
  } else {
    // dbeta, and dG with its sums from the right, once all shares are there: two steps a lane.  The decays' place is free
    // for the head after the next only when this warp has arrived for the next.
    if (lane == 0) mbar_arrive(&bars.empty);
    for (; wk.more(); wk.next()) {
      const uint32_t ph = wk.step & 1;
      const Chunk ch = wk.ch;
      if (!wait_warp(&bars.sums, ph, status, 133) || !wait_warp(&bars.empty, ph, status, 134)) break;
      const float* gt = reinterpret_cast<const float*>(smem + oGates) + ph * kGateRows * kC;
      const float *eg = gt, *be = gt + 2 * kC;
      const int hv = wk.hv();
      float dG[2], db[2], all = lane < kWorkWarps ? s_e[ph][lane] : 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int u = 2 * lane + n;
        const float a0 = (s_a[ph][0][u] + s_a[ph][1][u]) + (s_a[ph][2][u] + s_a[ph][3][u]);
        const float h = (s_h[ph][0][u] + s_h[ph][1][u]) + (s_h[ph][2][u] + s_h[ph][3][u]);
        dG[n] = fmaf(be[u], h, a0);
        db[n] = h + s_yv[ph][u];
      }
      const float ss = (s_ss[ph][0] + s_ss[ph][1]) + (s_ss[ph][2] + s_ss[ph][3]), decay = eg[kC - 1];
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.sums_read);
        mbar_arrive(&bars.empty);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      const float end = fmaf(decay, ss, all);
      float sum = dG[0] + dG[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float z = __shfl_down_sync(0xffffffffu, sum, o);
        if (lane + o < 32) sum += z;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int u = 2 * lane + n;
        if (u >= ch.rows) continue;
        put_gate(out.dbeta, (size_t)(ch.first + u) * d.HV + hv, db[n], d.gate_bf16);
        put_gate(out.dg, (size_t)(ch.first + u) * d.HV + hv, end + (n ? sum - dG[0] : sum), d.gate_bf16);
      }
    }
  }
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tm, kTmemCols);
  }
}

}  // namespace

cudaError_t chunk_grads(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const bf16* dout,
                        const bf16* S, const bf16* R, const bf16* dS, const bf16* dY, const GradOut& out, int* status,
                        cudaStream_t st) {
  const uint64_t steps = d.packed ? (uint64_t)d.T : (uint64_t)d.N * d.T;
  Maps maps = {};
  cudaError_t e = cudaSuccess;
  if (d.kvec) e = make_tmap_heads_bf16(&maps.k, in.k, d.K, d.H, steps, d.ks);
  if (e == cudaSuccess && d.qvec) e = make_tmap_heads_bf16(&maps.q, in.q, d.K, d.H, steps, d.qs);
  if (e == cudaSuccess && d.ovec) e = make_tmap_heads_bf16(&maps.dout, dout, d.V, d.HV, steps, (uint64_t)d.HV * d.V);
  int dev, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_delta_grads, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  const long long units = (long long)d.nc * d.H;
  SSD_LAUNCH("k_delta_grads", st,
             k_delta_grads<<<(unsigned)(units < sms ? units : sms), kThreads, kSmem, st>>>(
                 d, tb, in, maps, records, dout, S, R, dS, dY, out, status));
  return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
