// The gated delta rule with one decay per head, by chunks of 64 steps on the tensor cores: forward, its stash for
// training, and the backward pass.
//
// Per sequence and value head, with state S [K, V] and G the running sum of g inside a chunk:
//     A_ij = beta_i e^{G_i - G_j} k_i.k_j  (j < i),     T = (I + A)^-1
//     Y = beta (V - e^G K S),   R = T Y                 (row t of R is what step t writes along k_t)
//     O = scale (e^G Q S + P R),   P_ij = e^{G_i - G_j} q_i.k_j  (j <= i)
//     S' = e^{G_end} S + K^T (e^{G_end - G} R)
// The chunks of a sequence are independent but for S, so a call is
//     k_delta_prep   every (chunk, query/key head) at once: T, P and the decays of its value heads
//     k_delta_scan   per (sequence, value head) one chunk after another: R, S', O
// and the backward pass, given the S entering each chunk and R,
//     k_delta_rev    per (sequence, value head) in reverse: dR = scale P^T dO + e^{G_end-G} K dS', dY = T^T dR,
//                    dX = -beta e^G dY, dS = e^{G_end} dS' + scale Q^T e^G dO + K^T dX;  dV = beta dY
//     k_delta_grads  every (chunk, query/key head) at once: dQ, dK, dbeta, dg from S, dS', R, dY
//
// The scans hold the state transposed, S^T [V, K]: a warp owns 16 of its rows for the whole sequence, as fp32
// accumulators.  Every product of a chunk then has what the warp computed just before as its left operand, and the
// accumulator layout of one product is the left-operand layout of the next: the chain S -> X -> Y -> R -> S' never
// leaves the registers, and warps do not wait for one another but for the tiles they read.
//
// Precision.  q, k, v, dO are bf16 as given.  What the chain computes in fp32 and has to multiply again (S, Y, T, R)
// enters the tensor cores as two bf16 numbers, high and low, so a product of two such is three products; what is
// dropped is 2^-17 of each factor.  The state therefore keeps fp32 accuracy over any length (relative error about
// 1e-6 to 5e-6), which bf16 operands would not give: a state that is read for thousands of steps would carry 2^-9.
// P is rounded to bf16 (it meets only the bf16 output o, never the state).  The gradients' last products (k_delta_grads)
// take S, dS', R, dY and the two score matrices rounded to bf16: their results are gradients of bf16 inputs.
#include <initializer_list>

#include "delta_common.cuh"
#include "ssd.h"

namespace ssd {
namespace delta {
namespace {

// ---------------------------------------------------------------- packed sequences
// cu_seqlens -> start, length and first chunk of every sequence.  One block.  Bounds that leave the token axis or
// run backwards are pulled in (a running maximum), so no later kernel can leave its buffers whatever the values are.
__global__ void __launch_bounds__(1024) k_delta_table(const int* __restrict__ cu, int N, int T, Table tb) {
  __shared__ int s_max[1024], s_sum[1024];
  __shared__ int carry_end, carry_chunk;
  const int tid = threadIdx.x;
  if (tid == 0) {
    carry_end = min(max(cu[0], 0), T);
    carry_chunk = 0;
  }
  __syncthreads();
  for (int base = 0; base < N; base += 1024) {
    const int n = base + tid;
    s_max[tid] = n < N ? min(max(cu[n + 1], 0), T) : 0;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
      const int x = tid >= o ? s_max[tid - o] : 0;
      __syncthreads();
      s_max[tid] = max(s_max[tid], x);
      __syncthreads();
    }
    const int end = max(s_max[tid], carry_end);
    const int start = tid ? max(s_max[tid - 1], carry_end) : carry_end;
    const int nc = n < N ? (end - start + kC - 1) / kC : 0;
    s_sum[tid] = nc;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
      const int x = tid >= o ? s_sum[tid - o] : 0;
      __syncthreads();
      s_sum[tid] += x;
      __syncthreads();
    }
    if (n < N) {
      tb.start[n] = start;
      tb.len[n] = end - start;
      tb.chunk[n] = carry_chunk + s_sum[tid] - nc;
    }
    __syncthreads();
    if (tid == 1023) {
      carry_end = end;
      carry_chunk += s_sum[tid];
    }
    __syncthreads();
  }
  if (tid == 0) tb.chunk[N] = carry_chunk;
}

// ---------------------------------------------------------------- T, P and the decays of a chunk
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kFP = kC + 4;  // pitch of the fp32 [64][64] tiles

// c[16x16] = a[16 x n] b[n x 16], fp32 tiles in shared memory.  Each factor enters as two tf32 numbers (three
// products; 2^-21 of a factor is dropped): the inverse keeps fp32 accuracy.
__device__ __forceinline__ void mul16(float (&c)[2][4], const float* a, const float* b, int n, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
  for (int k = 0; k < n; k += 8) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[(g + 8 * (i & 1)) * kFP + k + t + 4 * (i >> 1)];
      ah[i] = tf32(x);
      al[i] = tf32(x - __uint_as_float(ah[i]));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = b[(k + t + 4 * i) * kFP + 8 * h + g];
        bh[i] = tf32(x);
        bl[i] = tf32(x - __uint_as_float(bh[i]));
      }
      mma_tf32(c[h], ah, bh[0], bh[1]);
      mma_tf32(c[h], ah, bl[0], bl[1]);
      mma_tf32(c[h], al, bh[0], bh[1]);
    }
  }
}
__device__ __forceinline__ void put16(float* dst, const float (&c)[2][4], float sign, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[(g + 8 * (j >> 1)) * kFP + 8 * h + 2 * t + (j & 1)] = sign * c[h][j];
}

// Four warps per (chunk, query/key head); warp w holds rows 16 w .. 16 w + 15 of K K^T and Q K^T, which the head's
// value heads share, and multiplies them by each head's decays.  (I + A)^-1: the four 16-blocks of the diagonal by
// forward substitution (a lane a column), then twice the block rule  [[a, 0], [c, b]]^-1 = [[a', 0], [-b' c a', b']].
// Substitution and block products stay small for strongly correlated keys, where a series in powers of A would not.
template <int KP>
__global__ void __launch_bounds__(128) k_delta_prep(Dims d, Table tb, In in, Prep pr, int* status) {
  constexpr int kP = KP + 8;
  extern __shared__ __align__(16) unsigned char smem[];
  bf16* Ks = reinterpret_cast<bf16*>(smem);
  bf16* Qs = Ks + kC * kP;
  float* Af = reinterpret_cast<float*>(Qs + kC * kP);
  float* Tf = Af + kC * kFP;
  float* Mf = Tf + kC * kFP;  // [32][kFP]
  __shared__ float s_hi[kC], s_lo[kC], s_beta[kC];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int c = blockIdx.x, hk = blockIdx.y;
  if (c == 0 && hk == 0 && tid == 0) *status = 0;
  const Chunk ch = chunk_of(d, tb, c);
  if (ch.rows == 0) return;
  load_rows(Ks, kP, KP, in.k + (long long)ch.first * d.ks + (long long)hk * d.K, d.ks, ch.rows, d.K, d.kvec, tid, 128);
  load_rows(Qs, kP, KP, in.q + (long long)ch.first * d.qs + (long long)hk * d.K, d.qs, ch.rows, d.K, d.qvec, tid, 128);
  cp_commit();
  for (int i = tid; i < kC * kFP; i += 128) Tf[i] = 0.f;
  cp_wait<0>();
  __syncthreads();
  const int r0 = 16 * w, g4 = lane >> 2, t2 = 2 * (lane & 3);
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
  const uint32_t ka = su32(Ks), qa = su32(Qs);
#pragma unroll
  for (int kb = 0; kb < KP / 16; ++kb) {
    uint32_t ak[4], aq[4];
    ldm4(ak, by_col(ka, kP, r0, 16 * kb, lane));
    ldm4(aq, by_col(qa, kP, r0, 16 * kb, lane));
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      if (jb > w) break;  // above the diagonal
      uint32_t b[4];
      ldm4(b, by_row(ka, kP, 16 * jb, 16 * kb, lane));
      mma(kk[2 * jb], ak, b[0], b[1]);
      mma(kk[2 * jb + 1], ak, b[2], b[3]);
      mma(qk[2 * jb], aq, b[0], b[1]);
      mma(qk[2 * jb + 1], aq, b[2], b[3]);
    }
  }
  for (int gi = 0; gi < d.G; ++gi) {
    const int hv = hk * d.G + gi;
    const size_t item = (size_t)c * d.HV + hv;
    if (w == 0) {  // G of two steps a lane; the sums in fp64, kept as a high and a low fp32 part
      double x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        float v = 0.f, b = 0.f;
        if (t < ch.rows) {
          const size_t at = (size_t)(ch.first + t) * d.HV + hv;
          v = gate(in.g, at, d.gate_bf16);
          b = gate(in.beta, at, d.gate_bf16);
          v = v < kMinG ? kMinG : v;
        }
        x[i] = v;
        s_beta[t] = b;
      }
      double sum = x[0] + x[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const double end = __shfl_sync(0xffffffffu, sum, 31);
      float* gr = pr.gates + item * (kGateRows * kC);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const double gt = i ? sum : sum - x[1];
        const float h = (float)gt, l = (float)(gt - (double)h);
        s_hi[t] = h;
        s_lo[t] = l;
        gr[t] = expf((float)gt);
        gr[kC + t] = expf((float)(end - gt));
        gr[2 * kC + t] = s_beta[t];
        gr[3 * kC + t] = h;
        gr[4 * kC + t] = l;
      }
    }
    __syncthreads();
    uint32_t* P32 = reinterpret_cast<uint32_t*>(pr.P + item * (kC * kC));
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt > 2 * w + 1) break;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = r0 + g4 + 8 * half, j = 8 * nt + t2;
        float a[2], p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float dec = expf((s_hi[i] - s_hi[j + e]) + (s_lo[i] - s_lo[j + e]));
          a[e] = i > j + e ? s_beta[i] * dec * kk[nt][2 * half + e] : 0.f;
          p[e] = i >= j + e ? dec * qk[nt][2 * half + e] : 0.f;
        }
        Af[i * kFP + j] = a[0];
        Af[i * kFP + j + 1] = a[1];
        P32[(i * kC + j) >> 1] = pack(p[0], p[1]);
      }
    }
    __syncwarp();
    if (lane < 16) {  // the diagonal block of this warp, column `lane`
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = fmaf(-Af[(r0 + i) * kFP + r0 + j], x[j], s);
        x[i] = s;
        Tf[(r0 + i) * kFP + r0 + lane] = s;
      }
    }
    __syncthreads();
    float m[2][4];
    if ((w & 1) == 0) {  // rows 16 .. 31 (warp 0) and 48 .. 63 (warp 2): -b' c a'
      const int a0 = 16 * w, b0 = a0 + 16;
      mul16(m, Af + b0 * kFP + a0, Tf + a0 * kFP + a0, 16, lane);
      put16(Mf + w * 8 * kFP, m, 1.f, lane);
      __syncwarp();
      mul16(m, Tf + b0 * kFP + b0, Mf + w * 8 * kFP, 16, lane);
      put16(Tf + b0 * kFP + a0, m, -1.f, lane);
    }
    __syncthreads();
    const int br = 16 * (w >> 1), bc = 16 * (w & 1);  // one 16-block of the 32 x 32 product a warp
    mul16(m, Af + (32 + br) * kFP, Tf + bc, 32, lane);
    put16(Mf + br * kFP + bc, m, 1.f, lane);
    __syncthreads();
    mul16(m, Tf + (32 + br) * kFP + 32, Mf + bc, 32, lane);
    put16(Tf + (32 + br) * kFP + bc, m, -1.f, lane);
    __syncthreads();
    {
      const int i = tid >> 1, j0 = 32 * (tid & 1);
      uint4* dh = reinterpret_cast<uint4*>(pr.Thi + item * (kC * kC) + i * kC + j0);
      uint4* dl = reinterpret_cast<uint4*>(pr.Tlo + item * (kC * kC) + i * kC + j0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          split(Tf[i * kFP + j0 + 8 * q + 2 * e], Tf[i * kFP + j0 + 8 * q + 2 * e + 1], h[e], l[e]);
        dh[q] = make_uint4(h[0], h[1], h[2], h[3]);
        dl[q] = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the scans
// Shared memory of one stage of a scan: K, Q, V (or dO), T high and low, P, the decays.
template <int KP>
struct Stage {
  bf16 *K, *Q, *V, *Th, *Tl, *P;
  float* gates;
  static __host__ __device__ size_t bytes(int nw) {
    return 2 * (size_t)(2 * kC * (KP + 8) + kC * (16 * nw + 8) + 3 * kC * kTP) + sizeof(float) * 3 * kC;
  }
  __device__ Stage(unsigned char* base, int nw) {
    K = reinterpret_cast<bf16*>(base);
    Q = K + kC * (KP + 8);
    V = Q + kC * (KP + 8);
    Th = V + kC * (16 * nw + 8);
    Tl = Th + kC * kTP;
    P = Tl + kC * kTP;
    gates = reinterpret_cast<float*>(P + kC * kTP);
  }
};

// `v`: the tensor whose columns the block's warps own (V forward, dO in reverse), `stride` elements from step to step.
template <int KP>
__device__ __forceinline__ void load_stage(const Stage<KP>& s, const Dims& d, const In& in, const Prep& pr,
                                           const bf16* v, long long stride, bool vvec, int first, int rows, int hk,
                                           int hv, size_t item, int v0, int nw) {
  const int tid = threadIdx.x, nt = blockDim.x;
  load_rows(s.K, KP + 8, KP, in.k + (long long)first * d.ks + (long long)hk * d.K, d.ks, rows, d.K, d.kvec, tid, nt);
  load_rows(s.Q, KP + 8, KP, in.q + (long long)first * d.qs + (long long)hk * d.K, d.qs, rows, d.K, d.qvec, tid, nt);
  load_rows(s.V, 16 * nw + 8, 16 * nw, v + (long long)first * stride + (long long)hv * d.V + v0, stride, rows,
            d.V - v0, vvec, tid, nt);
  load_dense(s.Th, kTP, kC / 8, pr.Thi + item * (kC * kC), kC, tid, nt);
  load_dense(s.Tl, kTP, kC / 8, pr.Tlo + item * (kC * kC), kC, tid, nt);
  load_dense(s.P, kTP, kC / 8, pr.P + item * (kC * kC), kC, tid, nt);
  for (int i = tid; i < 3 * kC / 4; i += nt)
    cp16(su32(s.gates + 4 * i), pr.gates + item * (kGateRows * kC) + 4 * i, true);
}

// The warp's 16 columns of a [64][..] tile in shared memory to rows of a tensor: row r to dst + r * stride.
__device__ __forceinline__ void store_cols(const bf16* tile, int pitch, bf16* dst, long long stride, int rows, int cols,
                                           bool vec, int lane) {
  if (vec) {
    const int c = 8 * (lane & 1);
    if (c < cols)
#pragma unroll
      for (int r = lane >> 1; r < kC; r += 16)
        if (r < rows)
          *reinterpret_cast<uint4*>(dst + (long long)r * stride + c) =
              *reinterpret_cast<const uint4*>(tile + r * pitch + c);
  } else {
    const int c = lane & 15;
    if (c < cols)
      for (int r = lane >> 4; r < rows; r += 2) dst[(long long)r * stride + c] = tile[r * pitch + c];
  }
}

// The transposed accumulators [16 v][64 t] as bf16 into the warp's columns of a [64 t][v] tile.
__device__ __forceinline__ void stage_t(bf16* tile, int pitch, const float (&x)[8][4], int lane) {
#pragma unroll
  for (int tb = 0; tb < 4; ++tb) {
    uint32_t r[4];
    round_a(x[2 * tb], x[2 * tb + 1], r);
    stm4t(by_row(su32(tile), pitch, 16 * tb, 0, lane), r);
  }
}

// The state accumulators [16 v][KP] as bf16 rows of dst (pitch KP), through a warp's own [16][KP + 8] buffer.
template <int KP>
__device__ __forceinline__ void store_state(bf16* buf, bf16* dst, const float (&S)[KP / 8][4], int lane) {
  constexpr int kP = KP + 8;
#pragma unroll
  for (int kb = 0; kb < KP / 16; ++kb) {
    uint32_t r[4];
    round_a(S[2 * kb], S[2 * kb + 1], r);
    stm4(by_col(su32(buf), kP, 0, 16 * kb, lane), r);
  }
  __syncwarp();
#pragma unroll
  for (int i = lane; i < 2 * KP; i += 32) {
    const int r = i / (KP / 8), c = 8 * (i % (KP / 8));
    *reinterpret_cast<uint4*>(dst + (size_t)r * KP + c) = *reinterpret_cast<const uint4*>(buf + r * kP + c);
  }
  __syncwarp();
}

// s [K, V] (fp32, row-major) to and from the accumulators of rows v0 .. v0 + 15 of its transpose.
template <int KP>
__device__ __forceinline__ void read_state(float (&S)[KP / 8][4], const float* s, int K, int V, int v0, int lane) {
#pragma unroll
  for (int nt = 0; nt < KP / 8; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 8 * nt + 2 * (lane & 3) + (j & 1), v = v0 + (lane >> 2) + 8 * (j >> 1);
      S[nt][j] = s && k < K && v < V ? s[(size_t)k * V + v] : 0.f;
    }
}
template <int KP>
__device__ __forceinline__ void write_state(float* s, const float (&S)[KP / 8][4], int K, int V, int v0, int lane) {
#pragma unroll
  for (int nt = 0; nt < KP / 8; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 8 * nt + 2 * (lane & 3) + (j & 1), v = v0 + (lane >> 2) + 8 * (j >> 1);
      if (k < K && v < V) s[(size_t)k * V + v] = S[nt][j];
    }
}

// One block of nw warps per (sequence, value head, 16 nw columns of V); two stages of tiles, the next chunk's copies in
// flight while a chunk is computed.  Sout / Rout (either may be null): the state entering each chunk, bf16
// [item][VP][KP], and R, bf16 [item][64][VP].
template <int KP>
__global__ void __launch_bounds__(256, 1)
    k_delta_scan(Dims d, Table tb, In in, Prep pr, bf16* o, float* s_final, bf16* Sout, bf16* Rout) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = blockIdx.x / d.HV, hv = blockIdx.x - n * d.HV, hk = hv / d.G;
  const int vb = 16 * nw * blockIdx.y, v0 = vb + 16 * w;  // the block's and the warp's first column
  const bool live = v0 < d.VP;
  const size_t sb = Stage<KP>::bytes(nw);
  bf16* sbuf = reinterpret_cast<bf16*>(smem + 2 * sb) + w * 16 * (KP + 8);
  const int vp = 16 * nw + 8;
  const Seq sq = sequence(d, tb, n);
  const size_t su = ((size_t)n * d.HV + hv) * d.K * d.V;
  float S[KP / 8][4];
  read_state<KP>(S, in.s0 ? in.s0 + su : nullptr, d.K, d.V, v0, lane);
  if (sq.nc > 0) {
    load_stage<KP>(Stage<KP>(smem + (0) * sb, nw), d, in, pr, in.v, d.vs, d.vvec, sq.start, min(kC, sq.len), hk, hv,
                   (size_t)sq.chunk * d.HV + hv, vb, nw);
  }
  cp_commit();
  const int t2 = 2 * (lane & 3);
  for (int c = 0; c < sq.nc; ++c) {
    const Stage<KP> cur(smem + (c & 1) * sb, nw);
    const size_t item = (size_t)(sq.chunk + c) * d.HV + hv;
    const int first = sq.start + c * kC, rows = min(kC, sq.len - c * kC);
    if (c + 1 < sq.nc)
      load_stage<KP>(Stage<KP>(smem + ((c + 1) & 1) * sb, nw), d, in, pr, in.v, d.vs, d.vvec, first + kC, min(kC, sq.len - (c + 1) * kC), hk,
                     hv, item + d.HV, vb, nw);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    if (live) {
      if (Sout) store_state<KP>(sbuf, Sout + (item * d.VP + v0) * KP, S, lane);
      const float *eg = cur.gates, *ee = cur.gates + kC, *be = cur.gates + 2 * kC;
      const uint32_t ka = su32(cur.K), qa = su32(cur.Q);
      float X[8][4], O[8][4];  // (K S)^T, (Q S)^T: [16 v][64 t]
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) X[i][j] = O[i][j] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KP / 16; ++kb) {
        uint32_t h[4], l[4];
        split_a(S[2 * kb], S[2 * kb + 1], h, l);
#pragma unroll
        for (int tb4 = 0; tb4 < 4; ++tb4) {
          uint32_t b[4];
          ldm4(b, by_row(ka, KP + 8, 16 * tb4, 16 * kb, lane));
          mma(X[2 * tb4], h, b[0], b[1]);
          mma(X[2 * tb4 + 1], h, b[2], b[3]);
          mma(X[2 * tb4], l, b[0], b[1]);
          mma(X[2 * tb4 + 1], l, b[2], b[3]);
          if (o) {
            ldm4(b, by_row(qa, KP + 8, 16 * tb4, 16 * kb, lane));
            mma(O[2 * tb4], h, b[0], b[1]);
            mma(O[2 * tb4 + 1], h, b[2], b[3]);
            mma(O[2 * tb4], l, b[0], b[1]);
            mma(O[2 * tb4 + 1], l, b[2], b[3]);
          }
        }
      }
      uint32_t yh[4][4], yl[4][4];
      const uint32_t va = su32(cur.V) + 2u * (uint32_t)(16 * w);
#pragma unroll
      for (int tb4 = 0; tb4 < 4; ++tb4) {
        uint32_t v[4];
        ldm4t(v, by_row(va, vp, 16 * tb4, 0, lane));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float(&x)[4] = X[2 * tb4 + half];
          const int t = 16 * tb4 + 8 * half + t2;
          const float2 e = *reinterpret_cast<const float2*>(eg + t), b = *reinterpret_cast<const float2*>(be + t);
          x[0] = b.x * fmaf(-e.x, x[0], lo_f(v[2 * half]));
          x[1] = b.y * fmaf(-e.y, x[1], hi_f(v[2 * half]));
          x[2] = b.x * fmaf(-e.x, x[2], lo_f(v[2 * half + 1]));
          x[3] = b.y * fmaf(-e.y, x[3], hi_f(v[2 * half + 1]));
          float(&oo)[4] = O[2 * tb4 + half];
          oo[0] *= e.x;
          oo[1] *= e.y;
          oo[2] *= e.x;
          oo[3] *= e.y;
        }
        split_a(X[2 * tb4], X[2 * tb4 + 1], yh[tb4], yl[tb4]);
      }
      // R^T = Y^T T^T: step i takes from the steps j <= i
      float(&R)[8][4] = X;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) R[i][j] = 0.f;
      const uint32_t th = su32(cur.Th), tl = su32(cur.Tl), pa = su32(cur.P);
#pragma unroll
      for (int jb = 0; jb < 4; ++jb)
#pragma unroll
        for (int ib = jb; ib < 4; ++ib) {
          uint32_t b[4];
          ldm4(b, by_row(th, kTP, 16 * ib, 16 * jb, lane));
          mma(R[2 * ib], yh[jb], b[0], b[1]);
          mma(R[2 * ib + 1], yh[jb], b[2], b[3]);
          mma(R[2 * ib], yl[jb], b[0], b[1]);
          mma(R[2 * ib + 1], yl[jb], b[2], b[3]);
          ldm4(b, by_row(tl, kTP, 16 * ib, 16 * jb, lane));
          mma(R[2 * ib], yh[jb], b[0], b[1]);
          mma(R[2 * ib + 1], yh[jb], b[2], b[3]);
        }
      bf16* own = cur.V + 16 * w;  // the warp's columns of the V tile, which only it reads: staging for R and o
      if (Rout) {
        __syncwarp();
        stage_t(own, vp, R, lane);
        __syncwarp();
        store_cols(own, vp, Rout + item * kC * d.VP + v0, d.VP, kC, 16, true, lane);
      }
      if (o) {
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          uint32_t h[4], l[4];
          split_a(R[2 * jb], R[2 * jb + 1], h, l);
#pragma unroll
          for (int ib = jb; ib < 4; ++ib) {
            uint32_t b[4];
            ldm4(b, by_row(pa, kTP, 16 * ib, 16 * jb, lane));
            mma(O[2 * ib], h, b[0], b[1]);
            mma(O[2 * ib + 1], h, b[2], b[3]);
            mma(O[2 * ib], l, b[0], b[1]);
            mma(O[2 * ib + 1], l, b[2], b[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) O[i][j] *= in.scale;
        __syncwarp();
        stage_t(own, vp, O, lane);
        __syncwarp();
        store_cols(own, vp, o + ((long long)first * d.HV + hv) * d.V + v0, (long long)d.HV * d.V, rows, d.V - v0,
                   d.ovec, lane);
      }
      // S' = e^{G_end} S + K^T (e^{G_end - G} R)
      const float keep = eg[kC - 1];
#pragma unroll
      for (int i = 0; i < KP / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] *= keep;
#pragma unroll
      for (int tb4 = 0; tb4 < 4; ++tb4) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float(&x)[4] = R[2 * tb4 + half];
          const float2 e = *reinterpret_cast<const float2*>(ee + 16 * tb4 + 8 * half + t2);
          x[0] *= e.x;
          x[1] *= e.y;
          x[2] *= e.x;
          x[3] *= e.y;
        }
        uint32_t h[4], l[4];
        split_a(R[2 * tb4], R[2 * tb4 + 1], h, l);
#pragma unroll
        for (int kb = 0; kb < KP / 16; ++kb) {
          uint32_t b[4];
          ldm4t(b, by_col(ka, KP + 8, 16 * tb4, 16 * kb, lane));
          mma(S[2 * kb], h, b[0], b[1]);
          mma(S[2 * kb + 1], h, b[2], b[3]);
          mma(S[2 * kb], l, b[0], b[1]);
          mma(S[2 * kb + 1], l, b[2], b[3]);
        }
      }
    }
    __syncthreads();
  }
  if (live && s_final) write_state<KP>(s_final + su, S, d.K, d.V, v0, lane);
}

// The reverse scan: dS^T [16 v][KP] a warp.  dSout: the gradient of the state leaving each chunk, bf16 [item][VP][KP];
// dYout: bf16 [item][64][VP].
template <int KP>
__global__ void __launch_bounds__(256, 1) k_delta_rev(Dims d, Table tb, In in, Prep pr, const bf16* dout,
                                                       bool dovec, const float* ds_final, bf16* dv, float* ds0,
                                                       bf16* dSout, bf16* dYout) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = blockIdx.x / d.HV, hv = blockIdx.x - n * d.HV, hk = hv / d.G;
  const int vb = 16 * nw * blockIdx.y, v0 = vb + 16 * w;
  const bool live = v0 < d.VP;
  const size_t sb = Stage<KP>::bytes(nw);
  bf16* sbuf = reinterpret_cast<bf16*>(smem + 2 * sb) + w * 16 * (KP + 8);
  const int vp = 16 * nw + 8;
  const long long os = (long long)d.HV * d.V;
  const Seq sq = sequence(d, tb, n);
  const size_t su = ((size_t)n * d.HV + hv) * d.K * d.V;
  float S[KP / 8][4];
  read_state<KP>(S, ds_final ? ds_final + su : nullptr, d.K, d.V, v0, lane);
  if (sq.nc > 0) {
    const int c = sq.nc - 1;
    load_stage<KP>(Stage<KP>(smem + (c & 1) * sb, nw), d, in, pr, dout, os, dovec, sq.start + c * kC, sq.len - c * kC, hk, hv,
                   (size_t)(sq.chunk + c) * d.HV + hv, vb, nw);
  }
  cp_commit();
  const int t2 = 2 * (lane & 3);
  for (int c = sq.nc - 1; c >= 0; --c) {
    const Stage<KP> cur(smem + (c & 1) * sb, nw);
    const size_t item = (size_t)(sq.chunk + c) * d.HV + hv;
    const int first = sq.start + c * kC, rows = min(kC, sq.len - c * kC);
    if (c > 0)
      load_stage<KP>(Stage<KP>(smem + ((c - 1) & 1) * sb, nw), d, in, pr, dout, os, dovec, first - kC, kC, hk, hv, item - d.HV, vb, nw);
    cp_commit();
    cp_wait<1>();
    __syncthreads();
    if (live) {
      store_state<KP>(sbuf, dSout + (item * d.VP + v0) * KP, S, lane);
      const float *eg = cur.gates, *ee = cur.gates + kC, *be = cur.gates + 2 * kC;
      const uint32_t ka = su32(cur.K), qa = su32(cur.Q), th = su32(cur.Th), tl = su32(cur.Tl), pa = su32(cur.P);
      const uint32_t da = su32(cur.V) + 2u * (uint32_t)(16 * w);
      float X[8][4], U[8][4];  // (K dS')^T and (P^T dO)^T: [16 v][64 t]
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) X[i][j] = U[i][j] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KP / 16; ++kb) {
        uint32_t h[4], l[4];
        split_a(S[2 * kb], S[2 * kb + 1], h, l);
#pragma unroll
        for (int tb4 = 0; tb4 < 4; ++tb4) {
          uint32_t b[4];
          ldm4(b, by_row(ka, KP + 8, 16 * tb4, 16 * kb, lane));
          mma(X[2 * tb4], h, b[0], b[1]);
          mma(X[2 * tb4 + 1], h, b[2], b[3]);
          mma(X[2 * tb4], l, b[0], b[1]);
          mma(X[2 * tb4 + 1], l, b[2], b[3]);
        }
      }
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        uint32_t a[4];
        ldm4t(a, by_row(da, vp, 16 * ib, 0, lane));  // dO^T: rows v, columns i
#pragma unroll
        for (int tb4 = 0; tb4 <= ib; ++tb4) {
          uint32_t b[4];
          ldm4t(b, by_col(pa, kTP, 16 * ib, 16 * tb4, lane));
          mma(U[2 * tb4], a, b[0], b[1]);
          mma(U[2 * tb4 + 1], a, b[2], b[3]);
        }
      }
      uint32_t rh[4][4], rl[4][4];  // dR
#pragma unroll
      for (int tb4 = 0; tb4 < 4; ++tb4) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float2 e = *reinterpret_cast<const float2*>(ee + 16 * tb4 + 8 * half + t2);
          float(&x)[4] = X[2 * tb4 + half];
          const float(&u)[4] = U[2 * tb4 + half];
          x[0] = fmaf(in.scale, u[0], e.x * x[0]);
          x[1] = fmaf(in.scale, u[1], e.y * x[1]);
          x[2] = fmaf(in.scale, u[2], e.x * x[2]);
          x[3] = fmaf(in.scale, u[3], e.y * x[3]);
        }
        split_a(X[2 * tb4], X[2 * tb4 + 1], rh[tb4], rl[tb4]);
      }
      // dY^T = dR^T T: step t takes from the steps i >= t
      float(&Y)[8][4] = X;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) Y[i][j] = 0.f;
#pragma unroll
      for (int ib = 0; ib < 4; ++ib)
#pragma unroll
        for (int tb4 = 0; tb4 <= ib; ++tb4) {
          uint32_t b[4];
          ldm4t(b, by_col(th, kTP, 16 * ib, 16 * tb4, lane));
          mma(Y[2 * tb4], rh[ib], b[0], b[1]);
          mma(Y[2 * tb4 + 1], rh[ib], b[2], b[3]);
          mma(Y[2 * tb4], rl[ib], b[0], b[1]);
          mma(Y[2 * tb4 + 1], rl[ib], b[2], b[3]);
          ldm4t(b, by_col(tl, kTP, 16 * ib, 16 * tb4, lane));
          mma(Y[2 * tb4], rh[ib], b[0], b[1]);
          mma(Y[2 * tb4 + 1], rh[ib], b[2], b[3]);
        }
      const float keep = eg[kC - 1];
#pragma unroll
      for (int i = 0; i < KP / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] *= keep;
#pragma unroll
      for (int tb4 = 0; tb4 < 4; ++tb4) {
        uint32_t a[4], h[4], l[4], xh[4], xl[4];
        ldm4t(a, by_row(da, vp, 16 * tb4, 0, lane));
        float dx[2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int t = 16 * tb4 + 8 * half + t2;
          const float2 e = *reinterpret_cast<const float2*>(eg + t), b = *reinterpret_cast<const float2*>(be + t);
          const float f0 = in.scale * e.x, f1 = in.scale * e.y;
          split(f0 * lo_f(a[2 * half]), f1 * hi_f(a[2 * half]), h[2 * half], l[2 * half]);
          split(f0 * lo_f(a[2 * half + 1]), f1 * hi_f(a[2 * half + 1]), h[2 * half + 1], l[2 * half + 1]);
          const float(&y)[4] = Y[2 * tb4 + half];
          dx[half][0] = -b.x * e.x * y[0];
          dx[half][1] = -b.y * e.y * y[1];
          dx[half][2] = -b.x * e.x * y[2];
          dx[half][3] = -b.y * e.y * y[3];
        }
        split_a(dx[0], dx[1], xh, xl);
#pragma unroll
        for (int kb = 0; kb < KP / 16; ++kb) {
          uint32_t b[4];
          ldm4t(b, by_col(qa, KP + 8, 16 * tb4, 16 * kb, lane));
          mma(S[2 * kb], h, b[0], b[1]);
          mma(S[2 * kb + 1], h, b[2], b[3]);
          mma(S[2 * kb], l, b[0], b[1]);
          mma(S[2 * kb + 1], l, b[2], b[3]);
          ldm4t(b, by_col(ka, KP + 8, 16 * tb4, 16 * kb, lane));
          mma(S[2 * kb], xh, b[0], b[1]);
          mma(S[2 * kb + 1], xh, b[2], b[3]);
          mma(S[2 * kb], xl, b[0], b[1]);
          mma(S[2 * kb + 1], xl, b[2], b[3]);
        }
      }
      bf16* own = cur.V + 16 * w;  // dO has been read for the last time: staging for dY and dV
      __syncwarp();
      stage_t(own, vp, Y, lane);
      __syncwarp();
      store_cols(own, vp, dYout + item * kC * d.VP + v0, d.VP, kC, 16, true, lane);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 b = *reinterpret_cast<const float2*>(be + 8 * nt + t2);
        Y[nt][0] *= b.x;
        Y[nt][1] *= b.y;
        Y[nt][2] *= b.x;
        Y[nt][3] *= b.y;
      }
      __syncwarp();
      stage_t(own, vp, Y, lane);
      __syncwarp();
      store_cols(own, vp, dv + ((long long)first * d.HV + hv) * d.V + v0, os, rows, d.V - v0, d.ovec, lane);
    }
    __syncthreads();
  }
  if (live && ds0) write_state<KP>(ds0 + su, S, d.K, d.V, v0, lane);
}

// ---------------------------------------------------------------- dQ, dK, dbeta, dg of a chunk
struct GradOut {
  bf16 *dq, *dk;
  void *dg, *dbeta;
};

__device__ __forceinline__ void put_gate(void* p, size_t i, float x, bool is_bf16) {
  if (is_bf16)
    static_cast<bf16*>(p)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(p)[i] = x;
}

__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int KP>
size_t grads_smem(int VP) {
  return 2 * (size_t)(2 * kC * (KP + 8) + 3 * kC * (VP + 8) + 2 * VP * (KP + 8) + 2 * kC * kTP) +
         sizeof(float) * kGateRows * kC;
}

// Eight warps per (chunk, query/key head), its value heads one after another: warp w holds rows 16 (w % 4) .. + 15 and
// half w / 4 of the columns of every product, and dQ, dK of the head stay in its accumulators (so the sum over the
// value heads has one order).  Every factor of a decay is applied in fp32 to a product's result.
template <int KP>
__global__ void __launch_bounds__(256, 1) k_delta_grads(Dims d, Table tb, In in, Prep pr, const bf16* __restrict__ dout,
                                                         bool dovec, const bf16* __restrict__ Sst,
                                                         const bf16* __restrict__ Rst, const bf16* __restrict__ dSst,
                                                         const bf16* __restrict__ dYst, GradOut out) {
  constexpr int kP = KP + 8, kNT = KP / 16;  // kNT: 8-column tiles of a warp's half of the key axis
  extern __shared__ __align__(16) unsigned char smem[];
  const int VP = d.VP, vp = VP + 8;
  bf16* Ks = reinterpret_cast<bf16*>(smem);
  bf16* Qs = Ks + kC * kP;
  bf16* Os = Qs + kC * kP;   // dO
  bf16* Rs = Os + kC * vp;
  bf16* Ys = Rs + kC * vp;   // dY
  bf16* Ss = Ys + kC * vp;   // S^T [VP][KP]
  bf16* Ds = Ss + VP * kP;   // dS'^T
  bf16* B1 = Ds + VP * kP;   // scale dO R^T . decay
  bf16* B2 = B1 + kC * kTP;  // -dY R^T . beta decay
  float* gt = reinterpret_cast<float*>(B2 + kC * kTP);
  __shared__ float s_row[2][kC], s_col[4][kC], s_beta[2][kC], s_q[2][kC], s_z[2][kC], s_e[2][kC], s_yv[kC], s_ss[8];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g4 = lane >> 2, t2 = 2 * (lane & 3);
  const int r0 = 16 * (w & 3), half = w >> 2, rb = w & 3;
  const int c = blockIdx.x, hk = blockIdx.y;
  const Chunk ch = chunk_of(d, tb, c);
  if (ch.rows == 0) return;
  load_rows(Ks, kP, KP, in.k + (long long)ch.first * d.ks + (long long)hk * d.K, d.ks, ch.rows, d.K, d.kvec, tid, 256);
  load_rows(Qs, kP, KP, in.q + (long long)ch.first * d.qs + (long long)hk * d.K, d.qs, ch.rows, d.K, d.qvec, tid, 256);
  cp_commit();
  const uint32_t ka = su32(Ks), qa = su32(Qs), oa = su32(Os), ra = su32(Rs), ya = su32(Ys), sa = su32(Ss),
                 dsa = su32(Ds), b1a = su32(B1), b2a = su32(B2);
  float kk[4][4], qk[4][4], dQ[kNT][4], dK[kNT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[i][j] = qk[i][j] = 0.f;
#pragma unroll
  for (int i = 0; i < kNT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dQ[i][j] = dK[i][j] = 0.f;
  for (int gi = 0; gi < d.G; ++gi) {
    const int hv = hk * d.G + gi;
    const size_t item = (size_t)c * d.HV + hv;
    load_rows(Os, vp, VP, dout + ((long long)ch.first * d.HV + hv) * d.V, (long long)d.HV * d.V, ch.rows, d.V, dovec,
              tid, 256);
    load_dense(Rs, vp, VP / 8, Rst + item * kC * VP, kC, tid, 256);
    load_dense(Ys, vp, VP / 8, dYst + item * kC * VP, kC, tid, 256);
    load_dense(Ss, kP, KP / 8, Sst + item * VP * KP, VP, tid, 256);
    load_dense(Ds, kP, KP / 8, dSst + item * VP * KP, VP, tid, 256);
    for (int i = tid; i < kGateRows * kC / 4; i += 256)
      cp16(su32(gt + 4 * i), pr.gates + item * (kGateRows * kC) + 4 * i, true);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    if (gi == 0) {
#pragma unroll
      for (int kb = 0; kb < KP / 16; ++kb) {
        uint32_t ak[4], aq[4];
        ldm4(ak, by_col(ka, kP, r0, 16 * kb, lane));
        ldm4(aq, by_col(qa, kP, r0, 16 * kb, lane));
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
          uint32_t b[4];
          ldm4(b, by_row(ka, kP, 32 * half + 16 * jb, 16 * kb, lane));
          mma(kk[2 * jb], ak, b[0], b[1]);
          mma(kk[2 * jb + 1], ak, b[2], b[3]);
          mma(qk[2 * jb], aq, b[0], b[1]);
          mma(qk[2 * jb + 1], aq, b[2], b[3]);
        }
      }
    }
    const float *eg = gt, *ee = gt + kC, *be = gt + 2 * kC, *gh = gt + 3 * kC, *gl = gt + 4 * kC;
    // scores: rows i, columns j = 32 half ..
    float m1[4][4], m2[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m1[i][j] = m2[i][j] = 0.f;
    if (32 * half <= r0 + 15)
      for (int vb = 0; vb < VP; vb += 16) {
        uint32_t ao[4], ay[4];
        ldm4(ao, by_col(oa, vp, r0, vb, lane));
        ldm4(ay, by_col(ya, vp, r0, vb, lane));
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
          uint32_t b[4];
          ldm4(b, by_row(ra, vp, 32 * half + 16 * jb, vb, lane));
          mma(m1[2 * jb], ao, b[0], b[1]);
          mma(m1[2 * jb + 1], ao, b[2], b[3]);
          mma(m2[2 * jb], ay, b[0], b[1]);
          mma(m2[2 * jb + 1], ay, b[2], b[3]);
        }
      }
    {
      float rsum[2] = {0.f, 0.f}, bsum[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const int j = 32 * half + 8 * nt + t2;
        float csum[2] = {0.f, 0.f};
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int i = r0 + g4 + 8 * hh;
          float p[2], a[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool le = j + e <= i, lt = j + e < i;
            const float dec = le ? __expf((gh[i] - gh[j + e]) + (gl[i] - gl[j + e])) : 0.f;
            const float dp = in.scale * m1[nt][2 * hh + e] * dec;   // d (q_i . k_j)
            const float da = lt ? -m2[nt][2 * hh + e] * dec : 0.f;  // d (beta_i k_i . k_j)
            p[e] = le ? dp : 0.f;
            a[e] = be[i] * da;
            const float kkv = kk[nt][2 * hh + e];
            const float mm = p[e] * qk[nt][2 * hh + e] + a[e] * kkv;
            rsum[hh] += mm;
            csum[e] += mm;
            bsum[hh] += da * kkv;
          }
          *reinterpret_cast<uint32_t*>(B1 + i * kTP + j) = pack(p[0], p[1]);
          *reinterpret_cast<uint32_t*>(B2 + i * kTP + j) = pack(a[0], a[1]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = csum[e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          if (g4 == 0) s_col[rb][j + e] = x;
        }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const float x = quad_sum(rsum[hh]), y = quad_sum(bsum[hh]);
        if ((lane & 3) == 0) {
          s_row[half][r0 + g4 + 8 * hh] = x;
          s_beta[half][r0 + g4 + 8 * hh] = y;
        }
      }
    }
    // the products with the states: rows t, columns key = half KP/2 ..
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const uint32_t aa = pass == 0 ? oa : pass == 1 ? ya : ra, ba = pass == 2 ? dsa : sa;
      float z[kNT][4];
#pragma unroll
      for (int i = 0; i < kNT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[i][j] = 0.f;
      for (int vb = 0; vb < VP; vb += 16) {
        uint32_t a[4];
        ldm4(a, by_col(aa, vp, r0, vb, lane));
#pragma unroll
        for (int nb = 0; nb < kNT / 2; ++nb) {
          uint32_t b[4];
          ldm4t(b, by_col(ba, kP, vb, half * (KP / 2) + 16 * nb, lane));
          mma(z[2 * nb], a, b[0], b[1]);
          mma(z[2 * nb + 1], a, b[2], b[3]);
        }
      }
      float sum[2] = {0.f, 0.f};
      const bf16* dotted = pass == 0 ? Qs : Ks;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int t = r0 + g4 + 8 * hh;
        const float f = pass == 0 ? in.scale * eg[t] : pass == 1 ? -be[t] * eg[t] : ee[t];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(dotted + t * kP + half * (KP / 2) + 8 * nt + t2);
          const float z0 = z[nt][2 * hh], z1 = z[nt][2 * hh + 1];
          sum[hh] += z0 * lo_f(x) + z1 * hi_f(x);
          float(&acc)[4] = pass == 0 ? dQ[nt] : dK[nt];
          acc[2 * hh] = fmaf(f, z0, acc[2 * hh]);
          acc[2 * hh + 1] = fmaf(f, z1, acc[2 * hh + 1]);
        }
        const float y = quad_sum(sum[hh]);
        if ((lane & 3) == 0) (pass == 0 ? s_q : pass == 1 ? s_z : s_e)[half][t] = y;
      }
    }
    {  // <dS', S>
      float x = 0.f;
      for (int i = tid; i < VP * KP / 8; i += 256) {
        const int r = i / (KP / 8), cc = 8 * (i % (KP / 8));
        const uint4 a = *reinterpret_cast<const uint4*>(Ss + r * kP + cc);
        const uint4 b = *reinterpret_cast<const uint4*>(Ds + r * kP + cc);
        x += lo_f(a.x) * lo_f(b.x) + hi_f(a.x) * hi_f(b.x) + lo_f(a.y) * lo_f(b.y) + hi_f(a.y) * hi_f(b.y) +
             lo_f(a.z) * lo_f(b.z) + hi_f(a.z) * hi_f(b.z) + lo_f(a.w) * lo_f(b.w) + hi_f(a.w) * hi_f(b.w);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) s_ss[w] = x;
    }
    {  // dY . V of a row, four lanes each
      const int t = tid >> 2;
      float x = 0.f;
      if (t < ch.rows) {
        const bf16* vr = in.v + (long long)(ch.first + t) * d.vs + (long long)hv * d.V;
        for (int i = 8 * (tid & 3); i < d.V; i += 32) {  // in one order, however V is read
          uint32_t a[4];
          if (d.vvec) {
            const uint4 y = *reinterpret_cast<const uint4*>(vr + i);
            a[0] = y.x, a[1] = y.y, a[2] = y.z, a[3] = y.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[j] = pack(i + 2 * j < d.V ? __bfloat162float(vr[i + 2 * j]) : 0.f,
                          i + 2 * j + 1 < d.V ? __bfloat162float(vr[i + 2 * j + 1]) : 0.f);
          }
          const uint4 b = *reinterpret_cast<const uint4*>(Ys + t * vp + i);
          x = fmaf(lo_f(a[0]), lo_f(b.x), fmaf(hi_f(a[0]), hi_f(b.x), x));
          x = fmaf(lo_f(a[1]), lo_f(b.y), fmaf(hi_f(a[1]), hi_f(b.y), x));
          x = fmaf(lo_f(a[2]), lo_f(b.z), fmaf(hi_f(a[2]), hi_f(b.z), x));
          x = fmaf(lo_f(a[3]), lo_f(b.w), fmaf(hi_f(a[3]), hi_f(b.w), x));
        }
      }
      x = quad_sum(x);
      if ((tid & 3) == 0) s_yv[t] = x;
    }
    __syncthreads();
    // the score matrices times K and Q (below the diagonal: k-blocks up to rb; transposed: from rb)
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      uint32_t a1[4], a2[4], a1t[4], a2t[4];
      const bool lower = jb <= rb, upper = jb >= rb;
      if (lower) {
        ldm4(a1, by_col(b1a, kTP, r0, 16 * jb, lane));
        ldm4(a2, by_col(b2a, kTP, r0, 16 * jb, lane));
      }
      if (upper) {
        ldm4t(a1t, by_row(b1a, kTP, 16 * jb, r0, lane));
        ldm4t(a2t, by_row(b2a, kTP, 16 * jb, r0, lane));
      }
#pragma unroll
      for (int nb = 0; nb < kNT / 2; ++nb) {
        uint32_t bk[4], bq[4];
        ldm4t(bk, by_col(ka, kP, 16 * jb, half * (KP / 2) + 16 * nb, lane));
        if (lower) {
          mma(dQ[2 * nb], a1, bk[0], bk[1]);
          mma(dQ[2 * nb + 1], a1, bk[2], bk[3]);
          mma(dK[2 * nb], a2, bk[0], bk[1]);
          mma(dK[2 * nb + 1], a2, bk[2], bk[3]);
        }
        if (upper) {
          ldm4t(bq, by_col(qa, kP, 16 * jb, half * (KP / 2) + 16 * nb, lane));
          mma(dK[2 * nb], a1t, bq[0], bq[1]);
          mma(dK[2 * nb + 1], a1t, bq[2], bq[3]);
          mma(dK[2 * nb], a2t, bk[0], bk[1]);
          mma(dK[2 * nb + 1], a2t, bk[2], bk[3]);
        }
      }
    }
    if (w == 0) {  // dbeta, dG and its sums from the right, two steps a lane
      float dG[2], e_all = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const float z = s_z[0][t] + s_z[1][t], e = ee[t] * (s_e[0][t] + s_e[1][t]);
        const float col = (s_col[0][t] + s_col[1][t]) + (s_col[2][t] + s_col[3][t]);
        dG[i] = (s_row[0][t] + s_row[1][t]) - col + in.scale * eg[t] * (s_q[0][t] + s_q[1][t]) - be[t] * eg[t] * z - e;
        e_all += e;
        if (t < ch.rows)
          put_gate(out.dbeta, (size_t)(ch.first + t) * d.HV + hv,
                   s_yv[t] - eg[t] * z + (s_beta[0][t] + s_beta[1][t]), d.gate_bf16);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) e_all += __shfl_xor_sync(0xffffffffu, e_all, o);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += s_ss[i];
      const float end = e_all + eg[kC - 1] * ss;
      float sum = dG[0] + dG[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, sum, o);
        if (lane + o < 32) sum += y;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        if (t < ch.rows)
          put_gate(out.dg, (size_t)(ch.first + t) * d.HV + hv, end + (i ? sum - dG[0] : sum), d.gate_bf16);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int t = r0 + g4 + 8 * hh;
    if (t >= ch.rows) continue;
    const size_t row = ((size_t)(ch.first + t) * d.H + hk) * d.K;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int k = half * (KP / 2) + 8 * nt + t2;
      const float q0 = dQ[nt][2 * hh], q1 = dQ[nt][2 * hh + 1], k0 = dK[nt][2 * hh], k1 = dK[nt][2 * hh + 1];
      if ((d.K & 1) == 0) {
        if (k < d.K) {
          *reinterpret_cast<uint32_t*>(out.dq + row + k) = pack(q0, q1);
          *reinterpret_cast<uint32_t*>(out.dk + row + k) = pack(k0, k1);
        }
      } else {
        if (k < d.K) {
          out.dq[row + k] = __float2bfloat16_rn(q0);
          out.dk[row + k] = __float2bfloat16_rn(k0);
        }
        if (k + 1 < d.K) {
          out.dq[row + k + 1] = __float2bfloat16_rn(q1);
          out.dk[row + k + 1] = __float2bfloat16_rn(k1);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host side
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What a training forward keeps for its backward, and a backward without it makes again.
struct Kept {
  Prep prep;
  bf16 *S, *R;
};
Prep carve_prep(const Dims& d, Carver& cv) {
  const size_t items = (size_t)d.nc * d.HV;
  Prep p;
  p.Thi = cv.take<bf16>(items * kC * kC);
  p.Tlo = cv.take<bf16>(items * kC * kC);
  p.P = cv.take<bf16>(items * kC * kC);
  p.gates = cv.take<float>(items * kGateRows * kC);
  return p;
}
Kept carve_kept(const Dims& d, Carver& cv) {
  const size_t items = (size_t)d.nc * d.HV;
  Kept k;
  k.prep = carve_prep(d, cv);
  k.S = cv.take<bf16>(items * d.VP * d.KP);
  k.R = cv.take<bf16>(items * kC * d.VP);
  return k;
}
Table carve_table(const Dims& d, Carver& cv) {
  Table t = {nullptr, nullptr, nullptr};
  if (d.packed) {
    t.start = cv.take<int>(d.N);
    t.len = cv.take<int>(d.N);
    t.chunk = cv.take<int>((size_t)d.N + 1);
  }
  return t;
}
struct Grads {
  bf16 *dS, *dY;
};
Grads carve_grads(const Dims& d, Carver& cv) {
  const size_t items = (size_t)d.nc * d.HV;
  Grads g;
  g.dS = cv.take<bf16>(items * d.VP * d.KP);
  g.dY = cv.take<bf16>(items * kC * d.VP);
  return g;
}

size_t workspace(const Dims& d, bool backward, bool stashed) {
  Carver cv(nullptr);
  carve_table(d, cv);
  if (backward) carve_grads(d, cv);
  if (!stashed) {
    if (backward)
      carve_kept(d, cv);
    else
      carve_prep(d, cv);
  }
  return cv.off;
}

ssd_status check(std::initializer_list<const void*> req, std::initializer_list<const void*> opt) {
  for (const void* p : req)
    if (!p) return SSD_ERR_INVALID_ARG;
  for (const void* p : req)
    if (!al16(p)) return SSD_ERR_ALIGNMENT;
  for (const void* p : opt)
    if (p && !al16(p)) return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}
// q, k, v may lie inside a wider tensor: they need the alignment of their type only.
ssd_status check_elem(std::initializer_list<const void*> req, unsigned bytes) {
  for (const void* p : req) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) % bytes) return SSD_ERR_ALIGNMENT;
  }
  return SSD_OK;
}

cudaError_t sm_count(int* n) {
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : e;
}

// Warps of a scan's block: a block has an SM to itself (its two stages take most of the shared memory), so the
// fewest warps a block with which one wave of blocks holds them all, at most eight.
cudaError_t scan_warps(const Dims& d, int* nw) {
  int sms;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long units = (long long)d.N * d.HV;
  const int vt = d.VP / 16;
  *nw = 1;
  while (*nw < 8 && *nw < vt && units * ((vt + *nw - 1) / *nw) > sms) *nw *= 2;
  return cudaSuccess;
}
template <int KP>
size_t scan_smem(int nw) {
  return 2 * Stage<KP>::bytes(nw) + 2 * (size_t)nw * 16 * (KP + 8);
}

template <typename F>
cudaError_t allow_smem(F* f, size_t bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int KP>
cudaError_t run_prep(const Dims& d, const Table& tb, const In& in, const Prep& pr, const int* cu, int* status,
                     cudaStream_t st) {
  if (d.packed) SSD_LAUNCH("k_delta_table", st, k_delta_table<<<1, 1024, 0, st>>>(cu, d.N, d.T, tb));
  const size_t sm = 2 * (size_t)(2 * kC * (KP + 8)) + sizeof(float) * (2 * kC + 32) * kFP;
  cudaError_t e = allow_smem(k_delta_prep<KP>, sm);
  if (e != cudaSuccess) return e;
  SSD_LAUNCH("k_delta_prep", st,
             k_delta_prep<KP><<<dim3((unsigned)d.nc, (unsigned)d.H), 128, sm, st>>>(d, tb, in, pr, status));
  return cudaGetLastError();
}

template <int KP>
cudaError_t run_scan(const Dims& d, const Table& tb, const In& in, const Prep& pr, bf16* o, float* s_final, bf16* S,
                     bf16* R, cudaStream_t st) {
  int nw;
  cudaError_t e = scan_warps(d, &nw);
  if (e == cudaSuccess) e = allow_smem(k_delta_scan<KP>, scan_smem<KP>(nw));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(d.N * d.HV), (unsigned)((d.VP / 16 + nw - 1) / nw));
  SSD_LAUNCH("k_delta_scan", st,
             k_delta_scan<KP><<<grid, 32 * nw, scan_smem<KP>(nw), st>>>(d, tb, in, pr, o, s_final, S, R));
  return cudaGetLastError();
}

template <int KP>
cudaError_t run_backward(const Dims& d, const Table& tb, const In& in, const Kept& kept, const Grads& gr,
                         const bf16* dout, const float* ds_final, const GradOut& out, bf16* dv, float* ds0,
                         cudaStream_t st) {
  int nw;
  cudaError_t e = scan_warps(d, &nw);
  if (e == cudaSuccess) e = allow_smem(k_delta_rev<KP>, scan_smem<KP>(nw));
  if (e == cudaSuccess) e = allow_smem(k_delta_grads<KP>, grads_smem<KP>(d.VP));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(d.N * d.HV), (unsigned)((d.VP / 16 + nw - 1) / nw));
  SSD_LAUNCH("k_delta_rev", st,
             k_delta_rev<KP><<<grid, 32 * nw, scan_smem<KP>(nw), st>>>(d, tb, in, kept.prep, dout, d.ovec, ds_final, dv,
                                                                       ds0, gr.dS, gr.dY));
  SSD_LAUNCH("k_delta_grads", st,
             k_delta_grads<KP><<<dim3((unsigned)d.nc, (unsigned)d.H), 256, grads_smem<KP>(d.VP), st>>>(
                 d, tb, in, kept.prep, dout, d.ovec, kept.S, kept.R, gr.dS, gr.dY, out));
  return cudaGetLastError();
}

}  // namespace

ssd_status make_dims(const ssd_delta_problem* p, bool f32_ok, Dims* d) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->io_dtype != SSD_F32 && p->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (p->gate_dtype != SSD_F32 && p->gate_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->value_heads < 1 || p->key_dim < 1 || p->value_dim < 1)
    return SSD_ERR_INVALID_ARG;
  if (p->packed != 0 && p->packed != 1) return SSD_ERR_INVALID_ARG;
  if (p->q_stride < 0 || p->k_stride < 0 || p->v_stride < 0) return SSD_ERR_INVALID_ARG;
  if (p->io_dtype == SSD_F32 && !f32_ok) return SSD_ERR_DTYPE;
  if (p->value_heads % p->nheads) return SSD_ERR_SHAPE;
  if (p->key_dim > 128 || p->value_dim > 128 || p->nheads > 65535) return SSD_ERR_SHAPE;
  constexpr long long kInt = 0x7fffffffll;
  if (p->batch > kInt || p->seqlen > kInt || p->value_heads > kInt) return SSD_ERR_SHAPE;
  const long long tokens = p->packed ? p->seqlen : p->batch * p->seqlen;
  if (tokens > kInt || p->batch * p->value_heads > kInt) return SSD_ERR_SHAPE;
  const long long qw = p->nheads * p->key_dim, vw = p->value_heads * p->value_dim;
  if ((p->q_stride && p->q_stride < qw) || (p->k_stride && p->k_stride < qw) || (p->v_stride && p->v_stride < vw))
    return SSD_ERR_SHAPE;
  const long long nc = p->packed ? p->seqlen / kC + p->batch : p->batch * ((p->seqlen + kC - 1) / kC);
  if (nc > kInt || nc * p->value_heads > (1ll << 36)) return SSD_ERR_SHAPE;
  d->N = (int)p->batch;
  d->T = (int)p->seqlen;
  d->H = (int)p->nheads;
  d->HV = (int)p->value_heads;
  d->G = d->HV / d->H;
  d->K = (int)p->key_dim;
  d->V = (int)p->value_dim;
  d->KP = d->K <= 64 ? 64 : 128;
  d->VP = (d->V + 15) / 16 * 16;
  d->nc = (int)nc;
  d->packed = p->packed != 0;
  d->f32 = p->io_dtype == SSD_F32;
  d->gate_bf16 = p->gate_dtype == SSD_BF16;
  d->qs = p->q_stride ? p->q_stride : qw;
  d->ks = p->k_stride ? p->k_stride : qw;
  d->vs = p->v_stride ? p->v_stride : vw;
  d->qvec = d->K % 8 == 0 && d->qs % 8 == 0;
  d->kvec = d->K % 8 == 0 && d->ks % 8 == 0;
  d->vvec = d->V % 8 == 0 && d->vs % 8 == 0;
  d->ovec = d->V % 8 == 0;
  return SSD_OK;
}

}  // namespace delta
}  // namespace ssd

using namespace ssd;
using namespace ssd::delta;

extern "C" {

ssd_status ssd_delta_workspace_size(const ssd_delta_problem* prob, int backward, int stashed, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARG;
  delta::Dims d;
  const ssd_status s = make_dims(prob, false, &d);
  if (s != SSD_OK) return s;
  *bytes = workspace(d, backward != 0, stashed != 0);
  return SSD_OK;
}

ssd_status ssd_delta_stash_size(const ssd_delta_problem* prob, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARG;
  delta::Dims d;
  const ssd_status s = make_dims(prob, false, &d);
  if (s != SSD_OK) return s;
  Carver cv(nullptr);
  carve_kept(d, cv);
  *bytes = cv.off;
  return SSD_OK;
}

ssd_status ssd_delta_forward(const ssd_delta_problem* prob, const void* q, const void* k, const void* v, const void* g,
                             const void* beta, const float* s0, const int32_t* cu_seqlens, float scale, void* o,
                             float* s_final, void* stash, size_t stash_bytes, void* ws, size_t ws_bytes,
                             void* cuda_stream) {
  delta::Dims d;
  ssd_status s = make_dims(prob, false, &d);
  if (s != SSD_OK) return s;
  if ((cu_seqlens != nullptr) != d.packed) return SSD_ERR_INVALID_ARG;
  if ((s = check_elem({q, k, v}, 2)) != SSD_OK) return s;
  if ((s = check({g, beta, o, ws}, {s0, s_final, stash})) != SSD_OK) return s;
  if (cu_seqlens && (s = check_elem({cu_seqlens}, 4)) != SSD_OK) return s;
  if (ws_bytes < workspace(d, false, stash != nullptr)) return SSD_ERR_WORKSPACE;
  if (stash) {
    Carver need(nullptr);
    carve_kept(d, need);
    if (stash_bytes < need.off) return SSD_ERR_WORKSPACE;
  }
  d.qvec = d.qvec && al16(q);
  d.kvec = d.kvec && al16(k);
  d.vvec = d.vvec && al16(v);
  Carver cv(ws);
  const Table tb = carve_table(d, cv);
  Kept kept = {};
  if (stash) {
    Carver cs(stash);
    kept = carve_kept(d, cs);
  } else {
    kept.prep = carve_prep(d, cv);
  }
  const In in{(const bf16*)q, (const bf16*)k, (const bf16*)v, g, beta, s0, scale};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (d.KP == 64) {
    e = run_prep<64>(d, tb, in, kept.prep, cu_seqlens, (int*)ws, st);
    if (e == cudaSuccess) e = run_scan<64>(d, tb, in, kept.prep, (bf16*)o, s_final, kept.S, kept.R, st);
  } else {
    e = run_prep<128>(d, tb, in, kept.prep, cu_seqlens, (int*)ws, st);
    if (e == cudaSuccess) e = run_scan<128>(d, tb, in, kept.prep, (bf16*)o, s_final, kept.S, kept.R, st);
  }
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_delta_backward(const ssd_delta_problem* prob, const void* dout, const float* ds_final, const void* q,
                              const void* k, const void* v, const void* g, const void* beta, const float* s0,
                              const int32_t* cu_seqlens, float scale, void* dq, void* dk, void* dv, void* dg,
                              void* dbeta, float* ds0, const void* stash, size_t stash_bytes, void* ws,
                              size_t ws_bytes, void* cuda_stream) {
  delta::Dims d;
  ssd_status s = make_dims(prob, false, &d);
  if (s != SSD_OK) return s;
  if ((cu_seqlens != nullptr) != d.packed) return SSD_ERR_INVALID_ARG;
  if ((s = check_elem({q, k, v}, 2)) != SSD_OK) return s;
  if ((s = check({dout, g, beta, dq, dk, dv, dg, dbeta, ws}, {ds_final, s0, ds0, stash})) != SSD_OK) return s;
  if (cu_seqlens && (s = check_elem({cu_seqlens}, 4)) != SSD_OK) return s;
  if (ws_bytes < workspace(d, true, stash != nullptr)) return SSD_ERR_WORKSPACE;
  if (stash) {
    Carver need(nullptr);
    carve_kept(d, need);
    if (stash_bytes < need.off) return SSD_ERR_WORKSPACE;
  }
  d.qvec = d.qvec && al16(q);
  d.kvec = d.kvec && al16(k);
  d.vvec = d.vvec && al16(v);
  Carver cv(ws);
  const Table tb = carve_table(d, cv);
  const Grads gr = carve_grads(d, cv);
  Kept kept;
  if (stash) {
    Carver cs(const_cast<void*>(stash));
    kept = carve_kept(d, cs);
  } else {
    kept = carve_kept(d, cv);
  }
  const In in{(const bf16*)q, (const bf16*)k, (const bf16*)v, g, beta, s0, scale};
  const GradOut out{(bf16*)dq, (bf16*)dk, dg, dbeta};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (stash) {
    if (d.packed) SSD_LAUNCH("k_delta_table", st, k_delta_table<<<1, 1024, 0, st>>>(cu_seqlens, d.N, d.T, tb));
    e = cudaMemsetAsync(ws, 0, sizeof(int32_t), st);
  } else if (d.KP == 64) {
    e = run_prep<64>(d, tb, in, kept.prep, cu_seqlens, (int*)ws, st);
    if (e == cudaSuccess) e = run_scan<64>(d, tb, in, kept.prep, nullptr, nullptr, kept.S, kept.R, st);
  } else {
    e = run_prep<128>(d, tb, in, kept.prep, cu_seqlens, (int*)ws, st);
    if (e == cudaSuccess) e = run_scan<128>(d, tb, in, kept.prep, nullptr, nullptr, kept.S, kept.R, st);
  }
  if (e == cudaSuccess)
    e = d.KP == 64 ? run_backward<64>(d, tb, in, kept, gr, (const bf16*)dout, ds_final, out, (bf16*)dv, ds0, st)
                   : run_backward<128>(d, tb, in, kept, gr, (const bf16*)dout, ds_final, out, (bf16*)dv, ds0, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
