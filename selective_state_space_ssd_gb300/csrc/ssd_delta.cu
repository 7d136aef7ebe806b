// The gated delta rule with one decay per head, by chunks of 64 steps on the tensor cores: forward, its stash for
// training, and the backward pass.
//
// Per sequence and value head, with state S [K, V] and G the running sum of g inside a chunk:
//     A_ij = beta_i e^{G_i - G_j} k_i.k_j  (j < i),     T = (I + A)^-1
//     Y = beta (V - e^G K S),   R = T Y                 (row t of R is what step t writes along k_t)
//     O = scale (e^G Q S + P R),   P_ij = e^{G_i - G_j} q_i.k_j  (j <= i)
//     S' = e^{G_end} S + K^T (e^{G_end - G} R)
// The chunks of a sequence are independent but for S, so a call is
//     k_delta_prep   every (chunk, value head) at once: T, P and the decays
//     k_delta_scan   per (sequence, value head) one chunk after another: R, S', O
// and the backward pass, given the S entering each chunk and R,
//     k_delta_rev    per (sequence, value head) in reverse: dR = scale P^T dO + e^{G_end-G} K dS', dY = T^T dR,
//                    dX = -beta e^G dY, dS = e^{G_end} dS' + scale Q^T e^G dO + K^T dX;  dV = beta dY
//     k_delta_grads  every (chunk, query/key head) at once: dQ, dK, dbeta, dg from S, dS', R, dY
// (the scans in ssd_delta_scan.cu, the gradients in ssd_delta_grads.cu).
//
// Precision.  q, k, v, dO are bf16 as given.  What a scan computes in fp32 and has to multiply again (S, Y, T, P, R and
// their gradients) enters the tensor cores as two bf16 numbers, high and low, so a product of two such is three
// products; what is dropped is 2^-17 of each factor.  The state itself is held and summed in fp32 over any length; with
// 16-bit factors it comes out at a relative error of 3e-6 to 4e-6 against 64 bits, where fp32 products give 1e-7 to 3e-7,
// and single bf16 operands would carry 2^-9 through thousands of steps.  The gradients' last products (k_delta_grads) take
// S, dS', R and dY rounded to bf16, as the stash holds them: their results are gradients of bf16 inputs (relative error
// 2.5e-3 for dq and dk; dg 2.5e-3 and dbeta 1.8e-3 in fp32, 2.9e-3 and 2.4e-3 in bf16; 1.7e-3 for o and dv, which is the
// rounding of a bf16 result).  Two parts there would leave only that rounding, and double the 0.8 GB that those four
// tensors are written and then read with in a training step of 8192 chunks and heads; the kernel's shared memory has no
// room for them.
#include <initializer_list>

#include "delta_common.cuh"
#include "ssd.h"

namespace ssd {
namespace delta {
namespace {

// ---------------------------------------------------------------- packed sequences
// Zeros into bytes a .. b - 1 (both even) of p (16-byte aligned) by `threads` threads, of which this is number t.
__device__ void zero_bytes(void* p, long long a, long long b, int t, int threads) {
  for (long long at = a / 16 * 16 + 16ll * t; at < b; at += 16ll * threads) {
    unsigned char* q = static_cast<unsigned char*>(p) + at;
    if (at >= a && at + 16 <= b) {
      *reinterpret_cast<uint4*>(q) = make_uint4(0, 0, 0, 0);
    } else {
      for (int i = 0; i < 16; i += 2)
        if (at + i >= a && at + i < b) *reinterpret_cast<unsigned short*>(q + i) = 0;
    }
  }
}

// cu_seqlens -> start, length and first chunk of every sequence, and their order by length, by the first block.  Bounds that
// leave the token axis or run backwards are pulled in (a running maximum), so no later kernel can leave its buffers whatever
// the values are.  The other blocks meanwhile write the outputs' rows of the steps that belong to no sequence: those before
// the first bound and those past the largest, on an axis that is padded.
constexpr int kTableBlocks = 64;
__global__ void __launch_bounds__(1024) k_delta_table(const int* __restrict__ cu, int N, int T, Table tb, StepRows rows) {
  __shared__ int s_max[1024], s_sum[1024];
  __shared__ int carry_end, carry_chunk;
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    int end = 0;
    for (int n = tid; n <= N; n += 1024) end = max(end, min(max(cu[n], 0), T));
    end = __reduce_max_sync(0xffffffffu, end);
    if ((tid & 31) == 0) s_max[tid >> 5] = end;
    __syncthreads();
    end = __reduce_max_sync(0xffffffffu, s_max[tid & 31]);
    const long long start = min(max(cu[0], 0), T);
    const int t = ((int)blockIdx.x - 1) * 1024 + tid, threads = (kTableBlocks - 1) * 1024;
    for (int i = 0; i < kStepOutputs; ++i) {
      if (!rows.p[i]) continue;
      zero_bytes(rows.p[i], 0, start * rows.bytes[i], t, threads);
      zero_bytes(rows.p[i], (long long)end * rows.bytes[i], (long long)T * rows.bytes[i], t, threads);
    }
    return;
  }
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
    if (N <= kRanked) {  // (one pass of this loop)
      s_max[tid] = nc;
      __syncthreads();
      int rank = 0;
      for (int m = 0; m < N; ++m) rank += s_max[m] > nc || (s_max[m] == nc && m < n);
      if (n < N) tb.order[rank] = n;
    }
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

// Four warps per (chunk, value head); warp w holds rows 16 w .. 16 w + 15 of K K^T and Q K^T, up to the diagonal, and
// multiplies them by the decays.  (I + A)^-1 in the place of A: the four 16-blocks of the diagonal by forward
// substitution (a lane a column), then twice the block rule  [[a, 0], [c, b]]^-1 = [[a', 0], [-b' c a', b']].
// Substitution and block products stay small for strongly correlated keys, where a series in powers of A would not.
// A chain of small steps, bound by its latency and its issue: five blocks an SM, at 96 registers, hide one another's.  A
// block a value head: the heads of a group share K K^T and Q K^T, but would come one after another.  8192 chunks and heads
// of K = 128 take 121 us (134 with the copies after the decays, and without the packed fp32 operations).
template <int KP>
__global__ void __launch_bounds__(128, 5) k_delta_prep(Dims d, Table tb, In in, uint8_t* records, int* status) {
  constexpr int kP = KP + 8;
  extern __shared__ __align__(16) unsigned char smem[];
  bf16* Ks = reinterpret_cast<bf16*>(smem);
  bf16* Qs = Ks + kC * kP;
  float* Af = reinterpret_cast<float*>(smem);  // over K and Q, once their products are in registers
  float* Pf = Af + kC * kFP;
  float* Mf = Pf + kC * kFP;  // [32][kFP]
  __shared__ float s_hi[kC], s_lo[kC], s_beta[kC];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int c = blockIdx.x, hv = blockIdx.y, hk = hv / d.G;
  if (c == 0 && hv == 0 && tid == 0) *status = 0;
  const Chunk ch = chunk_of(d, tb, c);
  if (ch.rows == 0) return;
  uint8_t* record = records + ((size_t)c * d.HV + hv) * kRecordBytes;
  if (w == 0) {  // G of two steps a lane; the sums in fp64, in units of log 2 as a high and a low fp32 part
    double x[2];
    float b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      float v = 0.f;
      b[i] = 0.f;
      if (t < ch.rows) {
        const size_t at = (size_t)(ch.first + t) * d.HV + hv;
        v = gate(in.g, at, d.gate_bf16);
        b[i] = gate(in.beta, at, d.gate_bf16);
        v = v < kMinG ? kMinG : v;
      }
      x[i] = (double)v * 1.4426950408889634;
    }
    double sum = x[0] + x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const double end = __shfl_sync(0xffffffffu, sum, 31);
    float2* gr = reinterpret_cast<float2*>(record + kRecordGates) + lane;
    float eg[2], ee[2], g2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const double gt = i ? sum : sum - x[1];
      const float h = (float)gt;
      s_hi[t] = h;
      s_lo[t] = (float)(gt - (double)h);
      s_beta[t] = b[i];
      eg[i] = exp2f(h);
      ee[i] = exp2f((float)(end - gt));
      g2[i] = h;
    }
    gr[0] = make_float2(eg[0], eg[1]);
    gr[kC / 2] = make_float2(ee[0], ee[1]);
    gr[kC] = make_float2(b[0], b[1]);
    gr[3 * kC / 2] = make_float2(g2[0], g2[1]);
    gr[2 * kC] = make_float2(in.scale * eg[0], in.scale * eg[1]);
  } else {  // the other warps copy the tiles meanwhile
    load_rows<KP, 96>(Ks, kP, in.k + (long long)ch.first * d.ks + (long long)hk * d.K, d.ks, ch.rows, d.K, d.kvec, tid - 32);
    load_rows<KP, 96>(Qs, kP, in.q + (long long)ch.first * d.qs + (long long)hk * d.K, d.qs, ch.rows, d.K, d.qvec, tid - 32);
    cp_commit();
  }
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
  __syncthreads();
  {
    const float2 hi = make_float2(s_hi[r0 + g4], s_hi[r0 + g4 + 8]), lo = make_float2(s_lo[r0 + g4], s_lo[r0 + g4 + 8]),
                 be = make_float2(s_beta[r0 + g4], s_beta[r0 + g4 + 8]);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt > 2 * w + 1) break;
      const int j = 8 * nt + t2;
      const float2 hj = *reinterpret_cast<const float2*>(s_hi + j), lj = *reinterpret_cast<const float2*>(s_lo + j);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = r0 + g4 + 8 * half;
        const float h = half ? hi.y : hi.x, l = half ? lo.y : lo.x, b = half ? be.y : be.x;
        float x0, x1, y0, y1;  // e^{G_i - G_j}, from its exponent's two parts
        fma2(x0, x1, hj.x, hj.y, -1.f, -1.f, h, h);
        fma2(y0, y1, lj.x, lj.y, -1.f, -1.f, l, l);
        fma2(x0, x1, x0, x1, 1.f, 1.f, y0, y1);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x0) : "f"(x0));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x1) : "f"(x1));
        if (nt >= 2 * w) {  // the diagonal's blocks
          x0 = i >= j ? x0 : 0.f;
          x1 = i >= j + 1 ? x1 : 0.f;
        }
        mul2(y0, y1, x0, x1, in.scale, in.scale);
        mul2(y0, y1, y0, y1, qk[nt][2 * half], qk[nt][2 * half + 1]);
        *reinterpret_cast<float2*>(Pf + i * kFP + j) = make_float2(y0, y1);
        mul2(x0, x1, x0, x1, b, b);
        mul2(x0, x1, x0, x1, kk[nt][2 * half], kk[nt][2 * half + 1]);
        if (nt >= 2 * w) {
          x0 = i > j ? x0 : 0.f;
          x1 = i > j + 1 ? x1 : 0.f;
        }
        *reinterpret_cast<float2*>(Af + i * kFP + j) = make_float2(x0, x1);
      }
    }
  }
  __syncwarp();
  {  // the diagonal block of this warp, column lane % 16
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == (lane & 15) ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const float4 a = *reinterpret_cast<const float4*>(Af + (r0 + i) * kFP + r0 + j);
        s = fmaf(-a.x, x[j], s);
        if (j + 1 < i) s = fmaf(-a.y, x[j + 1], s);
        if (j + 2 < i) s = fmaf(-a.z, x[j + 2], s);
        if (j + 3 < i) s = fmaf(-a.w, x[j + 3], s);
      }
      x[i] = s;
    }
    __syncwarp();
    if (lane < 16)
#pragma unroll
      for (int i = 0; i < 16; ++i) Af[(r0 + i) * kFP + r0 + lane] = x[i];
  }
  __syncthreads();
  float m[2][4];
  if ((w & 1) == 0) {  // rows 16 .. 31 (warp 0) and 48 .. 63 (warp 2): -b' c a'
    const int a0 = 16 * w, b0 = a0 + 16;
    mul16(m, Af + b0 * kFP + a0, Af + a0 * kFP + a0, 16, lane);
    put16(Mf + w * 8 * kFP, m, 1.f, lane);
    __syncwarp();
    mul16(m, Af + b0 * kFP + b0, Mf + w * 8 * kFP, 16, lane);
    put16(Af + b0 * kFP + a0, m, -1.f, lane);
  } else {  // the blocks above the diagonal that the next products read
    const int a0 = 16 * (w - 1);
    for (int i = lane; i < 64; i += 32)
      *reinterpret_cast<float4*>(Af + (a0 + (i >> 2)) * kFP + a0 + 16 + 4 * (i & 3)) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  const int br = 16 * (w >> 1), bc = 16 * (w & 1);  // one 16-block of the 32 x 32 product a warp
  mul16(m, Af + (32 + br) * kFP, Af + bc, 32, lane);
  put16(Mf + br * kFP + bc, m, 1.f, lane);
  __syncthreads();
  mul16(m, Af + (32 + br) * kFP + 32, Mf + bc, 32, lane);
  put16(Af + (32 + br) * kFP + bc, m, -1.f, lane);
  __syncthreads();
  // 16-byte pieces of the four tiles in the order of memory, up to the diagonal's blocks
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int i = (tid >> 3) + 16 * n, j = (tid & 7) ^ (i & 7);
    if (8 * j >= 16 * (n + 1)) continue;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float* f = (which ? Pf : Af) + i * kFP + 8 * j;
      const float4 x = *reinterpret_cast<const float4*>(f), y = *reinterpret_cast<const float4*>(f + 4);
      uint32_t h[4], l[4];
      split(x.x, x.y, h[0], l[0]);
      split(x.z, x.w, h[1], l[1]);
      split(y.x, y.y, h[2], l[2]);
      split(y.z, y.w, h[3], l[3]);
      uint4* dst = reinterpret_cast<uint4*>(record + which * 16384 + tile_off(i, 8 * j));
      dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
      dst[512] = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

// ---------------------------------------------------------------- host side
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What a training forward keeps for its backward, and a backward without it makes again.
struct Kept {
  uint8_t* records;
  bf16 *S, *R;
};
uint8_t* carve_records(const Dims& d, Carver& cv) { return cv.take<uint8_t>((size_t)d.nc * d.HV * kRecordBytes); }
Kept carve_kept(const Dims& d, Carver& cv) {
  const size_t items = (size_t)d.nc * d.HV;
  Kept k;
  k.records = carve_records(d, cv);
  k.S = cv.take<bf16>(items * d.VP * d.KP);
  k.R = cv.take<bf16>(items * kC * d.VP);
  return k;
}
Table carve_table(const Dims& d, Carver& cv) {
  Table t = {nullptr, nullptr, nullptr, nullptr};
  if (d.packed) {
    t.start = cv.take<int>(d.N);
    t.len = cv.take<int>(d.N);
    t.chunk = cv.take<int>((size_t)d.N + 1);
    t.order = cv.take<int>(d.N);
  }
  return t;
}
Split carve_split(const Dims& d, Carver& cv) {
  Split sp = {scan_parts(d), nullptr, nullptr};
  const size_t units = (size_t)d.N * d.HV;
  if (sp.parts > 1) {
    sp.states = cv.take<float>(units * (sp.parts - 1) * d.K * d.V);
    sp.maps = cv.take<float>(units * (sp.parts - 2) * d.KP * d.KP);
  }
  return sp;
}
struct Grads {
  bf16 *dS, *dY;
};
Grads carve_grads(const Dims& d, Carver& cv) {
  const size_t items = (size_t)d.nc * d.HV;
  Grads g;
  g.dS = cv.take<bf16>(items * d.VP * d.KP);
  g.dY = cv.take<bf16>(items * kC * ((d.VP + 63) / 64 * 64));
  return g;
}

size_t workspace(const Dims& d, bool backward, bool stashed) {
  Carver cv(nullptr);
  carve_table(d, cv);
  if (backward) carve_grads(d, cv);
  carve_split(d, cv);
  if (!stashed) {
    if (backward)
      carve_kept(d, cv);
    else
      carve_records(d, cv);
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

template <typename F>
cudaError_t allow_smem(F* f, size_t bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

void run_table(const Dims& d, const Table& tb, const int* cu, const StepRows& rows, cudaStream_t st) {
  if (d.packed) SSD_LAUNCH("k_delta_table", st, k_delta_table<<<kTableBlocks, 1024, 0, st>>>(cu, d.N, d.T, tb, rows));
}

template <int KP>
cudaError_t run_prep(const Dims& d, const Table& tb, const In& in, uint8_t* records, int* status, cudaStream_t st) {
  const size_t kq = 2 * (size_t)(2 * kC * (KP + 8)), at = sizeof(float) * (2 * kC + 32) * kFP, sm = kq > at ? kq : at;
  cudaError_t e = allow_smem(k_delta_prep<KP>, sm);
  if (e != cudaSuccess) return e;
  SSD_LAUNCH("k_delta_prep", st,
             k_delta_prep<KP><<<dim3((unsigned)d.nc, (unsigned)d.HV), 128, sm, st>>>(d, tb, in, records, status));
  return cudaGetLastError();
}

cudaError_t prepare(const Dims& d, const Table& tb, const In& in, uint8_t* records, int* status, cudaStream_t st) {
  return d.KP == 64 ? run_prep<64>(d, tb, in, records, status, st) : run_prep<128>(d, tb, in, records, status, st);
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
  if (p->key_dim > 128 || p->value_dim > 128 || p->value_heads > 65535) return SSD_ERR_SHAPE;
  constexpr long long kInt = 0x7fffffffll;
  if (p->nheads > kInt || p->batch > kInt || p->seqlen > kInt || p->value_heads > kInt) return SSD_ERR_SHAPE;
  const long long tokens = p->packed ? p->seqlen : p->batch * p->seqlen;
  if (tokens > kInt || p->batch * p->value_heads > kInt) return SSD_ERR_SHAPE;
  const long long qw = p->nheads * p->key_dim, vw = p->value_heads * p->value_dim;
  if ((p->q_stride && p->q_stride < qw) || (p->k_stride && p->k_stride < qw) || (p->v_stride && p->v_stride < vw))
    return SSD_ERR_SHAPE;
  const long long nc = p->packed ? p->seqlen / kC + p->batch : p->batch * ((p->seqlen + kC - 1) / kC);
  if (nc > kInt || nc * p->nheads > (1ll << 30) || nc * p->value_heads > (1ll << 36)) return SSD_ERR_SHAPE;
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
  const Split split = carve_split(d, cv);
  Kept kept = {};
  if (stash) {
    Carver cs(stash);
    kept = carve_kept(d, cs);
  } else {
    kept.records = carve_records(d, cv);
  }
  const In in{(const bf16*)q, (const bf16*)k, (const bf16*)v, g, beta, s0, scale};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  run_table(d, tb, cu_seqlens, StepRows{{o}, {d.HV * d.V * 2}}, st);
  cudaError_t e = prepare(d, tb, in, kept.records, (int*)ws, st);
  if (e == cudaSuccess) e = forward_scan(d, tb, in, kept.records, split, (bf16*)o, s_final, kept.S, kept.R, (int*)ws, st);
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
  const Split split = carve_split(d, cv);
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
  const int qk = d.H * d.K * 2, gate = d.HV * (d.gate_bf16 ? 2 : 4);
  run_table(d, tb, cu_seqlens, StepRows{{dq, dk, dv, dg, dbeta}, {qk, qk, d.HV * d.V * 2, gate, gate}}, st);
  cudaError_t e = cudaSuccess;
  if (stash) {
    e = cudaMemsetAsync(ws, 0, sizeof(int32_t), st);
  } else {
    e = prepare(d, tb, in, kept.records, (int*)ws, st);
    if (e == cudaSuccess) e = forward_scan(d, tb, in, kept.records, split, nullptr, nullptr, kept.S, kept.R, (int*)ws, st);
  }
  if (e == cudaSuccess)
    e = reverse_scan(d, tb, in, kept.records, split, (const bf16*)dout, ds_final, (bf16*)dv, ds0, gr.dS, gr.dY, (int*)ws, st);
  if (e == cudaSuccess)
    e = chunk_grads(d, tb, in, kept.records, (const bf16*)dout, kept.S, kept.R, gr.dS, gr.dY, out, (int*)ws, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
