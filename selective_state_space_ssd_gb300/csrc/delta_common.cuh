// Building blocks of the delta rule: its sizes and where its sequences lie, the records and kept tiles that its kernels
// hand to one another, warp-level bf16 products out of shared-memory tiles, and the split of an fp32 operand into two
// bf16 ones.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd.h"
#include "ssd_internal.h"

namespace ssd {
namespace delta {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;              // steps of a chunk
// Per-step records of a chunk: e^G, e^{G_end - G}, beta, G / ln 2, scale e^G.  G / ln 2 is one fp32 number: the gradients'
// decays e^{G_i - G_j} come from it alone and are good to 2^-24 |G|, 1e-3 at the steepest sum of 64 steps that kMinG
// allows and 1e-5 at a decay of e^-2 a step; the forward's (k_delta_prep) come from two.
constexpr int kGateRows = 5;
constexpr float kMinG = -200.f;     // e^g of anything below is 0; keeps G - G' defined where g is -inf

struct Dims {
  int N, T, H, HV, G, K, V;          // sequences, steps (packed: of all), heads, value heads, HV / H, widths
  int KP, VP;                        // K rounded up to 64 or 128, V rounded up to a multiple of 16
  int nc;                            // chunks (packed: the most there can be, over all sequences)
  bool packed, f32, gate_bf16;
  long long qs, ks, vs;              // elements from a token to the next in q, k, v
  bool qvec, kvec, vvec, ovec;       // rows of 16-byte pieces
};

// Where the sequences lie: sequence n has its steps at start[n] .. start[n] + len[n] - 1 of the token axis and its
// chunks at chunk[n] .. chunk[n + 1] - 1 of the chunk axis.  Filled from cu_seqlens for a packed batch; computed
// where it is read otherwise.
constexpr int kRanked = 1024;  // a packed batch of more sequences keeps their order: its many blocks even out by themselves
struct Table {
  int *start, *len, *chunk;
  int* order;  // the sequences, those with the most chunks first (up to kRanked of them)
};

// Outputs that hold one row a step (null: not there) and the bytes of a row, an even number: where a step of a packed axis
// belongs to no sequence they get zeros.
constexpr int kStepOutputs = 5;
struct StepRows {
  void* p[kStepOutputs];
  int bytes[kStepOutputs];
};

// One record per (chunk, value head), item = chunk * HV + head, in one piece of memory that one bulk copy brings in:
// four [64][64] bf16 tiles, swizzled as the tensor cores read them (element (i, j) at tile_off), and the decays.
//   (I + A)^-1 rounded to bf16; what that rounding left, rounded; P_ij = scale e^{G_i - G_j} q_i . k_j (j <= i) in the same
//   two parts (16-blocks above the diagonal are not written and not read); float [5][64] of kGateRows
constexpr int kRecordGates = 4 * kC * kC * 2;
constexpr int kRecordBytes = kRecordGates + kGateRows * kC * 4;
__host__ __device__ constexpr int tile_off(int i, int j) { return i * 128 + (((j >> 3) ^ (i & 7)) << 4) + 2 * (j & 7); }

// The sizes of a problem, or the error that it is refused with.
ssd_status make_dims(const ssd_delta_problem* p, bool f32_ok, Dims* d);

struct In {
  const bf16 *q, *k, *v;
  const void *g, *beta;
  const float* s0;
  float scale;
};

// A long sequence of few heads in parts.  The chunks of every sequence are cut into `parts` runs of the same number; a
// chunk's step is affine in the state, S_out = M S_in + B, so a first launch walks the runs but the last from a zero
// state (B; the first run from s0) and, with V = 0, from the identity (M), k_delta_join goes through the runs
// (S_in of run i + 1 = M_i S_in_i + B_i), and the scan proper walks all runs at once.  The reverse scan is affine in the
// gradient of the state that leaves a chunk and is split the same way, from the last run on.
struct Split {
  int parts;      // 1: none
  float* states;  // [N * HV][parts - 1][K][V]: B, then S_in of the run after it
  float* maps;    // [N * HV][parts - 2][KP][KP]: M of runs 1 .., zeros around it
};

// The scans (ssd_delta_scan.cu).  S / R (null: not kept): the state entering each chunk and R, both bf16 and transposed,
// as 128-byte-swizzled images: S^T [KP / 64][VP rows][64 keys], R^T [VP rows][64 steps].  o may be null (S and R only).
// dS / dY of the reverse scan: the gradient of the state leaving each chunk, laid out like S, and dY by steps,
// [ceil(VP / 64)][64 steps][64 columns].
cudaError_t forward_scan(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const Split& split,
                         bf16* o, float* s_final, bf16* S, bf16* R, int* status, cudaStream_t st);
cudaError_t reverse_scan(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const Split& split,
                         const bf16* dout, const float* ds_final, bf16* dv, float* ds0, bf16* dS, bf16* dY, int* status,
                         cudaStream_t st);
int scan_parts(const Dims& d);
// dQ, dK, dbeta, dg of every chunk (ssd_delta_grads.cu).
struct GradOut {
  bf16 *dq, *dk;
  void *dg, *dbeta;
};
cudaError_t chunk_grads(const Dims& d, const Table& tb, const In& in, const uint8_t* records, const bf16* dout,
                        const bf16* S, const bf16* R, const bf16* dS, const bf16* dY, const GradOut& out, int* status,
                        cudaStream_t st);

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: the 16 bytes are filled with zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8x8 tiles; lane l gives the address of row l % 8 of tile l / 8.
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// c[16x8] += a[16x16] b[16x8], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Two fp32 operations in one instruction: (d0, d1) = (a0, a1) (b0, b1) + (c0, c1), and without the sum.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 c, a, b, c; mov.b64 {%0, %1}, c; }"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};\n"
      "mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// (x, y) = h + l with both in bf16: h rounds to 8 bits and l holds the next 8, so h + l is within 2^-17 of each.
__device__ __forceinline__ void split(float x, float y, uint32_t& h, uint32_t& l) {
  h = pack(x, y);
  float a, b;
  fma2(a, b, lo_f(h), hi_f(h), -1.f, -1.f, x, y);
  l = pack(a, b);
}

// Lane addresses into a tile of rows of `pitch` elements, for ldm4 / ldm4t of 16 x 16 elements at
// (row, col).  by_row: tiles in the order (rows 0-7, cols 0-7), (rows 0-7, cols 8-15), (rows 8-15, cols 0-7), ...;
// by_col: (0-7, 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15).
__device__ __forceinline__ uint32_t by_row(uint32_t base, int pitch, int row, int col, int lane) {
  return base + 2u * (uint32_t)((row + (lane & 7) + ((lane >> 4) << 3)) * pitch + col + (((lane >> 3) & 1) << 3));
}
__device__ __forceinline__ uint32_t by_col(uint32_t base, int pitch, int row, int col, int lane) {
  return base + 2u * (uint32_t)((row + (lane & 7) + (((lane >> 3) & 1) << 3)) * pitch + col + ((lane >> 4) << 3));
}

// 64 rows of W (64 or 128) elements into a tile by NT threads: row r from src + r * stride, zeros past `rows` and `cols`.
// vec: every row starts on 16 bytes and cols is a multiple of 8 (asynchronous copies; the caller commits and waits);
// otherwise element by element.
template <int W, int NT>
__device__ __forceinline__ void load_rows(bf16* dst, int pitch, const bf16* src, long long stride, int rows, int cols,
                                          bool vec, int tid) {
  constexpr int w8 = W / 8, kStep = NT / w8;
  static_assert(NT % w8 == 0, "whole rows a step");
  if (vec) {
    const int r0 = tid / w8, c = 8 * (tid % w8);
    const bf16* s = src + (long long)r0 * stride + c;
    uint32_t a = su32(dst) + 2u * (uint32_t)(r0 * pitch + c);
    for (int r = r0; r < kC; r += kStep) {
      const bool ok = r < rows && c < cols;
      cp16(a, ok ? s : src, ok);
      s += kStep * stride;
      a += 2u * (uint32_t)(kStep * pitch);
    }
  } else {
    for (int i = tid; i < kC * W; i += NT) {
      const int r = i / W, c = i - r * W;
      dst[r * pitch + c] = r < rows && c < cols ? src[(long long)r * stride + c] : __float2bfloat16_rn(0.f);
    }
  }
}

__device__ __forceinline__ float gate(const void* p, size_t i, bool is_bf16) {
  return is_bf16 ? __bfloat162float(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}

struct Seq {
  int start, len, chunk, nc;  // first step, steps, first chunk, chunks
};
__device__ __forceinline__ Seq sequence(const Dims& d, const Table& t, int n) {
  Seq s;
  if (d.packed) {
    s.start = t.start[n];
    s.len = t.len[n];
    s.chunk = t.chunk[n];
  } else {
    s.start = n * d.T;
    s.len = d.T;
    s.chunk = n * ((d.T + kC - 1) / kC);
  }
  s.nc = (s.len + kC - 1) / kC;
  return s;
}

// The sequence of chunk c, and how many steps of it the chunk holds (0: past the last chunk) from which step.
struct Chunk {
  int n, first, rows;
};
__device__ __forceinline__ Chunk chunk_of(const Dims& d, const Table& t, int c) {
  Chunk r;
  if (!d.packed) {
    const int per = (d.T + kC - 1) / kC;
    r.n = c / per;
    const int at = (c - r.n * per) * kC;
    r.first = r.n * d.T + at;
    r.rows = min(kC, d.T - at);
    return r;
  }
  r.n = 0;
  r.first = 0;
  r.rows = 0;
  if (c >= t.chunk[d.N]) return r;
  int lo = 0, hi = d.N - 1;  // the last n with chunk[n] <= c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int at = (c - t.chunk[lo]) * kC;
  r.n = lo;
  r.first = t.start[lo] + at;
  r.rows = min(kC, t.len[lo] - at);
  return r;
}

}  // namespace delta
}  // namespace ssd
