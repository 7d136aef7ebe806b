// What the tcgen05 kernels of the delta rule share (beside tc_common.cuh): MMAs whose left operand lies in tensor memory,
// waits and signals of whole warps, and copies into swizzled tiles.
#pragma once

#include "delta_common.cuh"
#include "tc_common.cuh"

namespace ssd {
namespace delta {

using namespace ssd::tc;

constexpr int kLoadWarps = 2, kLoadThreads = 32 * kLoadWarps;

// D[tmem] (+)= A[tmem] B[smem]^T
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void st8u(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void st4u(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The other way: a tile of shared memory to global memory, as part of the issuing thread's bulk group.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// A wait of a whole warp: every lane learns the same answer, so a bound that runs out stops the warp as one.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t phase, int* status, int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, phase, status, code)) != 0;
}
// The warp's tensor-memory stores are done and visible to whoever waits on the barrier.
__device__ __forceinline__ void signal_tmem(uint64_t* bar, int lane) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// The warp has read what it needs (tensor or shared memory).
__device__ __forceinline__ void signal_read(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void ld16(uint32_t addr, float (&x)[16]) {
  uint32_t u[16];
  tmem_ld16_nowait(addr, u);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void lds16(const float* p, float (&x)[16]) {  // the same 16 floats for every lane
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
  }
}

__device__ __forceinline__ void lds8(const float* p, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
  }
}

// A value that the compiler takes for a new one: what is computed from it stays where it is used, and is not kept in
// registers around a loop that has none to spare.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

__device__ __forceinline__ uint32_t v_off(int t, int v) {  // element (t, v) of the V tile
  return (uint32_t)((v >> 6) * (kC * 128)) + sw128_chunk(t, (v & 63) >> 3) + 2u * (v & 7);
}

// 64 rows of `cols` valid elements, zeros past `rows` and `cols`, into a 128-byte-swizzled tile whose 64-column atoms
// hold R rows each, element by element (rows that are not whole 16-byte pieces): eight loads in flight a thread.
__device__ __forceinline__ void load_elements(uint8_t* tile, int R, int width, const bf16* src, long long stride,
                                              int rows, int cols, int tid) {
  constexpr int kN = kLoadThreads, kBatch = 8;
  const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
  for (int base = tid; base < kC * width; base += kN * kBatch) {
    unsigned short x[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = base + j * kN, r = i / width, c = i - r * width;
      x[j] = r < rows && c < cols ? s[(long long)r * stride + c] : (unsigned short)0;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = base + j * kN, r = i / width, c = i - r * width;
      if (r < kC) *reinterpret_cast<unsigned short*>(tile + (c >> 6) * R * 128 + sw128_chunk(r, (c & 63) >> 3) + 2 * (c & 7)) = x[j];
    }
  }
}
__device__ __forceinline__ void zero_rows(uint8_t* tile, int R, int atoms, int rows, int tid) {
  for (int i = tid; i < (kC - rows) * atoms * 8; i += kLoadThreads) {
    const int r = rows + i / (atoms * 8), j = i % (atoms * 8);
    *reinterpret_cast<uint4*>(tile + (j >> 3) * R * 128 + r * 128 + (j & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* p) {
  return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u);
}


}  // namespace delta
}  // namespace ssd
