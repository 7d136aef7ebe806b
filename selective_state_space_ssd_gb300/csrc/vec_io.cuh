// Loads, stores and copies of a few bf16 or fp32 elements at a time.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace ssd {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ void unpack(uint32_t w, float (&v)[1]) { v[0] = __uint_as_float(w); }
__device__ __forceinline__ void unpack(uint32_t w, float (&v)[2]) {
  v[0] = __uint_as_float(w << 16);
  v[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Asynchronous copies to shared memory; not ok: zeros, and nothing is read.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4_of(void* dst, const void* src, int bytes) {  // the first bytes, the others are zeros
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool ok) { copy4_of(dst, src, ok ? 4 : 0); }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void copies_wait() {  // all but the last kN groups have arrived
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

// kW elements as fp32: 1, or 2 or 4 at an address that is a multiple of their size.
template <typename T, int kW>
__device__ __forceinline__ void load(const T* p, float (&v)[kW]) {
  if constexpr (kW == 1) {
    if constexpr (sizeof(T) == 4)
      v[0] = *p;
    else
      v[0] = __bfloat162float(*p);
  } else if constexpr (kW == 2) {
    if constexpr (sizeof(T) == 4) {
      const float2 q = *reinterpret_cast<const float2*>(p);
      v[0] = q.x, v[1] = q.y;
    } else {
      unpack(*reinterpret_cast<const uint32_t*>(p), v);
    }
  } else if constexpr (sizeof(T) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
}
template <typename T, int kW>
__device__ __forceinline__ void save(T* p, const float (&v)[kW]) {
  if constexpr (kW == 1) {
    if constexpr (sizeof(T) == 4)
      *p = v[0];
    else
      *p = __float2bfloat16_rn(v[0]);
  } else if constexpr (kW == 2) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = pack2(v[0], v[1]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
  }
}

inline bool off(const void* p, uintptr_t align) { return reinterpret_cast<uintptr_t>(p) % align != 0; }

}  // namespace ssd
