// gdn_elem.cuh -- element types of the generation and q/k entry points: loads of 8 consecutive
// values into FP32 and stores rounded to the type once, to nearest even; and the host's check of pointers to
// 4-byte elements.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

__host__ __device__ constexpr int elem_bytes(int dtype) { return dtype == GDN_FP32 ? 4 : 2; }

// tables, counters and weights lie on their elements' boundary (or are null): else a load faults
template <typename... P> inline bool on_words(const P*... p) { return ((((uintptr_t)p & 3) == 0) && ...); }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E> __device__ __forceinline__ E from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ float2 pair_f32(uint32_t u, const __nv_bfloat16*) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_f32(uint32_t u, const __half*) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t f32_pair(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f32_pair(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 consecutive values as they lie in memory (16 or 32 bytes, 16-byte aligned)
template <typename E> struct Raw8 {
  uint4 u;
  __device__ __forceinline__ void load(const E* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair_f32(w[i], (const E*)nullptr);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void put(const float (&v)[8]) {
    u = make_uint4(f32_pair(v[0], v[1], (const E*)nullptr), f32_pair(v[2], v[3], (const E*)nullptr),
                   f32_pair(v[4], v[5], (const E*)nullptr), f32_pair(v[6], v[7], (const E*)nullptr));
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void put(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// V consecutive values (4 to 16 bytes) as they lie in memory
template <typename E, int V> struct RawV {
  static constexpr int WORDS = V * (int)sizeof(E) / 4;
  uint32_t u[WORDS];
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (WORDS == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
    } else if constexpr (WORDS == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      u[0] = x.x; u[1] = x.y;
    } else {
      u[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  // from shared memory, by one access of the whole (left to itself the compiler reads 16-bit values one by one)
  __device__ __forceinline__ void load_shared(uint32_t at) {
    if constexpr (WORDS == 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at) : "memory");
    else if constexpr (WORDS == 2)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "r"(at) : "memory");
    else
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u[0]) : "r"(at) : "memory");
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    else if constexpr (WORDS == 2) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint32_t*>(p) = u[0];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) u[i] = 0u;
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(E) == 4) {
        v[i] = __uint_as_float(u[i]);
      } else {
        const float2 f = pair_f32(u[i], (const E*)nullptr);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void put(const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(E) == 4) u[i] = __float_as_uint(v[i]);
      else u[i] = f32_pair(v[2 * i], v[2 * i + 1], (const E*)nullptr);
    }
  }
};

}  // namespace gdn
