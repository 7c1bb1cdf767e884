// Shared pieces of the operators around the layer: typed loads and stores of
// one to eight consecutive elements, and warp reductions in a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace moe {

// Programmatic dependent launch: a kernel launched with op_launch may be set up
// while the one before it in the stream still runs, and touches no memory before
// pdl_wait(), which returns when that one is complete and its writes are visible.
// pdl_next() says that the kernel after may be set up from here on (once every
// block has said so or has ended).  Without the launch attribute both do nothing.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Elements of a 16-byte load.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ float op_f32(float v) { return v; }
__device__ __forceinline__ float op_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float op_f32(__half v) { return __half2float(v); }

// Nearest value of type T (ties to even).
template <typename T>
__device__ __forceinline__ T op_from(float v);
template <>
__device__ __forceinline__ float op_from<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 op_from<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half op_from<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float2 op_unpack(uint32_t u, float) { return make_float2(__uint_as_float(u), 0.f); }
__device__ __forceinline__ float2 op_unpack(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ float2 op_unpack(uint32_t u, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ uint32_t op_pack(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t op_pack(float lo, float hi, __half) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The 16 bytes q as kVec<T> floats, and back.
template <typename T>
__device__ __forceinline__ void op_unpack16(const uint4& q, float* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = op_unpack(w[i], T());
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 op_pack16(const float* f) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    return make_uint4(op_pack(f[0], f[1], T()), op_pack(f[2], f[3], T()), op_pack(f[4], f[5], T()),
                      op_pack(f[6], f[7], T()));
  }
}

// VL consecutive elements: one 16-byte access (VL = kVec<T>, p 16-byte
// aligned) or one element (VL = 1).
template <typename T, int VL>
__device__ __forceinline__ void op_load(const T* p, float* f) {
  static_assert(VL == 1 || VL == kVec<T>, "one element or 16 bytes");
  if constexpr (VL == 1)
    f[0] = op_f32(*p);
  else
    op_unpack16<T>(*reinterpret_cast<const uint4*>(p), f);
}

template <typename T, int VL>
__device__ __forceinline__ void op_store(T* p, const float* f) {
  static_assert(VL == 1 || VL == kVec<T>, "one element or 16 bytes");
  if constexpr (VL == 1)
    *p = op_from<T>(f[0]);
  else
    *reinterpret_cast<uint4*>(p) = op_pack16<T>(f);
}

// VL consecutive fp32 values at p (16-byte aligned when VL > 1).
template <int VL>
__device__ __forceinline__ void op_load_f32(const float* p, float* f) {
  if constexpr (VL == 1) {
    f[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < VL; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      f[i] = q.x;
      f[i + 1] = q.y;
      f[i + 2] = q.z;
      f[i + 3] = q.w;
    }
  }
}

// Two fp32 numbers in a register pair, for the packed arithmetic of sm_100 (one
// instruction for both, each rounded as the scalar one is).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float f2_sum(F2 a) {
  const float2 r = f2_get(a);
  return r.x + r.y;
}

// The 16 bytes q as kVec<T> / 2 pairs, and back.
template <typename T>
__device__ __forceinline__ void op_unpack16(const uint4& q, F2* f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4) {
    f[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    f[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = op_unpack(w[i], T());
      f[i] = f2(p.x, p.y);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 op_pack16(const F2* f) {
  float g[kVec<T>];
#pragma unroll
  for (int i = 0; i < kVec<T> / 2; ++i) {
    const float2 p = f2_get(f[i]);
    g[2 * i] = p.x;
    g[2 * i + 1] = p.y;
  }
  return op_pack16<T>(g);
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Largest value of the warp (no NaN), by the hardware's reduction.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace moe
