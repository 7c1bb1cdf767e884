// Global norm over many tensors, and clipping: one pass that adds up squares
// (or takes the largest magnitude) into one fp64 partial per block, and one that
// reads the partials, forms the factor and scales.  Both are bound by memory;
// the second walks the chunks backwards, so that what the first read last is
// still in L2.
//
// The tensor list travels in the kernel's parameters (at most CLIP_MAX tensors
// a launch), so a captured graph holds it and nothing has to be copied.
#pragma once

#include "ops_common.cuh"

namespace moe {

constexpr int CLIP_THREADS = 512;
constexpr int CLIP_MAX = 1024;  // 29 bytes of parameters each, below the 32764 a launch may have

enum ClipType : uint8_t { kClipF32 = 0, kClipBF16 = 1, kClipF16 = 2 };

template <int MAXT>
struct ClipList {
  const void* in[MAXT];
  void* out[MAXT];
  long long n[MAXT];
  int first[MAXT];  // number of chunks before the tensor's
  uint8_t type[MAXT];
  int count, chunks;
  int chunk;  // elements of a chunk: a multiple of 64, so chunks keep a tensor's alignment
};

// The tensor of chunk c: the last one whose first chunk is not after c.
template <int MAXT>
__device__ __forceinline__ int clip_find(const ClipList<MAXT>& l, int c) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Squares of one 16-byte vector (or one element): added up in fp32, and again in
// fp64 where the fp32 sum may have overflowed, lost small squares or met a NaN.
template <typename T, int VL>
__device__ __forceinline__ double clip_squares(const float* f) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VL; ++i) s = fmaf(f[i], f[i], s);
  if (s >= 1e-30f && s <= 3e38f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < VL; ++i) d += static_cast<double>(f[i]) * static_cast<double>(f[i]);
  return d;
}

// Elements before the first 16-byte boundary of p (at most n).
template <typename T>
__device__ __forceinline__ int clip_head(const T* p, int n) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
  const int h = off ? (16 - off) / static_cast<int>(sizeof(T)) : 0;
  return h < n ? h : n;
}

template <int V>
struct ClipWidth {
  static constexpr int value = V;
};

template <typename T, bool MAX>
__device__ __forceinline__ void clip_reduce_chunk(const T* p, int n, double& sum, uint32_t& top) {
  constexpr int VL = kVec<T>;
  const int head = clip_head(p, n);
  auto take = [&](const float* f, auto vl) {
    constexpr int W = decltype(vl)::value;
    if constexpr (MAX) {
      // magnitudes as integers: a NaN is above everything and stays
#pragma unroll
      for (int i = 0; i < W; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    } else {
      sum += clip_squares<T, W>(f);
    }
  };
  if (static_cast<int>(threadIdx.x) < head) {
    const float f = op_f32(p[threadIdx.x]);
    take(&f, ClipWidth<1>());
  }
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  const int nv = (n - head) / VL;
  int i = threadIdx.x;
  for (; i + 3 * CLIP_THREADS < nv; i += 4 * CLIP_THREADS) {
    uint4 a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) a[u] = q[i + u * CLIP_THREADS];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[VL];
      op_unpack16<T>(a[u], f);
      take(f, ClipWidth<VL>());
    }
  }
  for (; i < nv; i += CLIP_THREADS) {
    float f[VL];
    op_unpack16<T>(q[i], f);
    take(f, ClipWidth<VL>());
  }
  const int done = head + nv * VL;
  if (static_cast<int>(threadIdx.x) < n - done) {
    const float f = op_f32(p[done + threadIdx.x]);
    take(&f, ClipWidth<1>());
  }
}

// partial[blockIdx.x] = the block's sum of squares, or largest magnitude.
template <int MAXT, bool MAX>
__global__ void __launch_bounds__(CLIP_THREADS)
    clip_norm_kernel(const __grid_constant__ ClipList<MAXT> l, double* __restrict__ partial) {
  __shared__ double red[CLIP_THREADS / 32];
  pdl_next();
  pdl_wait();
  double sum = 0.0;
  uint32_t top = 0u;
  for (int c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const int k = clip_find(l, c);
    const long long at = static_cast<long long>(c - l.first[k]) * l.chunk;
    const int n = static_cast<int>(min(static_cast<long long>(l.chunk), l.n[k] - at));
    if (l.type[k] == kClipF32)
      clip_reduce_chunk<float, MAX>(static_cast<const float*>(l.in[k]) + at, n, sum, top);
    else if (l.type[k] == kClipBF16)
      clip_reduce_chunk<__nv_bfloat16, MAX>(static_cast<const __nv_bfloat16*>(l.in[k]) + at, n, sum, top);
    else
      clip_reduce_chunk<__half, MAX>(static_cast<const __half*>(l.in[k]) + at, n, sum, top);
  }
  if constexpr (MAX) sum = static_cast<double>(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
  else sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = red[0];
    for (int w = 1; w < CLIP_THREADS / 32; ++w) {
      if constexpr (MAX) a = red[w] > a || red[w] != red[w] ? red[w] : a;
      else a += red[w];
    }
    partial[blockIdx.x] = a;
  }
}

template <typename T>
__device__ __forceinline__ void clip_scale_chunk(const T* p, T* o, int n, float coef) {
  constexpr int VL = kVec<T>;
  // one alignment for both: head, vectors, tail; else element by element
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15u) != 0u) {
    for (int i = threadIdx.x; i < n; i += CLIP_THREADS) o[i] = op_from<T>(op_f32(p[i]) * coef);
    return;
  }
  const int head = clip_head(p, n);
  if (static_cast<int>(threadIdx.x) < head) o[threadIdx.x] = op_from<T>(op_f32(p[threadIdx.x]) * coef);
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  uint4* r = reinterpret_cast<uint4*>(o + head);
  const int nv = (n - head) / VL;
  int i = threadIdx.x;
  for (; i + 3 * CLIP_THREADS < nv; i += 4 * CLIP_THREADS) {
    uint4 a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) a[u] = q[i + u * CLIP_THREADS];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[VL];
      op_unpack16<T>(a[u], f);
#pragma unroll
      for (int j = 0; j < VL; ++j) f[j] *= coef;
      r[i + u * CLIP_THREADS] = op_pack16<T>(f);
    }
  }
  for (; i < nv; i += CLIP_THREADS) {
    float f[VL];
    op_unpack16<T>(q[i], f);
#pragma unroll
    for (int j = 0; j < VL; ++j) f[j] *= coef;
    r[i] = op_pack16<T>(f);
  }
  const int done = head + nv * VL;
  if (static_cast<int>(threadIdx.x) < n - done)
    o[done + threadIdx.x] = op_from<T>(op_f32(p[done + threadIdx.x]) * coef);
}

template <int MAXT, bool MAX>
__global__ void __launch_bounds__(CLIP_THREADS)
    clip_scale_kernel(const __grid_constant__ ClipList<MAXT> l, const double* __restrict__ partial, int parts,
                      float max_norm, float* __restrict__ norm_out) {
  __shared__ double red[CLIP_THREADS / 32];
  __shared__ float s_coef;
  pdl_next();
  pdl_wait();
  // every block forms the same norm, in the same order
  double a = 0.0;
  for (int i = threadIdx.x; i < parts; i += CLIP_THREADS) {
    const double v = partial[i];
    if constexpr (MAX) a = v > a || v != v ? v : a;
    else a += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double v = __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (MAX) a = v > a || v != v ? v : a;
    else a += v;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    a = red[0];
    for (int w = 1; w < CLIP_THREADS / 32; ++w) {
      if constexpr (MAX) a = red[w] > a || red[w] != red[w] ? red[w] : a;
      else a += red[w];
    }
    const double norm = MAX ? a : sqrt(a);
    const double coef = static_cast<double>(max_norm) / (norm + 1e-6);
    // not below 1, or no number: nothing is scaled
    s_coef = isfinite(norm) && coef < 1.0 ? static_cast<float>(coef) : 1.0f;
    if (norm_out != nullptr && blockIdx.x == 0) *norm_out = static_cast<float>(norm);
  }
  __syncthreads();
  const float coef = s_coef;
  for (int b = blockIdx.x; b < l.chunks; b += gridDim.x) {
    const int c = l.chunks - 1 - b;
    const int k = clip_find(l, c);
    if (coef == 1.0f && l.in[k] == l.out[k]) continue;
    const long long at = static_cast<long long>(c - l.first[k]) * l.chunk;
    const int n = static_cast<int>(min(static_cast<long long>(l.chunk), l.n[k] - at));
    if (l.type[k] == kClipF32)
      clip_scale_chunk(static_cast<const float*>(l.in[k]) + at, static_cast<float*>(l.out[k]) + at, n, coef);
    else if (l.type[k] == kClipBF16)
      clip_scale_chunk(static_cast<const __nv_bfloat16*>(l.in[k]) + at, static_cast<__nv_bfloat16*>(l.out[k]) + at, n,
                       coef);
    else
      clip_scale_chunk(static_cast<const __half*>(l.in[k]) + at, static_cast<__half*>(l.out[k]) + at, n, coef);
  }
}

}  // namespace moe
