// Global norm over many tensors, and clipping: one pass that adds up squares
// (or takes the largest magnitude) into one fp64 partial per block, and one that
// reads the partials, forms the factor and scales.  Both are bound by memory;
// the second walks the chunks backwards, so that what the first read last is
// still in L2.  In the first a block takes a run of chunks that follow one another
// and so looks at few entries of the list, which is slow to index; in the second
// chunks are dealt out in turn, which the writes prefer (for 322M fp32 gradients
// 205 against 238 us in the first pass, 445 against 490 in the second).  Whole vectors
// go without bounds, a chunk's last round with all of its loads at once.  Together 613 to
// 651 us for the 322M gradients in 393 tensors, about a third and two thirds (5.9 to 6.3 TB/s).
//
// The tensor list travels in the kernel's parameters (at most CLIP_MAX tensors
// a launch), so a captured graph holds it and nothing has to be copied.
#pragma once

#include "ops_common.cuh"

namespace moe {

constexpr int CLIP_THREADS = 256;
constexpr int CLIP_LOADS = 8;  // in flight a thread
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
  int chunk;  // 16-byte vectors of a chunk; chunks start at whole vectors of the input's memory
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

// The tensor of the chunk at hand.
template <int MAXT>
struct ClipCursor {
  const ClipList<MAXT>& l;
  int k = -1, lo = 0, hi = 0;  // tensor, its chunks [lo, hi)
  const void* in = nullptr;
  void* out = nullptr;
  long long n = 0;
  int type = 0;
  __device__ __forceinline__ explicit ClipCursor(const ClipList<MAXT>& list) : l(list) {}
  __device__ __forceinline__ void seek(int c) {
    if (c >= lo && c < hi) return;
    k = c == hi && k >= 0 ? k + 1 : clip_find(l, c);
    lo = l.first[k];
    hi = k + 1 < l.count ? l.first[k + 1] : l.chunks;
    in = l.in[k];
    out = l.out[k];
    n = l.n[k];
    type = l.type[k];
  }
};

// The chunks of block b of nb: [first, second).
__device__ __forceinline__ int2 clip_share(int chunks, int b, int nb) {
  return make_int2(static_cast<int>(static_cast<long long>(chunks) * b / nb),
                   static_cast<int>(static_cast<long long>(chunks) * (b + 1) / nb));
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

// Elements before p in its 16-byte vector.
template <typename T>
__device__ __forceinline__ int clip_skew(const T* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / static_cast<int>(sizeof(T));
}

template <int V>
struct ClipWidth {
  static constexpr int value = V;
};

// Calls take(elements, how many, index) for the elements of vectors [v0, v0 + nv) of
// a tensor of n elements at p, counted from the vector that p lies in.
template <typename T, typename F>
__device__ __forceinline__ void clip_chunk(const T* p, long long n, long long v0, int nv, F take) {
  constexpr int VL = kVec<T>;
  const int skew = clip_skew(p);
  const T* base = p - skew;  // (only dereferenced inside the tensor)
  const long long end = n + skew;
  // the chunk's whole vectors
  const long long lo = v0 == 0 && skew > 0 ? 1 : v0;
  const int count = static_cast<int>(min(v0 + nv, end / VL) - lo);
  const uint4* q = reinterpret_cast<const uint4*>(base) + lo;
  const long long e0 = lo * VL - skew;
  int i = threadIdx.x;
  for (; i + (CLIP_LOADS - 1) * CLIP_THREADS < count; i += CLIP_LOADS * CLIP_THREADS) {
    uint4 a[CLIP_LOADS];
#pragma unroll
    for (int u = 0; u < CLIP_LOADS; ++u) a[u] = q[i + u * CLIP_THREADS];
#pragma unroll
    for (int u = 0; u < CLIP_LOADS; ++u) {
      float f[VL];
      op_unpack16<T>(a[u], f);
      take(f, ClipWidth<VL>(), e0 + (i + u * CLIP_THREADS) * VL);
    }
  }
  if (i < count) {
    // the last round: all loads at once here too, what lies behind the end is not used
    uint4 a[CLIP_LOADS];
#pragma unroll
    for (int u = 0; u < CLIP_LOADS; ++u) a[u] = q[min(i + u * CLIP_THREADS, count - 1)];
#pragma unroll
    for (int u = 0; u < CLIP_LOADS; ++u) {
      if (i + u * CLIP_THREADS >= count) break;
      float f[VL];
      op_unpack16<T>(a[u], f);
      take(f, ClipWidth<VL>(), e0 + (i + u * CLIP_THREADS) * VL);
    }
  }
  // the elements of cut vectors: the tensor's first, in its first chunk, and its last,
  // in the chunk they lie in (a tensor inside one vector: in the first alone)
  if (threadIdx.x < 2 * VL) {
    const int j = threadIdx.x & (VL - 1);
    const long long v = threadIdx.x < VL ? 0 : end / VL;
    const long long e = v * VL + j;
    const bool cut = threadIdx.x < VL ? skew > 0 : end % VL != 0 && (v > 0 || skew == 0);
    if (cut && v >= v0 && v < v0 + nv && e >= skew && e < end) {
      const float f = op_f32(base[e]);
      take(&f, ClipWidth<1>(), e - skew);
    }
  }
}

template <typename T, bool MAX>
__device__ __forceinline__ void clip_reduce_chunk(const void* p, long long n, long long v0, int nv, double& sum, uint32_t& top) {
  clip_chunk(static_cast<const T*>(p), n, v0, nv, [&](const float* f, auto vl, long long) {
    constexpr int W = decltype(vl)::value;
    if constexpr (MAX) {
      // magnitudes as integers: a NaN is above everything and stays
#pragma unroll
      for (int i = 0; i < W; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    } else {
      sum += clip_squares<T, W>(f);
    }
  });
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
  ClipCursor<MAXT> cur(l);
  const int2 share = clip_share(l.chunks, blockIdx.x, gridDim.x);
  for (int c = share.x; c < share.y; ++c) {
    cur.seek(c);
    const long long v0 = static_cast<long long>(c - cur.lo) * l.chunk;
    if (cur.type == kClipF32)
      clip_reduce_chunk<float, MAX>(cur.in, cur.n, v0, l.chunk, sum, top);
    else if (cur.type == kClipBF16)
      clip_reduce_chunk<__nv_bfloat16, MAX>(cur.in, cur.n, v0, l.chunk, sum, top);
    else
      clip_reduce_chunk<__half, MAX>(cur.in, cur.n, v0, l.chunk, sum, top);
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
__device__ __forceinline__ void clip_scale_chunk(const void* p, void* out, long long n, long long v0, int nv, float2 coef) {
  T* o = static_cast<T*>(out);
  // one alignment for both: whole vectors are written as such
  const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0u;
  clip_chunk(static_cast<const T*>(p), n, v0, nv, [&](const float* f, auto vl, long long at) {
    constexpr int W = decltype(vl)::value;
    float g[W];
#pragma unroll
    for (int j = 0; j < W; ++j) g[j] = (f[j] * coef.x) * coef.y;
    if (W > 1 && same) {
      if constexpr (W > 1) *reinterpret_cast<uint4*>(o + at) = op_pack16<T>(g);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) o[at + j] = op_from<T>(g[j]);
    }
  });
}

template <int MAXT, bool MAX>
__global__ void __launch_bounds__(CLIP_THREADS)
    clip_scale_kernel(const __grid_constant__ ClipList<MAXT> l, const double* __restrict__ partial, int parts,
                      float max_norm, float* __restrict__ norm_out) {
  __shared__ double red[CLIP_THREADS / 32];
  __shared__ float2 s_coef;
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
    const float norm32 = static_cast<float>(norm);
    const double coef = static_cast<double>(max_norm) / (norm + 1e-6);
    // not below 1, or a norm that is no fp32 number: nothing is scaled.  A factor below
    // the smallest normal number (gradients near the largest ones) goes in two steps,
    // the second of them 2^-64, or its digits would be lost.
    const bool small = coef < 0x1p-126;
    s_coef = isfinite(norm32) && coef < 1.0
                 ? make_float2(static_cast<float>(small ? coef * 0x1p64 : coef), small ? 0x1p-64f : 1.0f)
                 : make_float2(1.0f, 1.0f);
    if (norm_out != nullptr && blockIdx.x == 0) *norm_out = norm32;
  }
  __syncthreads();
  const float2 coef = s_coef;
  ClipCursor<MAXT> cur(l);
  for (int c = l.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    cur.seek(c);
    if (coef.x == 1.0f && cur.in == cur.out) continue;
    const long long v0 = static_cast<long long>(c - cur.lo) * l.chunk;
    if (cur.type == kClipF32)
      clip_scale_chunk<float>(cur.in, cur.out, cur.n, v0, l.chunk, coef);
    else if (cur.type == kClipBF16)
      clip_scale_chunk<__nv_bfloat16>(cur.in, cur.out, cur.n, v0, l.chunk, coef);
    else
      clip_scale_chunk<__half>(cur.in, cur.out, cur.n, v0, l.chunk, coef);
  }
}

}  // namespace moe
