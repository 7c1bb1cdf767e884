// Layer norm and RMS norm of rows, and their gradients.
//
// Forward: a row stays in registers between its one read and its one write, so
// the variance is that of the centred values (no sum of squares minus square of
// sums).  Rows of at most 128 16-byte vectors take a warp each, longer ones a
// block.  Bound by the read and the write.
//
// Backward: a block keeps its columns of dgamma and dbeta in registers while it
// walks over rows, writes them to the workspace once, and a second kernel adds
// up the blocks' parts in a fixed order; x and dy are read once.
#pragma once

#include "ops_common.cuh"

namespace moe {

struct NormParams {
  const void* x;
  const float* gamma;  // may be null
  const float* beta;   // may be null
  void* y;
  float* mean;  // may be null
  float* rstd;  // may be null
  long long T;
  int H;
  float eps, inv_h;
  int rms;
};

constexpr int NORM_WARP_ROWS = 4;  // rows (warps) per block where a warp takes a row

// Sum over the threads of a row (a warp or the block), the same bits in all of them.
template <bool WARP>
__device__ __forceinline__ float norm_row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (!WARP) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = warp_sum(lane < nw ? red[lane] : 0.f);
  }
  return v;
}

// NV loads of VL elements per thread of the row.
template <typename T, int VL, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * NORM_WARP_ROWS : 1024) norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int tpr = WARP ? 32 : blockDim.x;
  const long long t = WARP ? static_cast<long long>(blockIdx.x) * NORM_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.T) return;  // whole warps (WARP) only
  const T* x = static_cast<const T*>(p.x) + t * p.H;
  T* y = static_cast<T*>(p.y) + t * p.H;
  const int nvec = p.H / VL;
  float v[NV][VL];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * tpr;
    if (c < nvec) {
      op_load<T, VL>(x + static_cast<long long>(c) * VL, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VL; ++j) v[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < VL; ++j) sum += v[i][j];
  }
  float mean = 0.f;
  if (!p.rms) mean = norm_row_sum<WARP>(sum, red[0]) * p.inv_h;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = tid + i * tpr < nvec;
#pragma unroll
    for (int j = 0; j < VL; ++j) {
      v[i][j] -= mean;
      if (in) sq = fmaf(v[i][j], v[i][j], sq);
    }
  }
  const float rstd = 1.0f / sqrtf(norm_row_sum<WARP>(sq, red[1]) * p.inv_h + p.eps);
  if (tid == 0) {
    if (p.mean != nullptr) p.mean[t] = mean;
    if (p.rstd != nullptr) p.rstd[t] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * tpr;
    if (c >= nvec) continue;
    float g[VL], b[VL];
#pragma unroll
    for (int j = 0; j < VL; ++j) g[j] = 1.f, b[j] = 0.f;
    if (p.gamma != nullptr) op_load_f32<VL>(p.gamma + c * VL, g);
    if (p.beta != nullptr) op_load_f32<VL>(p.beta + c * VL, b);
#pragma unroll
    for (int j = 0; j < VL; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[j], b[j]);
    op_store<T, VL>(y + static_cast<long long>(c) * VL, v[i]);
  }
}

// ------------------------------------------------------------------------------ backward
struct NormBwdParams {
  const void* dy;
  const void* x;
  const float* gamma;  // may be null
  const float* mean;   // null for RMS norm
  const float* rstd;
  void* dx;
  float* part;  // [gridDim.x][2][H]: the blocks' dgamma and dbeta
  long long T;
  int H;
  float inv_h;
};

// Rows are taken by groups of tpr threads (a warp, or the whole block), block b
// taking rows b * groups + group + i * gridDim.x * groups.
template <typename T, int VL, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) norm_backward_kernel(const NormBwdParams p) {
  __shared__ float2 red[2][32];
  extern __shared__ float norm_acc[];  // WARP: [2][H]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = WARP ? blockDim.x >> 5 : 1;
  const int tid = WARP ? lane : threadIdx.x;
  const int tpr = WARP ? 32 : blockDim.x;
  const int nvec = p.H / VL;
  const bool rms = p.mean == nullptr;
  float dg[NV][VL], db[NV][VL], gm[NV][VL];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * tpr;
#pragma unroll
    for (int j = 0; j < VL; ++j) dg[i][j] = 0.f, db[i][j] = 0.f, gm[i][j] = 1.f;
    if (p.gamma != nullptr && c < nvec) op_load_f32<VL>(p.gamma + c * VL, gm[i]);
  }
  int buf = 0;
  for (long long t = static_cast<long long>(blockIdx.x) * groups + (WARP ? warp : 0); t < p.T;
       t += static_cast<long long>(gridDim.x) * groups) {
    const T* x = static_cast<const T*>(p.x) + t * p.H;
    const T* dy = static_cast<const T*>(p.dy) + t * p.H;
    T* dx = static_cast<T*>(p.dx) + t * p.H;
    const float mean = rms ? 0.f : p.mean[t], rstd = p.rstd[t];
    float xh[NV][VL], g[NV][VL];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * tpr;
      if (c < nvec) {
        op_load<T, VL>(x + static_cast<long long>(c) * VL, xh[i]);
        op_load<T, VL>(dy + static_cast<long long>(c) * VL, g[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VL; ++j) xh[i][j] = mean, g[i][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        xh[i][j] = (xh[i][j] - mean) * rstd;
        dg[i][j] = fmaf(g[i][j], xh[i][j], dg[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= gm[i][j];
        s1 += g[i][j];
        s2 = fmaf(g[i][j], xh[i][j], s2);
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (!WARP) {
      // two buffers: one barrier per row
      if (lane == 0) red[buf][warp] = make_float2(s1, s2);
      __syncthreads();
      const float2 r = lane < (tpr >> 5) ? red[buf][lane] : make_float2(0.f, 0.f);
      s1 = warp_sum(r.x);
      s2 = warp_sum(r.y);
      buf ^= 1;
    }
    s1 = rms ? 0.f : s1 * p.inv_h;
    s2 *= p.inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * tpr;
      if (c >= nvec) continue;
#pragma unroll
      for (int j = 0; j < VL; ++j) g[i][j] = rstd * (g[i][j] - s1 - xh[i][j] * s2);
      op_store<T, VL>(dx + static_cast<long long>(c) * VL, g[i]);
    }
  }
  float* part = p.part + static_cast<long long>(blockIdx.x) * 2 * p.H;
  if constexpr (WARP) {
    // the warps' sums in warp order
    for (int w = 0; w < groups; ++w) {
      if (warp == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = tid + i * tpr;
          if (c >= nvec) continue;
#pragma unroll
          for (int j = 0; j < VL; ++j) {
            float* a = norm_acc + c * VL + j;
            a[0] = w == 0 ? dg[i][j] : a[0] + dg[i][j];
            a[p.H] = w == 0 ? db[i][j] : a[p.H] + db[i][j];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * p.H; c += blockDim.x) part[c] = norm_acc[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * tpr;
      if (c >= nvec) continue;
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        part[c * VL + j] = dg[i][j];
        part[p.H + c * VL + j] = db[i][j];
      }
    }
  }
}

// Sum of column c of part[parts][width], in order within each of 32 slices, then
// over the slices: columns [0, H) go to a_out, the others to b_out (either may
// be null).
__global__ void __launch_bounds__(1024)
    column_sum_kernel(const float* __restrict__ part, int parts, int width, int H, float* __restrict__ a_out,
                      float* __restrict__ b_out) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < width)
    for (int i = threadIdx.y; i < parts; i += 32) a += part[static_cast<long long>(i) * width + c];
  red[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  a = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < width) {
    if (col < H) {
      if (a_out != nullptr) a_out[col] = a;
    } else if (b_out != nullptr) {
      b_out[col - H] = a;
    }
  }
}

}  // namespace moe
