// Layer norm and RMS norm of rows, and their gradients.
//
// Both kernels run one block per SM.  Its threads form groups (a warp for short
// rows, up to all of them for long ones) that each walk over rows of their own;
// the rows come through a ring of shared-memory stages that bulk copies fill
// several rows ahead, so that loads stay in flight while a row's sums are formed
// and its barriers waited for.  (A block per row with the row in registers leaves
// the memory idle there: 16384 x 7168 bf16 took 115 us forward against 71 for its
// bytes.)  A thread has the same columns in all of its rows.  Layer norm of 16384 x 7168
// bf16: 92 us forward, 130 us backward, 138 in a long run of calls (5.1 and 5.4 TB/s; a copy
// reaches 6.6); RMS norm of 4097 x 5001 fp16: 21 and 50 us out of memory, 18 and 44 where a
// part is still in L2.
//
// Rows are read and written in 16-byte windows of the memory they lie in: where
// the row length is no multiple of a window, row t starts `a` elements into one,
// a = t H mod VL (VL elements a window), and window v holds the columns
// v VL - a ... + VL - 1.  The rows of a block all have the same `a` (they lie a
// multiple of VL rows apart).  The columns of such a row's first and last window,
// which its neighbours share, are taken one by one, by the first lanes of each
// group, with a row's lead.
//
// Forward: the variance is that of the centred values (no sum of squares minus
// square of sums).  Backward: x and dy are read once; the sums of dgamma and dbeta
// stay in registers, the blocks' sums go to the workspace and a second kernel adds
// them up in a fixed order.  Both are bound by memory, closely followed by their
// arithmetic: hence the packed fp32 instructions, and four windows a thread, which
// share the cost of a row's sums and barriers.
#pragma once

#include "ops_common.cuh"

namespace moe {

struct NormParams {
  const void* x;
  const void* dy;      // backward
  const float* gamma;  // may be null
  const float* beta;   // may be null (forward)
  void* out;           // y or dx
  float* mean;         // forward: may be null; backward: null for RMS norm
  float* rstd;         // forward: may be null
  float* part;         // backward: [gridDim.x][2][H], the blocks' dgamma and dbeta
  long long T;
  int H;
  float eps, inv_h;
  int rms;
  int tpg;         // threads of a group, whole warps
  int groups;      // groups of a block
  int stages;      // of a group's ring
  int row_bytes;   // of a row's windows in a stage
  int par_floats;  // of gamma (and as many of beta) in shared memory; 0: read where they lie
  long long walkers;  // gridDim.x * groups: group g of block b takes rows g gridDim.x + b, + walkers, ...
};

constexpr int kFaultNormWait = 16;
constexpr int NORM_MAX_RING = 8;
// Threads of a block, at most: 88 registers each forward, 128 backward.  (With 896
// threads in two groups the backward pass of rows of 7168 had too few registers.)
constexpr int NORM_FWD_THREADS = 704;
constexpr int NORM_BWD_THREADS = 512;

// Bulk copy of `bytes` (a multiple of 16, both ends 16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 16 bytes of shared memory.  (Through 32-bit addresses: with pointers the compiler
// spent as many instructions on addresses as on the arithmetic.)
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(addr) : "memory");
  return q;
}

// Shared memory: [groups][ring] mbarriers, [groups][2][32] float2 for the row
// sums, gamma and beta, then [groups][stages][operands] rows; the blocks' column
// sums reuse the rows.
__host__ __device__ constexpr size_t norm_head(int groups) {
  return static_cast<size_t>(groups) * (NORM_MAX_RING * 8 + 2 * 32 * 8);
}
// gamma and beta lie in shared memory by window, in the place of the block's rows;
// where a window has two quads of them, the even quads lie before the odd ones, so
// that a warp reads neighbours (in their own order each read is a two-way bank
// conflict).

// A group's place and its ring of OPS operands (x, or x and dy).
template <typename T, int OPS, int NW, bool ALIGNED, bool PAR>
struct NormRing {
  static constexpr int VL = kVec<T>;
  static_assert(ALIGNED || PAR, "unaligned parameters are read from shared memory");
  const NormParams& p;
  int g, tid, lane, warp, a;
  int v0;          // the thread's first window; the others follow 32 apart
  int col0;        // its first column
  int v_lo, v_hi;  // the row's whole windows
  int edge;        // the thread's column outside them, or -1
  uint64_t* bars;
  float2* red;
  uint8_t* ring;
  uint32_t mine;       // shared address of the thread's first window of stage 0, operand 0
  uint32_t par[2];     // and of gamma's two first quads for it
  uint32_t stage_b, op_b;  // bytes of a stage, of an operand in it
  long long first;

  __device__ __forceinline__ NormRing(const NormParams& q, uint8_t* smem) : p(q) {
    g = threadIdx.x / p.tpg;
    tid = threadIdx.x - g * p.tpg;
    lane = threadIdx.x & 31;
    warp = tid >> 5;
    bars = reinterpret_cast<uint64_t*>(smem) + g * NORM_MAX_RING;
    red = reinterpret_cast<float2*>(smem + p.groups * NORM_MAX_RING * 8) + g * 64;
    float* const par0 = reinterpret_cast<float*>(smem + norm_head(p.groups));
    op_b = p.row_bytes;
    stage_b = OPS * op_b;
    ring = reinterpret_cast<uint8_t*>(par0 + (OPS == 1 ? 2 : 1) * p.par_floats) + static_cast<size_t>(g) * p.stages * stage_b;
    first = static_cast<long long>(g) * gridDim.x + blockIdx.x;
    a = ALIGNED ? 0 : static_cast<int>(static_cast<long long>(blockIdx.x) * p.H % VL);
    v0 = warp * 32 * NW + lane;
    col0 = v0 * VL - a;
    v_lo = a > 0 ? 1 : 0;
    v_hi = (a + p.H) / VL;
    edge = -1;
    if (!ALIGNED) {
      const int c0 = v_hi > v_lo ? v_lo * VL - a : p.H, c1 = v_hi > v_lo ? v_hi * VL - a : p.H;
      const int j = tid < c0 ? tid : c1 + tid - c0;
      if (j < p.H) edge = j;
    }
    mine = smem_u32(ring) + v0 * 16;
    par[0] = smem_u32(par0 + quad(v0 * (VL / 4)));
    par[1] = smem_u32(par0 + quad(v0 * (VL / 4) + 1));
    if (tid == 0) {
      for (int i = 0; i < p.stages; ++i) mbar_init(&bars[i], 1);
      fence_mbar_init();
      long long t = first;
      for (int i = 0; i < p.stages && t < p.T; ++i, t += p.walkers) issue(t, i);
    }
    if constexpr (PAR) {
      const float* from[2] = {p.gamma, p.beta};
#pragma unroll
      for (int k = 0; k < (OPS == 1 ? 2 : 1); ++k) {
        const float none = k == 0 ? 1.f : 0.f;
#pragma unroll 4
        for (int i = threadIdx.x; i < p.par_floats / 4; i += blockDim.x) {
          const int j = 4 * i - a;
          float4 v = make_float4(none, none, none, none);
          if (from[k] != nullptr) {
            if ((a & 3) == 0 && j >= 0 && j + 4 <= p.H) {
              v = *reinterpret_cast<const float4*>(from[k] + j);
            } else {
              if (inside(j)) v.x = from[k][j];
              if (inside(j + 1)) v.y = from[k][j + 1];
              if (inside(j + 2)) v.z = from[k][j + 2];
              if (inside(j + 3)) v.w = from[k][j + 3];
            }
          }
          *reinterpret_cast<float4*>(par0 + k * p.par_floats + quad(i)) = v;
        }
      }
    }
  }
  // Place of quad i of a parameter, in floats.
  __device__ __forceinline__ int quad(int i) const {
    return VL == 4 ? 4 * i : (i & 1) * (p.par_floats / 2) + (i >> 1) * 4;
  }
  // Copies of row t's whole windows into a stage, by one thread of the group.
  __device__ __forceinline__ void issue(long long t, int stage) {
    const uint32_t bytes = v_hi > v_lo ? static_cast<uint32_t>(v_hi - v_lo) * 16u : 0u;
    mbar_arrive_expect_tx(&bars[stage], OPS * bytes);
    if (bytes != 0u) {
      const long long at = t * p.H + v_lo * VL - a;
      uint8_t* dst = ring + static_cast<size_t>(stage) * OPS * p.row_bytes + v_lo * 16;
      bulk_load(dst, static_cast<const T*>(p.x) + at, bytes, &bars[stage]);
      if constexpr (OPS == 2) bulk_load(dst + p.row_bytes, static_cast<const T*>(p.dy) + at, bytes, &bars[stage]);
    }
  }
  // The thread's edge column of row t of an operand (`none` without one).
  __device__ __forceinline__ float edge_load(const void* base, long long t, float none) const {
    return !ALIGNED && edge >= 0 && t < p.T ? op_f32(static_cast<const T*>(base)[t * p.H + edge]) : none;
  }
  __device__ __forceinline__ void bar() {
    __syncwarp();
    if (p.tpg > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(p.tpg) : "memory");
  }
  // Sum over the group, the same bits in all threads; buf: 0 and 1 in turn.
  __device__ __forceinline__ float sum(float v, int buf) {
    v = warp_sum(v);
    if (p.tpg > 32) {
      float* r = reinterpret_cast<float*>(red + buf * 32);
      if (lane == 0) r[warp] = v;
      bar();
      v = warp_sum(lane < (p.tpg >> 5) ? r[lane] : 0.f);
    }
    return v;
  }
  // Two sums over a group of at most 16 warps, in two steps with a bar() between
  // them: half the warp carries one each.
  __device__ __forceinline__ float sum2_put(float u, float v, int buf) {
    const bool low = lane < 16;
    float keep = low ? u : v;
    keep += __shfl_xor_sync(0xffffffffu, low ? v : u, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
    if (p.tpg > 32 && (lane & 15) == 0) reinterpret_cast<float*>(red + buf * 32)[(lane & 16) + warp] = keep;
    return keep;
  }
  __device__ __forceinline__ float2 sum2_get(float keep, int buf) {
    if (p.tpg > 32) {
      keep = (lane & 15) < (p.tpg >> 5) ? reinterpret_cast<const float*>(red + buf * 32)[lane] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
    }
    return make_float2(__shfl_sync(0xffffffffu, keep, 0), __shfl_sync(0xffffffffu, keep, 16));
  }
  __device__ __forceinline__ int col(int w) const { return col0 + w * 32 * VL; }  // of the thread's window w
  // Whether the thread's window w is one of the row's whole windows.
  __device__ __forceinline__ bool has(int w) const {
    const int v = v0 + w * 32;
    return (ALIGNED || v >= v_lo) && v < v_hi;
  }
  __device__ __forceinline__ bool inside(int j) const { return j >= 0 && j < p.H; }
  // window w of an operand at its shared address
  __device__ __forceinline__ void load(uint32_t addr, int w, F2* f) const { op_unpack16<T>(ld_shared16(addr + w * 512), f); }
  // `out`: the thread's first column in the row
  __device__ __forceinline__ void store(T* out, int w, const F2* f) const {
    *reinterpret_cast<uint4*>(out + w * 32 * VL) = op_pack16<T>(f);
  }
  // gamma (k = 0) or beta (1) of window w: from shared memory, or (PAR false) from
  // `q` or, without one, `none`.
  __device__ __forceinline__ void param(int k, const float* q, float none, int w, F2* f) const {
    float v[VL];
    if constexpr (!PAR) {
      if (q == nullptr) {
#pragma unroll
        for (int i = 0; i < VL; ++i) v[i] = none;
      } else {
        op_load_f32<VL>(q + col(w), v);
      }
    } else {
      // 32 windows on are 32 quads on in either half, or 32 in all (VL = 4)
      const uint32_t at = static_cast<uint32_t>(k * p.par_floats * 4 + w * 512);
      op_unpack16<float>(ld_shared16(par[0] + at), v);
      if constexpr (VL == 8) op_unpack16<float>(ld_shared16(par[1] + at), v + 4);
    }
#pragma unroll
    for (int i = 0; i < VL; i += 2) f[i / 2] = f2(v[i], v[i + 1]);
  }
};

// NW windows per thread.
template <typename T, int NW, bool ALIGNED, bool PAR>
__global__ void __launch_bounds__(NORM_FWD_THREADS, 1) norm_kernel(const NormParams p) {
  constexpr int VL = kVec<T>, NP = VL / 2;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ int abort_flag;
  if (threadIdx.x == 0) abort_flag = 0;
  pdl_next();
  pdl_wait();
  NormRing<T, 1, NW, ALIGNED, PAR> r(p, norm_smem);
  __syncthreads();
  int s = 0, buf = 0;
  uint32_t phase = 0;
  uint32_t x = r.mine;
  T* out = static_cast<T*>(p.out) + r.first * p.H + r.col0;
  const long long stride = static_cast<long long>(p.walkers) * p.H;
  const float gamma_e = !ALIGNED && r.edge >= 0 && p.gamma != nullptr ? p.gamma[r.edge] : 1.f;
  const float beta_e = !ALIGNED && r.edge >= 0 && p.beta != nullptr ? p.beta[r.edge] : 0.f;
  float xe_n = r.edge_load(p.x, r.first, 0.f);
  for (long long t = r.first; t < p.T; t += p.walkers) {
    // (a wait that gave up is recorded; the row's results are void)
    mbar_wait(&r.bars[s], phase, &abort_flag, kFaultNormWait);
    F2 v[NW][NP];
    float mean = 0.f;
    F2 acc = f2(0.f);
    const float xe = xe_n;
    xe_n = r.edge_load(p.x, t + p.walkers, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (!r.has(w)) continue;
      r.load(x, w, v[w]);
#pragma unroll
      for (int i = 0; i < NP; ++i) acc = f2_add(acc, v[w][i]);
    }
    if (!p.rms) {
      mean = r.sum(f2_sum(acc) + xe, buf) * p.inv_h;
      buf ^= 1;
    }
    acc = f2(0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (!r.has(w)) continue;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[w][i] = f2_add(v[w][i], f2(-mean));
        acc = f2_fma(v[w][i], v[w][i], acc);
      }
    }
    const float ce = !ALIGNED && r.edge >= 0 ? xe - mean : 0.f;
    const float rstd = 1.0f / sqrtf(r.sum(fmaf(ce, ce, f2_sum(acc)), buf) * p.inv_h + p.eps);
    buf ^= 1;
    if (r.tid == 0) {
      // past the last barrier the row is in registers: its stage is filled again
      const long long ahead = t + static_cast<long long>(p.stages) * p.walkers;
      if (ahead < p.T) r.issue(ahead, s);
      if (p.mean != nullptr) p.mean[t] = mean;
      if (p.rstd != nullptr) p.rstd[t] = rstd;
    }
    if (!ALIGNED && r.edge >= 0) out[r.edge - r.col0] = op_from<T>(fmaf(ce * rstd, gamma_e, beta_e));
    const F2 rs = f2(rstd);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (!r.has(w)) continue;
      F2 m[NP], b[NP];
      r.param(0, p.gamma, 1.f, w, m);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[w][i] = f2_mul(v[w][i], rs);
      if (p.beta != nullptr) {
        r.param(1, p.beta, 0.f, w, b);
#pragma unroll
        for (int i = 0; i < NP; ++i) v[w][i] = f2_fma(v[w][i], m[i], b[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) v[w][i] = f2_mul(v[w][i], m[i]);
      }
      r.store(out, w, v[w]);
    }
    x += r.stage_b;
    out += stride;
    if (++s == p.stages) {
      s = 0;
      phase ^= 1u;
      x = r.mine;
    }
  }
}

template <typename T, int NW, bool ALIGNED, bool PAR>
__global__ void __launch_bounds__(NORM_BWD_THREADS, 1) norm_backward_kernel(const NormParams p) {
  constexpr int VL = kVec<T>, NP = VL / 2;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ int abort_flag;
  if (threadIdx.x == 0) abort_flag = 0;
  pdl_next();
  pdl_wait();
  NormRing<T, 2, NW, ALIGNED, PAR> r(p, norm_smem);
  __syncthreads();
  F2 dg[NW][NP], db[NW][NP];
#pragma unroll
  for (int w = 0; w < NW; ++w)
#pragma unroll
    for (int i = 0; i < NP; ++i) dg[w][i] = db[w][i] = f2(0.f);
  int s = 0, buf = 0;
  uint32_t phase = 0;
  uint32_t x = r.mine;
  T* out = static_cast<T*>(p.out) + r.first * p.H + r.col0;
  const long long stride = static_cast<long long>(p.walkers) * p.H;
  float mean = 0.f, rstd = 0.f;
  if (r.first < p.T) {
    mean = p.rms ? 0.f : p.mean[r.first];
    rstd = p.rstd[r.first];
  }
  const float gamma_e = !ALIGNED && r.edge >= 0 && p.gamma != nullptr ? p.gamma[r.edge] : 1.f;
  float xe_n = r.edge_load(p.x, r.first, 0.f), de_n = r.edge_load(p.dy, r.first, 0.f);
  float dg_e = 0.f, db_e = 0.f;
  for (long long t = r.first; t < p.T; t += p.walkers) {
    const float xe = xe_n, de = de_n;
    xe_n = r.edge_load(p.x, t + p.walkers, 0.f);
    de_n = r.edge_load(p.dy, t + p.walkers, 0.f);
    float mean_n = 0.f, rstd_n = 0.f;
    if (t + p.walkers < p.T) {
      mean_n = p.rms ? 0.f : p.mean[t + p.walkers];
      rstd_n = p.rstd[t + p.walkers];
    }
    // (a wait that gave up is recorded; the row's results are void)
    mbar_wait(&r.bars[s], phase, &abort_flag, kFaultNormWait);
    // xh = (x - mean) rstd: the mean first, or (x rstd - mean rstd) rows far from zero
    // lose the digits that both have in common
    const F2 rs = f2(rstd), shift = f2(-mean);
    F2 a1 = f2(0.f), a2 = f2(0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (!r.has(w)) continue;
      F2 v[NP], d[NP], m[NP];
      r.load(x, w, v);
      r.load(x + r.op_b, w, d);
      r.param(0, p.gamma, 1.f, w, m);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const F2 e = f2_mul(d[i], f2_mul(f2_add(v[i], shift), rs));
        dg[w][i] = f2_add(dg[w][i], e);
        db[w][i] = f2_add(db[w][i], d[i]);
        a1 = f2_fma(d[i], m[i], a1);
        a2 = f2_fma(e, m[i], a2);
      }
    }
    float e1 = 0.f, e2 = 0.f;
    if (!ALIGNED && r.edge >= 0) {
      const float e = de * ((xe - mean) * rstd);
      dg_e += e;
      db_e += de;
      e1 = de * gamma_e;
      e2 = e * gamma_e;
    }
    const float keep = r.sum2_put(f2_sum(a1) + e1, f2_sum(a2) + e2, buf);
    r.bar();
    const float2 sums = r.sum2_get(keep, buf);
    buf ^= 1;
    // past this barrier the group is done with the row before: its stage is filled again
    if (r.tid == 0 && p.stages > 1 && t != r.first) {
      const long long ahead = t + static_cast<long long>(p.stages - 1) * p.walkers;
      if (ahead < p.T) r.issue(ahead, s == 0 ? p.stages - 1 : s - 1);
    }
    // dx = rstd (dy gamma - s1 - xh s2) = (rstd gamma) dy + k1 (x - mean) + k0
    const float s1 = p.rms ? 0.f : sums.x * p.inv_h, s2 = sums.y * p.inv_h;
    const float k1e = -rstd * rstd * s2, k0e = -rstd * s1;
    const F2 k1 = f2(k1e), k0 = f2(k0e);
    if (!ALIGNED && r.edge >= 0) out[r.edge - r.col0] = op_from<T>(fmaf(de, gamma_e * rstd, fmaf(xe - mean, k1e, k0e)));
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (!r.has(w)) continue;
      F2 v[NP], d[NP], m[NP];
      r.load(x, w, v);
      r.load(x + r.op_b, w, d);
      r.param(0, p.gamma, 1.f, w, m);
#pragma unroll
      for (int i = 0; i < NP; ++i) d[i] = f2_fma(d[i], f2_mul(m[i], rs), f2_fma(f2_add(v[i], shift), k1, k0));
      r.store(out, w, d);
    }
    if (p.stages == 1) {
      r.bar();
      if (r.tid == 0 && t + p.walkers < p.T) r.issue(t + p.walkers, 0);
    }
    mean = mean_n;
    rstd = rstd_n;
    x += r.stage_b;
    out += stride;
    if (++s == p.stages) {
      s = 0;
      phase ^= 1u;
      x = r.mine;
    }
  }

  // the groups' sums side by side in the memory of the rows (every copy has been
  // waited for), then added in group order
  float* part = p.part + static_cast<long long>(blockIdx.x) * 2 * p.H;
  float* acc = part;
  if (p.groups > 1) {
    __syncthreads();
    acc = reinterpret_cast<float*>(norm_smem + norm_head(p.groups)) + p.par_floats + static_cast<size_t>(r.g) * 2 * p.H;
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (!r.has(w)) continue;
#pragma unroll
    for (int i = 0; i < VL; i += 2) {
      const int j = r.col(w) + i;
      const float2 e = f2_get(dg[w][i / 2]), d = f2_get(db[w][i / 2]);
      if (ALIGNED) {
        *reinterpret_cast<float2*>(acc + j) = e;
        *reinterpret_cast<float2*>(acc + p.H + j) = d;
      } else {
        acc[j] = e.x, acc[p.H + j] = d.x;
        acc[j + 1] = e.y, acc[p.H + j + 1] = d.y;
      }
    }
  }
  if (!ALIGNED && r.edge >= 0) acc[r.edge] = dg_e, acc[p.H + r.edge] = db_e;
  if (p.groups > 1) {
    __syncthreads();
    const float* all = reinterpret_cast<const float*>(norm_smem + norm_head(p.groups)) + p.par_floats;
    for (int c = threadIdx.x; c < 2 * p.H; c += blockDim.x) {
      float v = 0.f;
      for (int g = 0; g < p.groups; ++g) v += all[static_cast<size_t>(g) * 2 * p.H + c];
      part[c] = v;
    }
  }
}

// Sum of column c of part[parts][width], in order within each of 16 slices, then
// over the slices: columns [0, H) go to a_out, the others to b_out (either may
// be null).  Four columns a thread where the width allows (W = 4).
constexpr int COLSUM_SLICES = 16;

template <int W>
__global__ void __launch_bounds__(32 * COLSUM_SLICES)
    column_sum_kernel(const float* __restrict__ part, int parts, int width, int H, float* __restrict__ a_out,
                      float* __restrict__ b_out) {
  __shared__ float red[COLSUM_SLICES][32 * W];
  pdl_next();
  pdl_wait();
  const int c = (blockIdx.x * 32 + threadIdx.x) * W;
  float a[W];
#pragma unroll
  for (int i = 0; i < W; ++i) a[i] = 0.f;
  if (c < width) {
    constexpr int kBatch = 10;  // loads in flight
    for (int k0 = threadIdx.y; k0 < parts; k0 += kBatch * COLSUM_SLICES) {
      float v[kBatch][W];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + u * COLSUM_SLICES;
#pragma unroll
        for (int i = 0; i < W; ++i) v[u][i] = 0.f;
        if (k < parts) op_load_f32<W>(part + static_cast<long long>(k) * width + c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int i = 0; i < W; ++i) a[i] += v[u][i];
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) red[threadIdx.y][threadIdx.x * W + i] = a[i];
  __syncthreads();
  for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * W; i += 32 * COLSUM_SLICES) {
    const int col = blockIdx.x * 32 * W + i;
    if (col >= width) break;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < COLSUM_SLICES; ++k) v += red[k][i];
    if (col < H) {
      if (a_out != nullptr) a_out[col] = v;
    } else if (b_out != nullptr) {
      b_out[col - H] = v;
    }
  }
}

}  // namespace moe
