// Dense products with an epilogue on the tensor cores, forward and backward:
//
//   out[q, p] = f( sum_r Q(q, r) * P(p, r) )        p contiguous in out
//
//   y  = act(x W^T + b) + res:  q = token, p = weight row,     r = feature
//   dx = dp W:                  q = token, p = feature,        r = weight row
//   dW = dp^T x:                q = weight row, p = feature,   r = token
//
// Each operand is either r-contiguous ("K-major": x, W and dp as they lie) or
// contiguous along its own rows ("MN-major": W for dx, dp and x for dW); both
// come by TMA with the 128-byte swizzle and need no transposed copy:
//   K-major   boxes of 64 r x n rows; 8-row groups 1024 bytes apart
//   MN-major  boxes of 64 rows x 64 r, 128 bytes a step of r; 64-row boxes 8192
//             bytes apart
// Tails of every dimension are the zeros that TMA fills in.
//
// linear_wide_kernel: CTA pairs (tcgen05.mma.cta_group::2, 256 x BN tiles, BN a
// multiple of 32 up to 256), persistent, two accumulators in tensor memory so
// that a tile's epilogue runs under the next one's products.  For large
// products; bound by the tensor cores and, close behind, by what the SMs can
// fetch from L2 (a narrower tile costs nearly as much a k-block as a wide one).
// The tiles of a last, partly filled wave are split along r over all the pairs;
// their fp32 partial sums go to the workspace and linear_fixup_kernel adds them
// up in order and finishes those tiles.  8192 x 7168 x 3584 bf16 with bias, residual and
// gelu: 315 us (1.34 PFLOP/s) at the burst clock, 369 us under the power cap; the library's
// plain product alone 286 and 330 us.
//
// linear_skinny_kernel: P on the MMA's 128-row side and at most 128 rows of Q
// beside it, the sum over r split over the CTAs of a cluster, which add up each
// other's partial sums through distributed shared memory in rank order.  For
// few rows, where the read of P bounds the call and a 256-row tile would be
// mostly padding, and for outputs too small to fill the machine.  4 x 7168 x 3584: 13.4 us,
// 51 MB of weights in 7.8 at the copy's rate.
#pragma once

#include "gemm_expert.cuh"
#include "ops_common.cuh"

namespace moe {

constexpr int LIN_BK = 64;
constexpr uint32_t LIN_BOX_MN = 64 * LIN_BK * 2;  // bytes of an MN-major box

// Descriptor of an MN-major tile in the layout above.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(LIN_BOX_MN >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) |
         (static_cast<uint64_t>(2u) << 61);
}

// Instruction descriptor of kind::f16 with fp32 accumulation: operand format
// (0 f16, 1 bf16; the same for both), transpose bits 15 (A) and 16 (B) for
// MN-major operands.
__host__ __device__ constexpr uint32_t lin_idesc(int M, int N, bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

enum LinAct : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// Hardware reciprocal (within 1 ulp) and 2^x (within 2 ulp + that of x); results
// below 2^-126 are 0.
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2E = 1.4426950408889634f;

// sigmoid: relative error below 2^-23 (4 + 1.2 |a|); 0 below a = -87.3 (the value is
// under 2^-126 there).
__device__ __forceinline__ float lin_sigmoid(float a) { return rcp_fast(1.0f + ex2_fast(-kLog2E * a)); }

constexpr float kSqrt2OverPi = 0.7978845608028654f;

// erfc(x) = e^(-x^2) t P(t), t = 1 / (1 + 0.375 x), at x = |a| / sqrt 2, with a polynomial
// fitted for the least relative error over 0 <= x <= 9.5 (weighted least squares,
// the weights moved to the largest errors until these were level): 6.4e-7.  Fewer
// instructions than erff's, and no branch.  (The bound has to be relative: gelu's values are
// small where a is negative.  Five terms with an absolute error of 1.5e-7 are off by 5e-4
// of the value at a = -4.)
constexpr float kErfcX = 0.375f * 0.7071067811865476f;
constexpr float kErfc0 = 0.21133945f, kErfc1 = 0.21568917f, kErfc2 = 0.16666461f, kErfc3 = 0.28306143f, kErfc4 = -0.12959715f,
                kErfc5 = 0.38793772f, kErfc6 = -0.13509587f;
// *e receives the exponential.
__device__ __forceinline__ float lin_erfc_abs(float a, float* e) {
  const float t = rcp_fast(fmaf(kErfcX, fabsf(a), 1.0f));
  *e = ex2_fast(a * (a * (-0.5f * kLog2E)));
  const float hi = fmaf(fmaf(fmaf(kErfc6, t, kErfc5), t, kErfc4), t, kErfc3);
  const float q = fmaf(fmaf(fmaf(hi, t, kErfc2), t, kErfc1), t, kErfc0);
  return q * t * *e;
}

// a Phi(a) = max(a, 0) - |a| erfc(|a| / sqrt 2) / 2, on both sides of 0, of two values
// at once (ten instructions a value: what the epilogue's warps issue beside the
// product's is seen in its time).  Beyond 100 erfc is 0, and no infinity meets it; a
// NaN stays one.
__device__ __forceinline__ void lin_gelu2(float& a, float& b) {
  const F2 v = f2(a, b);
  const F2 t = f2(rcp_fast(fmaf(kErfcX, fabsf(a), 1.0f)), rcp_fast(fmaf(kErfcX, fabsf(b), 1.0f)));
  const float2 x = f2_get(f2_mul(v, f2_mul(v, f2(-0.5f * kLog2E))));
  const F2 e = f2(ex2_fast(x.x), ex2_fast(x.y));
  F2 q = f2(-0.5f * kErfc6);
  q = f2_fma(q, t, f2(-0.5f * kErfc5));
  q = f2_fma(q, t, f2(-0.5f * kErfc4));
  q = f2_fma(q, t, f2(-0.5f * kErfc3));
  q = f2_fma(q, t, f2(-0.5f * kErfc2));
  q = f2_fma(q, t, f2(-0.5f * kErfc1));
  q = f2_fma(q, t, f2(-0.5f * kErfc0));
  q = f2_mul(f2_mul(q, t), e);
  const float2 y = f2_get(f2_fma(f2(fminf(fabsf(a), 100.f), fminf(fabsf(b), 100.f)), q, f2(fmaxf(a, 0.f), fmaxf(b, 0.f))));
  a = y.x;
  b = y.y;
}

// a sigmoid(a (k1 + k2 a^2)) of two values at once: silu with k = (1, 0), and gelu's tanh
// form, (1 + tanh u) / 2 being sigmoid(2 u).
__device__ __forceinline__ void lin_gate2(float& a, float& b, float k1, float k2) {
  const F2 v = f2(a, b);
  const F2 k = k2 == 0.f ? f2(-kLog2E * k1) : f2_fma(f2_mul(v, v), f2(-kLog2E * k2), f2(-kLog2E * k1));
  const float2 x = f2_get(f2_mul(v, k));
  const float2 d = f2_get(f2_add(f2(ex2_fast(x.x), ex2_fast(x.y)), f2(1.f)));
  const float2 y = f2_get(f2_mul(v, f2(rcp_fast(d.x), rcp_fast(d.y))));
  a = y.x;
  b = y.y;
}
constexpr float kTanh1 = 2.f * kSqrt2OverPi, kTanh2 = kTanh1 * 0.044715f;

__device__ __forceinline__ float lin_act(float a, int act) {
  switch (act) {
    case kActRelu:
      return a > 0.f ? a : (a == a ? 0.f : a);
    case kActSilu:
      return a * lin_sigmoid(a);
    case kActGelu: {
      float other = 0.f;
      lin_gelu2(a, other);
      return a;
    }
    case kActGeluTanh: {
      float other = 0.f;
      lin_gate2(a, other, kTanh1, kTanh2);
      return a;
    }
    default:
      return a;
  }
}

__device__ __forceinline__ float lin_act_grad(float a, int act) {
  // beyond 100 every slope is 0 or 1 to the last bit; no infinity meets a 0 there
  if (fabsf(a) > 100.f) return act == kActNone ? 1.f : a > 0.f ? 1.f : 0.f;
  switch (act) {
    case kActRelu:
      return a > 0.f ? 1.f : 0.f;
    case kActSilu: {
      const float s = lin_sigmoid(a);
      return s * (1.0f + a * (1.0f - s));
    }
    case kActGelu: {
      float e;
      const float c = 0.5f * lin_erfc_abs(a, &e);
      return (a > 0.f ? 1.0f - c : c) + a * 0.3989422804014327f * e;
    }
    case kActGeluTanh: {
      const float s = lin_sigmoid(2.f * kSqrt2OverPi * (a + 0.044715f * a * a * a));
      return s + a * 2.f * s * (1.f - s) * kSqrt2OverPi * (1.f + 3.f * 0.044715f * a * a);
    }
    default:
      return 1.f;
  }
}

struct LinMaps {
  CUtensorMap p, q;
  // wide, 16-bit outputs: boxes of 32 x 32 of out, residual and pre
  CUtensorMap out, res, pre;
};

struct LinParams {
  long long Q;
  int P, nkb;       // contraction blocks of 64
  int p_mn, q_mn;   // operand layouts
  int bf16;         // operand type: bf16 or f16
  int p_tiles, q_tiles, bn;  // wide: bn columns (P) a tile; skinny: bn rows (Q) a tile
  const float* bias;         // [P] or null
  const void* residual;      // [Q, P] in the type of out, or null
  void* pre;                 // [Q, P] in the operand type, or null
  void* out;
  int act;
  int fault_site;
  // wide: the first `full` tiles whole, each later one in `split` parts, whose sums go
  // to partial[part][bn / 4][256][4]
  int full, split;
  float* partial;
};

// bias, pre, activation and residual of NC consecutive outputs of a row (NC a
// multiple of 4; 16-bit types in 8-byte, or for NC = 32 in 16-byte accesses).
template <typename OutT, int NC>
__device__ __forceinline__ void lin_finish(const LinParams& p, long long q, int col, float* a) {
  const long long at = q * p.P + col;
  if (p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + col + i));
      a[i] += b.x;
      a[i + 1] += b.y;
      a[i + 2] += b.z;
      a[i + 3] += b.w;
    }
  }
  if (p.pre != nullptr) {
    uint2* d = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.pre) + at);
#pragma unroll
    for (int i = 0; i < NC; i += 4)
      d[i / 4] = p.bf16 ? make_uint2(op_pack(a[i], a[i + 1], __nv_bfloat16()), op_pack(a[i + 2], a[i + 3], __nv_bfloat16()))
                        : make_uint2(op_pack(a[i], a[i + 1], __half()), op_pack(a[i + 2], a[i + 3], __half()));
  }
  if (p.act != kActNone) {
#pragma unroll
    for (int i = 0; i < NC; ++i) a[i] = lin_act(a[i], p.act);
  }
  OutT* out = static_cast<OutT*>(p.out) + at;
  const OutT* res = static_cast<const OutT*>(p.residual) + at;
  constexpr int W = sizeof(OutT) == 4 ? 4 : NC % 8 == 0 ? 8 : 4;  // outputs per access
#pragma unroll
  for (int i = 0; i < NC; i += W) {
    if constexpr (sizeof(OutT) == 4) {
      if (p.residual != nullptr) {
        const float4 r = *reinterpret_cast<const float4*>(res + i);
        a[i] += r.x;
        a[i + 1] += r.y;
        a[i + 2] += r.z;
        a[i + 3] += r.w;
      }
      *reinterpret_cast<float4*>(out + i) = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
    } else if constexpr (W == 8) {
      if (p.residual != nullptr) {
        float r[8];
        op_unpack16<OutT>(*reinterpret_cast<const uint4*>(res + i), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[i + j] += r[j];
      }
      *reinterpret_cast<uint4*>(out + i) = op_pack16<OutT>(a + i);
    } else {
      if (p.residual != nullptr) {
        const uint2 u = *reinterpret_cast<const uint2*>(res + i);
        const float2 r0 = op_unpack(u.x, OutT()), r1 = op_unpack(u.y, OutT());
        a[i] += r0.x;
        a[i + 1] += r0.y;
        a[i + 2] += r1.x;
        a[i + 3] += r1.y;
      }
      *reinterpret_cast<uint2*>(out + i) = make_uint2(op_pack(a[i], a[i + 1], OutT()), op_pack(a[i + 2], a[i + 3], OutT()));
    }
  }
}

// ------------------------------------------------------------------------------ wide
constexpr int LW_STAGES = 5;
constexpr uint32_t LW_OPER_BYTES = 128 * LIN_BK * 2;  // one operand's stage in a CTA
constexpr int LW_THREADS = 32 * 10;
// An epilogue warp's boxes of 32 x 32 16-bit values: two for out (and the residual
// in its place), two for pre.
constexpr uint32_t LW_BOX = 32 * 32 * 2;
constexpr uint32_t LW_WARP_BYTES = 4 * LW_BOX;
constexpr size_t LW_SMEM = 1024 + static_cast<size_t>(LW_STAGES) * 2 * LW_OPER_BYTES + 8 * LW_WARP_BYTES + 512;
constexpr int LW_GROUP = 16;  // Q tiles that share a run of P tiles through L2

// Store of a box from shared memory; parts outside the tensor are left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}

__device__ __forceinline__ void lin_add2(float& a, float& b, F2 c) {
  const float2 y = f2_get(f2_add(f2(a, b), c));
  a = y.x;
  b = y.y;
}

// The activation of 32 values, chosen once.
__device__ __forceinline__ void lin_act32(float (&a)[32], int act) {
  switch (act) {
    case kActNone:
      break;
    case kActRelu:
#pragma unroll
      for (int i = 0; i < 32; ++i) a[i] = lin_act(a[i], kActRelu);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < 32; i += 2) lin_gate2(a[i], a[i + 1], 1.f, 0.f);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < 32; i += 2) lin_gelu2(a[i], a[i + 1]);
      break;
    default:
#pragma unroll
      for (int i = 0; i < 32; i += 2) lin_gate2(a[i], a[i + 1], kTanh1, kTanh2);
  }
}

struct LinTile {
  int q, p;
};

// Tiles in groups of LW_GROUP rows of tiles, the P tile outside and the Q tile
// inside a group: the pairs at work at one time share few operand rows.
__device__ __forceinline__ LinTile lw_tile(int w, const LinParams& p) {
  const int per = LW_GROUP * p.p_tiles;
  const int grp = w / per, r = w - grp * per;
  const int rows = min(LW_GROUP, p.q_tiles - grp * LW_GROUP);
  const int pt = r / rows;
  return {grp * LW_GROUP + (r - pt * rows), pt};
}

// Work item w: a tile and its k-blocks [kb0, kb1); part < 0: all of them.
struct LinItem {
  LinTile t;
  int kb0, kb1, part;
};
__device__ __forceinline__ LinItem lw_item(int w, const LinParams& p) {
  if (w < p.full) return {lw_tile(w, p), 0, p.nkb, -1};
  const int i = w - p.full, tile = i / p.split, k = i - tile * p.split;
  return {lw_tile(p.full + tile, p), static_cast<int>(static_cast<long long>(p.nkb) * k / p.split),
          static_cast<int>(static_cast<long long>(p.nkb) * (k + 1) / p.split), i};
}

template <typename OutT>
__global__ void __launch_bounds__(LW_THREADS, 1)
    linear_wide_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
  extern __shared__ uint8_t lw_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lw_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;                                // Q rows
  uint8_t* sB = smem + LW_STAGES * LW_OPER_BYTES;    // P rows
  uint8_t* sE = sB + LW_STAGES * LW_OPER_BYTES;      // the epilogue warps' boxes
  uint64_t* full = reinterpret_cast<uint64_t*>(sE + 8 * LW_WARP_BYTES);
  uint64_t* empty = full + LW_STAGES;
  uint64_t* acc_full = empty + LW_STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* res_full = drain + 1;                    // [8 warps][2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(res_full + 16);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int total = p.full + (p.q_tiles * p.p_tiles - p.full) * p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < LW_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 16);  // the eight epilogue warps of both CTAs
    }
    for (int i = 0; i < 16; ++i) mbar_init(&res_full[i], 1);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.p);
    tma_prefetch_desc(&maps.q);
  }
  if (warp == 1) ex_tmem_alloc<2>(tmem_holder);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  pdl_next();
  pdl_wait();
  const uint32_t tmem_base = *tmem_holder;
  const int half = p.bn >> 1;  // P rows that this CTA stages

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0u, issued_parity = 0u;
      bool ok = true;
      const int p_boxes = (half + 63) >> 6;
      const uint32_t bytes = 2u * (LW_OPER_BYTES + (p.p_mn ? p_boxes * LIN_BOX_MN : static_cast<uint32_t>(half) * 128u));
      for (int w = pair; w < total && ok; w += npairs) {
        const LinItem it = lw_item(w, p);
        const int q0 = it.t.q * 256 + static_cast<int>(rank) * 128;
        const int p0 = it.t.p * p.bn + static_cast<int>(rank) * half;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort, p.fault_site + 1)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const int kc = kb * LIN_BK;
          uint8_t* a_dst = sA + stage * LW_OPER_BYTES;
          uint8_t* b_dst = sB + stage * LW_OPER_BYTES;
          if (p.q_mn) {
            ex_tma_load<2>(a_dst, &maps.q, &full[stage], q0, kc);
            ex_tma_load<2>(a_dst + LIN_BOX_MN, &maps.q, &full[stage], q0 + 64, kc);
          } else {
            ex_tma_load<2>(a_dst, &maps.q, &full[stage], kc, q0);
          }
          if (p.p_mn) {
            for (int b = 0; b < p_boxes; ++b)
              ex_tma_load<2>(b_dst + b * LIN_BOX_MN, &maps.p, &full[stage], p0 + b * 64, kc);
          } else {
            ex_tma_load<2>(b_dst, &maps.p, &full[stage], kc, p0);
          }
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == LW_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the even CTA's barriers count both CTAs' bytes: every load lands before
      // the pair may exit
      if (leader) {
        volatile int never = 0;
        for (int s = 0; s < LW_STAGES; ++s)
          if ((issued >> s) & 1u) mbar_wait(&full[s], (issued_parity >> s) & 1u, &never, p.fault_site + 2);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && leader) {
      const uint32_t idesc = lin_idesc(256, p.bn, p.bf16 != 0, p.q_mn != 0, p.p_mn != 0);
      // an MMA takes 16 steps of r: 32 bytes of a K-major row, two 8-step groups of an MN-major tile
      const uint32_t a_step = p.q_mn ? 2048u : 32u, b_step = p.p_mn ? 2048u : 32u;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int w = pair; w < total && ok; w += npairs) {
        const LinItem it = lw_item(w, p);
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, abort, p.fault_site + 3)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort, p.fault_site + 4)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + stage * LW_OPER_BYTES);
          const uint32_t b_addr = smem_u32(sB + stage * LW_OPER_BYTES);
          const uint64_t ad = p.q_mn ? sw128_mnmajor_desc(a_addr) : sw128_kmajor_desc(a_addr);
          const uint64_t bd = p.p_mn ? sw128_mnmajor_desc(b_addr) : sw128_kmajor_desc(b_addr);
#pragma unroll
          for (int kk = 0; kk < LIN_BK / 16; ++kk)
            ex_mma<2>(d_tmem, ad + ((kk * a_step) >> 4), bd + ((kk * b_step) >> 4), idesc,
                      kb != it.kb0 || kk != 0 ? 1u : 0u);
          ex_commit<2>(&empty[stage]);
          if (++stage == LW_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ex_commit<2>(&acc_full[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      ex_commit<2>(drain);
    }
    // both CTAs: every MMA that touches this CTA's memory is done
    if (lane == 0) {
      volatile int never = 0;
      mbar_wait(drain, 0u, &never, p.fault_site + 5);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    // two sets of four warps take alternate chunks of 32 columns
    const int quarter = warp & 3;
    const int set = warp >= 6 ? 1 : 0;
    const uint32_t acc_empty_leader = map_to_rank(smem_u32(&acc_empty[0]), 0u);
    int acc = 0;
    uint32_t acc_phase = 0;
    // 16-bit outputs go through shared memory and TMA, 32 x 32 at a time, the
    // residual's box loaded one chunk ahead into the place of the output's
    // (straight from registers each lane writes a row of its own: 32 lines an
    // access, and a sixth of the whole kernel's time at 8192 x 7168 x 3584)
    constexpr bool kBoxes = sizeof(OutT) == 2;
    uint8_t* boxes = sE + (warp - 2) * LW_WARP_BYTES;
    uint64_t* res_bar = res_full + (warp - 2) * 2;
    const bool has_res = p.residual != nullptr, has_pre = p.pre != nullptr;
    int n = 0, ahead = 0;  // chunks done by this warp, residual boxes asked for
    int w_next = pair, c_next = set * 32;  // the next chunk to load a residual for
    auto chunk_row = [&](int w) { return lw_tile(w, p).q * 256 + static_cast<int>(rank) * 128 + quarter * 32; };
    // moves (w, c) to the first chunk at or after it that this warp has rows and columns in
    auto settle = [&](int& w, int& c) {
      for (; w < p.full; w += npairs, c = set * 32) {  // (parts have no residual)
        const LinTile t = lw_tile(w, p);
        if (c < p.bn && t.p * p.bn + c < p.P && chunk_row(w) < p.Q) return;
      }
    };
    auto load_res = [&](int slot) {  // one lane
      const LinTile t = lw_tile(w_next, p);
      mbar_arrive_expect_tx(&res_bar[slot], LW_BOX);
      tma_load_2d(boxes + slot * LW_BOX, &maps.res, &res_bar[slot], t.p * p.bn + c_next, chunk_row(w_next));
    };
    if (kBoxes && has_res) {
      settle(w_next, c_next);
      if (w_next < p.full) {
        if (lane == 0) load_res(0);
        ++ahead;
        c_next += 64;
        settle(w_next, c_next);
      }
    }
    for (int w = pair; w < total; w += npairs) {
      const LinItem it = lw_item(w, p);
      const LinTile t = it.t;
      // warp-uniform decision: tcgen05.ld below needs the whole warp
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase, abort, p.fault_site + 6))) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * 256);
      const int row0 = t.q * 256 + static_cast<int>(rank) * 128 + quarter * 32;
      const long long q = static_cast<long long>(row0) + lane;
#pragma unroll 1
      for (int c = set * 32; c < p.bn; c += 64) {
        const int col = t.p * p.bn + c;
        if (col >= p.P) break;  // warp-uniform
        float a[32];
        tmem_ld32(tbase + c, a);
        if (it.part >= 0) {
          // lanes (rows) beside one another, four columns each
          float4* to = reinterpret_cast<float4*>(p.partial) + static_cast<long long>(it.part) * (p.bn / 4) * 256 +
                       (c / 4) * 256 + static_cast<int>(rank) * 128 + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < 8; ++i) to[i * 256] = make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
        } else if constexpr (kBoxes) {
          if (row0 < p.Q) {  // warp-uniform
            const int slot = n & 1;
            if (lane == 0) {
              // the box of the chunk before last has been written out; with a residual
              // also the last one's, whose place the next residual takes
              if (has_res) {
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                if (w_next < p.full) load_res(slot ^ 1);
              } else {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
              }
            }
            if (has_res && w_next < p.full) {
              ++ahead;
              c_next += 64;
              settle(w_next, c_next);
            }
            __syncwarp();
            if (has_res) mbar_wait(&res_bar[slot], (n >> 1) & 1, abort, p.fault_site + 7);
            uint8_t* box = boxes + slot * LW_BOX + lane * 64;
            const int swz = (lane >> 1) & 3;  // 64-byte swizzle: 16-byte word j of row r at j ^ (r / 2 % 4)
            if (p.bias != nullptr) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                if (col + i < p.P) {
                  const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + col + i));
                  lin_add2(a[i], a[i + 1], f2(b.x, b.y));
                  lin_add2(a[i + 2], a[i + 3], f2(b.z, b.w));
                }
              }
            }
            if (has_pre) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(box + 2 * LW_BOX + ((j ^ swz) << 4)) = op_pack16<OutT>(a + 8 * j);
            }
            lin_act32(a, p.act);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4* at = reinterpret_cast<uint4*>(box + ((j ^ swz) << 4));
              if (has_res) {
                F2 r[4];
                op_unpack16<OutT>(*at, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) lin_add2(a[8 * j + 2 * i], a[8 * j + 2 * i + 1], r[i]);
              }
              *at = op_pack16<OutT>(a + 8 * j);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.out, boxes + slot * LW_BOX, col, row0);
              if (has_pre) tma_store_2d(&maps.pre, boxes + (2 + slot) * LW_BOX, col, row0);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            ++n;
          }
        } else if (q < p.Q) {
          if (col + 32 <= p.P) {
            lin_finish<OutT, 32>(p, q, col, a);
          } else {
            // P is a multiple of 8
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              if (col + i < p.P) lin_finish<OutT, 8>(p, q, col + i, a + i);
          }
        }
        __syncwarp();
      }
      __syncwarp();
      tc_fence_before();
      if (lane == 0) mbar_arrive_cluster(acc_empty_leader + static_cast<uint32_t>(acc * sizeof(uint64_t)));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    // the stores have read their boxes, and (after a wait that gave up) a residual's
    // has landed, before the memory goes
    if (ahead > n) {
      volatile int never = 0;
      mbar_wait(&res_bar[n & 1], (n >> 1) & 1, &never, p.fault_site + 8);
    }
    if (kBoxes && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  __syncwarp();  // reconverge lanes that skipped the single-thread roles
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    ex_tmem_dealloc<2>(tmem_base);
  }
}

// The tiles that linear_wide_kernel left in parts: four columns of a row a thread,
// the parts added in order.
template <typename OutT>
__global__ void __launch_bounds__(256) linear_fixup_kernel(const LinParams p) {
  pdl_next();
  pdl_wait();
  const int quads = p.bn / 4;
  const int tile = blockIdx.x / quads, cq = blockIdx.x - tile * quads, row = threadIdx.x;
  const LinTile t = lw_tile(p.full + tile, p);
  const long long q = static_cast<long long>(t.q) * 256 + row;
  const int col = t.p * p.bn + cq * 4;
  if (q >= p.Q || col >= p.P) return;
  const float4* from = reinterpret_cast<const float4*>(p.partial) + (static_cast<long long>(tile) * p.split * quads + cq) * 256 + row;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int k = 0; k < p.split; ++k) {
    const float4 v = from[static_cast<long long>(k) * quads * 256];
    a[0] += v.x;
    a[1] += v.y;
    a[2] += v.z;
    a[3] += v.w;
  }
  lin_finish<OutT, 4>(p, q, col, a);
}

// ------------------------------------------------------------------------------ skinny
constexpr int LS_THREADS = 192;
constexpr uint32_t LS_BUDGET = 108 * 1024;  // operand stages: two CTAs an SM
constexpr int LS_MAX_SPLIT = 8;

// BN rows of Q a tile; an MN-major Q takes whole boxes of 64 rows.
template <int BN, bool QMN>
struct LsCfg {
  static constexpr uint32_t kP = 128 * LIN_BK * 2;
  static constexpr uint32_t kQ = (QMN && BN < 64 ? 64 : BN) * LIN_BK * 2;
  static constexpr uint32_t kStage = kP + kQ;
  static constexpr int kStages = LS_BUDGET / kStage > 8 ? 8 : static_cast<int>(LS_BUDGET / kStage);
  static constexpr uint32_t kCols = BN < 32 ? 32 : BN;  // tensor memory columns
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + 256;
  static_assert(kStages >= 2 && BN * 128 * 4 <= kStages * kStage, "the partial sums reuse the stages");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <typename OutT, int BN, bool QMN>
__global__ void __launch_bounds__(LS_THREADS, 2)
    linear_skinny_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
  using C = LsCfg<BN, QMN>;
  extern __shared__ uint8_t ls_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ls_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = gridDim.x / p.p_tiles;  // CTAs of the cluster
  const int rank = static_cast<int>(cluster_ctarank());
  const int p0 = static_cast<int>(blockIdx.x) / split * 128;
  const long long q0 = static_cast<long long>(blockIdx.y) * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(p.nkb) * rank / split);
  const int nkb = static_cast<int>(static_cast<long long>(p.nkb) * (rank + 1) / split) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    tma_prefetch_desc(&maps.p);
    tma_prefetch_desc(&maps.q);
    mbar_init(done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_next();
  pdl_wait();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0u, issued_parity = 0u;
      constexpr uint32_t bytes = C::kP + C::kQ;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort, p.fault_site + 1)) break;
        mbar_arrive_expect_tx(&full[stage], bytes);
        const int kc = (kb0 + kb) * LIN_BK;
        uint8_t* a_dst = smem + stage * C::kStage;
        uint8_t* b_dst = a_dst + C::kP;
        if (p.p_mn) {
          tma_load_2d(a_dst, &maps.p, &full[stage], p0, kc);
          tma_load_2d(a_dst + LIN_BOX_MN, &maps.p, &full[stage], p0 + 64, kc);
        } else {
          tma_load_2d(a_dst, &maps.p, &full[stage], kc, p0);
        }
        if constexpr (QMN) {
          for (uint32_t b = 0; b < C::kQ / LIN_BOX_MN; ++b)
            tma_load_2d(b_dst + b * LIN_BOX_MN, &maps.q, &full[stage], static_cast<int>(q0) + b * 64, kc);
        } else {
          tma_load_2d(b_dst, &maps.q, &full[stage], kc, static_cast<int>(q0));
        }
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // every load has landed before its memory is used again
      volatile int never = 0;
      for (int s = 0; s < C::kStages; ++s)
        if ((issued >> s) & 1u) mbar_wait(&full[s], (issued_parity >> s) & 1u, &never, p.fault_site + 2);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = lin_idesc(128, BN, p.bf16 != 0, p.p_mn != 0, QMN);
      const uint32_t a_step = p.p_mn ? 2048u : 32u, b_step = QMN ? 2048u : 32u;
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort, p.fault_site + 3)) break;
        tc_fence_after();
        const uint32_t a_addr = smem_u32(smem + stage * C::kStage);
        const uint32_t b_addr = a_addr + C::kP;
        const uint64_t ad = p.p_mn ? sw128_mnmajor_desc(a_addr) : sw128_kmajor_desc(a_addr);
        const uint64_t bd = QMN ? sw128_mnmajor_desc(b_addr) : sw128_kmajor_desc(b_addr);
#pragma unroll
        for (int kk = 0; kk < LIN_BK / 16; ++kk)
          tc_mma_bf16(tmem_base, ad + ((kk * a_step) >> 4), bd + ((kk * b_step) >> 4), idesc, (kb | kk) != 0 ? 1u : 0u);
        tc_commit(&empty[stage]);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // also after a wait that gave up: what was issued completes
      tc_commit(done);
    }
    __syncwarp();
  }
  // everyone waits for the last MMA (the producer's loads have landed by then:
  // the MMAs read them, or its own wait saw them)
  {
    volatile int never = 0;
    __syncwarp();
    mbar_wait(done, 0u, &never, p.fault_site + 4);
  }
  __syncthreads();
  tc_fence_after();
  // partial sums to shared memory as [Q row][128], over the stages
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int quarter = warp & 3;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
    for (int c = 0; c < BN; c += 32) {
      float a[32];
      tmem_ld32(tbase + c, a);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < BN) part[(c + i) * 128 + quarter * 32 + lane] = a[i];
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  // the cluster's CTAs share the outputs: four columns of a row each time,
  // partial sums added in rank order
  const uint32_t part_addr = smem_u32(part);
  for (int i = rank * LS_THREADS + threadIdx.x; i < BN * 32; i += split * LS_THREADS) {
    const int row = i >> 5, col = p0 + (i & 31) * 4;
    if (q0 + row >= p.Q || col >= p.P) continue;
    float4 v[LS_MAX_SPLIT];
#pragma unroll
    for (int s = 0; s < LS_MAX_SPLIT; ++s)
      v[s] = s < split ? ld_cluster_f4(map_to_rank(part_addr + static_cast<uint32_t>(i) * 16u, static_cast<uint32_t>(s)))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < LS_MAX_SPLIT; ++s) {
      a[0] += v[s].x;
      a[1] += v[s].y;
      a[2] += v[s].z;
      a[3] += v[s].w;
    }
    lin_finish<OutT, 4>(p, q0 + row, col, a);
  }
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while its partial sums are read
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kCols);
  }
}

// ------------------------------------------------------------------------------ dp and dbias
// dp = dy act'(pre), rounded to the operand type (skipped where dp is null): the tensor
// cores take 16-bit operands, and a second product over what the rounding cut off would
// double the gradients' time for an error of 1.7e-3 instead of 2.3e-3 (bf16); and
// each block's column sums of the unrounded dp (skipped where part is null):
// part[blockIdx.y][N].  Thread = 8 columns; a block walks over `rows` rows from
// blockIdx.y * rows on.
constexpr int LIN_DP_THREADS = 128;

template <typename T>
__global__ void __launch_bounds__(LIN_DP_THREADS)
    linear_dp_kernel(const T* __restrict__ dy, const T* __restrict__ pre, T* __restrict__ dp, float* __restrict__ part,
                     long long M, int N, long long rows, int act) {
  pdl_next();
  pdl_wait();
  const int col = (blockIdx.x * LIN_DP_THREADS + threadIdx.x) * 8;
  if (col >= N) return;
  const long long r0 = blockIdx.y * rows, r1 = min(M, r0 + rows);
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
#pragma unroll 4
  for (long long r = r0; r < r1; ++r) {
    float d[8];
    op_load<T, 8>(dy + r * N + col, d);
    if (act != kActNone) {
      float a[8];
      op_load<T, 8>(pre + r * N + col, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] *= lin_act_grad(a[i], act);
      if (dp != nullptr) op_store<T, 8>(dp + r * N + col, d);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += d[i];
  }
  if (part != nullptr) {
    float* o = part + static_cast<long long>(blockIdx.y) * N + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = sum[i];
  }
}

}  // namespace moe
