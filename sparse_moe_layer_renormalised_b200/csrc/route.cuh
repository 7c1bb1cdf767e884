// Routing from logits: scores (softmax or sigmoid), selection bias, groups,
// top-k in the exact order of the keys, weights; and the weights' gradient.
//
// Forward: one warp per token, its row of at most 1024 logits in registers.  (Many
// short rows: route_short.cuh.)  What it costs are the instructions next to the one read
// of the logits (16384 x 896 fp32, sigmoid + bias, top 16: 27 us, 59 MB in 9; 59 % of the
// issue slots taken) and the waits of a token's one chain of steps, which the 32 warps
// of an SM that the registers allow do not cover.  So the top-k does not run k arg-max
// rounds over all keys: the k-th largest of the 32 lanes' own maxima is a lower bound
// of the k-th key, and only the few keys at or above it (22 of 896 at k = 16, on
// average) are listed and sorted, 32 at a time.  For the same reason sigmoid + bias
// keys are first formed with one hardware tanh each, to 2.6e-4, and exactly enough to
// be sorted for the candidates alone.
//
// Exact order from fp32 arithmetic: the fp32 keys carry an error of at most
// route_tol; where two neighbours in the sorted list (or the last chosen and
// one left out) are nearer than twice that, and are not equal in both logit and
// bias, the warp orders the candidates again by fp64 keys, and likewise the
// groups where the last kept one is as near.  At k = 16 of 896 with normal logits and
// sigmoid scores about one row in a thousand does so, with softmax scores several
// in a hundred.
#pragma once

#include <cfloat>

#include "ops_common.cuh"
#include "routing.cuh"

namespace moe {

constexpr int ROUTE_WARPS = 4;
constexpr int ROUTE_MAX_E = 1024;

struct RouteParams {
  const void* logits;
  const float* bias;  // may be null
  int32_t* idx;
  float* w;
  long long T;
  int E, k, groups, gsize, keep, gtop;
  unsigned gmagic;  // ceil(2^20 / gsize): e / gsize = (e * gmagic) >> 20 for e, gsize <= 1024
  int softmax, renorm;
  float scale;
};

// A logit as the selection sees it: NaN counts as masked, -0 as 0.
__device__ __forceinline__ float route_logit(float l) { return l == l ? l + 0.0f : -INFINITY; }

// Order-preserving image of an fp32 number (no NaN) in the unsigned integers.
__device__ __forceinline__ uint32_t f32_order(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float f32_unorder(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

// Bound of the error of an fp32 key, score (at most smax in the row) plus bias.
// The score, in steps of 2^-23 of smax: sigmoid: s (1 - s) times the fast
// exponential's 2 + 1.173 |l|, at most 0.63, half for 1 + e and 2 for the fast
// division: 3.2, 3.8e-7.  Softmax: at most 2 for the exponential and the
// difference l - m beside it (the largest of e^-d (2 + 1.67 d)); the sum's, which
// scales all scores: the exponentials' weighted mean, 2 + 1.67 * ln 1024, and 14
// roundings of 2^-24 in its tree; 1 for the reciprocal: 24, 2.9e-6.  The sum with
// the bias rounds by 2^-24.
__device__ __forceinline__ float route_tol(int softmax, float smax, float key) {
  return (softmax ? 3e-6f : 4e-7f) * smax + 7e-8f * fabsf(key);
}

// Bound of the error of a group's score in fp32, key a or the sum of keys a and b
// (b -inf: a alone), with the bound taken off it or added.  Each key's error goes
// with its own size, which may be far above the sum's: route_tol's 7e-8 for each,
// once more for the sum's rounding, and once for that of score - bound.
__device__ __forceinline__ float route_group_tol(int softmax, float smax, float a, float b) {
  const bool two = b != -INFINITY;
  const float keys = fabsf(a) + (two ? fabsf(b) : 0.f), sum = fabsf(two ? a + b : a);
  return fminf((two ? 2.f : 1.f) * (softmax ? 3e-6f : 4e-7f) * smax + 7e-8f * (keys + 2.f * sum), FLT_MAX);
}

// e^(l - m) over the row's maximum m; the limit where m is infinite.
__device__ __forceinline__ float route_exp(float l, float m) {
  if (isinf(m)) return l == m && m > 0.f ? 1.f : 0.f;
  return __expf(l - m);
}

// The score of one logit in fp32 to a few ulp, for the weights.
__device__ __forceinline__ float route_score(float l, int softmax, float m, float inv_z) {
  if (softmax) {
    if (isinf(m)) return l == m && m > 0.f ? inv_z : 0.f;
    return expf(l - m) * inv_z;
  }
  return 1.0f / (1.0f + expf(-l));
}

// Share of each lane's chosen logit (-inf: none) in the sum of the chosen scores;
// what underflows is a share below 1e-20: softmax scores relative to the largest
// chosen one; sigmoid scores as they are, or, where all are below 1e-18, as e^l
// (sigmoid(l) = e^l up to a relative e^l) relative to the largest.  0 everywhere
// where all are masked.
__device__ __forceinline__ float route_share(float l, int softmax) {
  float s = 0.f, total = 0.f;
  if (!softmax) {
    s = route_score(l, 0, 0.f, 1.f);
    total = warp_sum(s);
  }
  if (total < 1e-18f) {
    s = route_score(l, 1, warp_max(l), 1.f);
    total = warp_sum(s);
  }
  return total > 0.f ? s / total : 0.f;
}

// 64-bit sort key: larger fp32 key first, lower expert first among equals.
// Never 0 for a real entry, so 0 is the empty one.
__device__ __forceinline__ unsigned long long route_pack(float key, int e) {
  return (static_cast<unsigned long long>(f32_order(key)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e));
}
__device__ __forceinline__ int route_expert(unsigned long long c) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(c));
}

// Compare-exchange steps of a descending bitonic network over the warp.
template <typename V>
__device__ __forceinline__ V cmpx(V v, int lane, int j, bool up) {
  const V o = __shfl_xor_sync(0xffffffffu, v, j);
  const bool low = (lane & j) == 0;
  return (low == up) ? (o < v ? v : o) : (o < v ? o : v);
}
template <typename V>
__device__ __forceinline__ V warp_sort_desc(V v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) v = cmpx(v, lane, j, (lane & k) == 0);
  return v;
}

// The 32 largest of two descending lists, descending; `drop` keeps the largest
// entry that fell out, per lane.
__device__ __forceinline__ unsigned long long route_merge(unsigned long long top, unsigned long long v, int lane,
                                                          unsigned long long& drop) {
  const unsigned long long o = __shfl_sync(0xffffffffu, v, 31 - lane);
  unsigned long long hi = top > o ? top : o;
  const unsigned long long lo = top > o ? o : top;
  drop = drop > lo ? drop : lo;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) hi = cmpx(hi, lane, j, true);
  return hi;
}

// Sum of e^(l - m) over the row in fp64 (limits as in route_exp), in all lanes.
template <typename T>
__device__ __noinline__ double route_sum64(const T* row, int E, double m, int lane) {
  double z[4] = {0.0, 0.0, 0.0, 0.0};
  for (int e0 = lane; e0 < E; e0 += 128) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + 32 * i;
      const double l = e < E ? static_cast<double>(route_logit(op_f32(row[e]))) : -INFINITY;
      z[i] += isinf(m) ? (l == m && m > 0 ? 1.0 : 0.0) : exp(l - m);
    }
  }
  return warp_sum((z[0] + z[1]) + (z[2] + z[3]));
}

// The key of an unmasked logit l in fp64; z is route_sum64's (softmax only).
__device__ __noinline__ double route_key64(int softmax, float l, float b, double m, double z) {
  const double x = l;
  const double s = softmax ? (isinf(m) ? (x == m ? 1.0 : 0.0) : exp(x - m)) / z : 1.0 / (1.0 + exp(-x));
  return s + static_cast<double>(b);
}

// An expert with its fp64 key; a larger key, then a lower expert, comes first.
struct Ranked {
  double v;
  int e;
};
__device__ __forceinline__ bool before(const Ranked& a, const Ranked& b) {
  return a.v > b.v || (a.v == b.v && a.e < b.e);
}
__device__ __forceinline__ Ranked shfl_xor(const Ranked& r, int j) {
  return {__shfl_xor_sync(0xffffffffu, r.v, j), __shfl_xor_sync(0xffffffffu, r.e, j)};
}
__device__ __forceinline__ Ranked cmpx(const Ranked& r, int lane, int j, bool up) {
  const Ranked o = shfl_xor(r, j);
  return (((lane & j) == 0) == up) == before(r, o) ? r : o;
}

// The candidates in the order of their fp64 keys: lane j gets the j-th expert
// (-1: none).  32 at a time are sorted and merged into the 32 best.
template <typename T>
__device__ __noinline__ int route_resolve(const RouteParams& p, const T* row, const uint16_t* cand, int cnt, double m,
                                          double z, int lane) {
  Ranked top{-INFINITY, 0x7fffffff - 31 + lane};
  for (int at = 0; at < cnt; at += 32) {
    Ranked r{-INFINITY, 0x7fffffff - 63 + lane};  // (never equal to another lane's)
    if (at + lane < cnt) {
      r.e = cand[at + lane];
      const double v = route_key64(p.softmax, route_logit(op_f32(row[r.e])), p.bias[r.e], m, z);
      if (v == v) r.v = v;
    }
    __syncwarp();
#pragma unroll 1
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll 1
      for (int j = k >> 1; j > 0; j >>= 1) r = cmpx(r, lane, j, (lane & k) == 0);
    const Ranked o{__shfl_sync(0xffffffffu, r.v, 31 - lane), __shfl_sync(0xffffffffu, r.e, 31 - lane)};
    if (before(o, top)) top = o;
#pragma unroll 1
    for (int j = 16; j > 0; j >>= 1) top = cmpx(top, lane, j, true);
  }
  return top.e < ROUTE_MAX_E ? top.e : -1;
}

// Bit mask of the kept groups.  score: lane g's group score.  Equal scores go to
// the lower group.
template <typename V>
__device__ __forceinline__ uint32_t route_keep(V score, int groups, int keep, int lane) {
  int rank = 0;
  for (int o = 0; o < groups; ++o) {
    const V so = __shfl_sync(0xffffffffu, score, o);
    rank += (so > score || (so == score && o < lane)) ? 1 : 0;
  }
  return __ballot_sync(0xffffffffu, lane < groups && rank < keep);
}

// The kept groups from fp64 scores: only the values of a group that fp32 puts
// within twice the error of the last one that counts are formed again.
template <typename T>
__device__ __noinline__ uint32_t route_keep64(const RouteParams& p, const T* row, const float* val, float smax, double m,
                                              double z, int lane, int lpg) {
  const int g = lane / lpg, sub = lane - g * lpg;
  float a = -INFINITY, b = -INFINITY;
  if (g < p.groups) {
    for (int j = sub; j < p.gsize; j += lpg) {
      const float v = val[g * p.gsize + j];
      b = fmaxf(b, fminf(a, v));
      a = fmaxf(a, v);
    }
  }
  for (int o = lpg >> 1; o > 0; o >>= 1) {
    const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    b = fmaxf(fmaxf(b, ob), fminf(a, oa));
    a = fmaxf(a, oa);
  }
  float thr = p.gtop == 2 ? b : a;
  thr = fmaxf(thr - 2.f * route_tol(p.softmax, smax, thr), -FLT_MAX);
  double a64 = -INFINITY, b64 = -INFINITY;
  if (g < p.groups) {
    for (int j = sub; j < p.gsize; j += lpg) {
      const int e = g * p.gsize + j;
      if (!(val[e] >= thr)) continue;
      const double v = route_key64(p.softmax, route_logit(op_f32(row[e])), p.bias != nullptr ? p.bias[e] : 0.f, m, z);
      b64 = fmax(b64, fmin(a64, v));
      a64 = fmax(a64, v);
    }
  }
  __syncwarp();
  for (int o = lpg >> 1; o > 0; o >>= 1) {
    const double oa = __shfl_xor_sync(0xffffffffu, a64, o), ob = __shfl_xor_sync(0xffffffffu, b64, o);
    b64 = fmax(fmax(b64, ob), fmin(a64, oa));
    a64 = fmax(a64, oa);
  }
  double score = p.gtop == 2 && !(isinf(b64) && b64 < 0) ? a64 + b64 : a64;
  score = __shfl_sync(0xffffffffu, score, (lane * lpg) & 31);
  return route_keep(score, p.groups, p.keep, lane);
}

// Bytes of shared memory a warp uses: two lists of 32 sort keys and one of 32
// (logit, bias), then the candidates' numbers or, before them, the keys that the
// groups are ranked by.
constexpr int ROUTE_LISTS = 768;
__host__ __device__ constexpr int route_warp_bytes(int E, bool grouped) {
  return ROUTE_LISTS + (E * (grouped ? 4 : 2) + 15) / 16 * 16;
}

// tanh by the hardware's approximation: relative error up to 2^-11.
__device__ __forceinline__ float tanh_approx(float x) {
  float y;
  asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bound of the error of 0.5 tanh_approx(l / 2) + bias, which orders the experts
// as sigmoid(l) + bias does.
__device__ __forceinline__ float route_coarse_tol(float key) { return 2.6e-4f + 1.5e-7f * fabsf(key); }

// CH loads of VL elements per lane; expert of value (c, i): (c * 32 + lane) * VL + i.
template <typename T, int VL, int CH>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, 8) route_kernel(const RouteParams p) {
  constexpr int NV = VL * CH;
  extern __shared__ __align__(16) uint8_t route_smem[];
  pdl_next();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * ROUTE_WARPS + warp;
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const bool biased = p.bias != nullptr;
  const bool grouped = p.keep < p.groups;
  const T* row = static_cast<const T*>(p.logits) + t * E;
  uint8_t* smem = route_smem + warp * route_warp_bytes(E, grouped);
  unsigned long long* list = reinterpret_cast<unsigned long long*>(smem);  // [64]
  float2* list_lb = reinterpret_cast<float2*>(smem + 512);                 // [32]
  uint16_t* cand = reinterpret_cast<uint16_t*>(smem + ROUTE_LISTS);
  float* val = reinterpret_cast<float*>(smem + ROUTE_LISTS);

  // logits, -inf where the row ends (a NaN is below every number in the comparisons
  // and maxima below)
  float key[NV];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * 32 + lane) * VL;
    if (e0 < E) {
      op_load<T, VL>(row + e0, key + c * VL);
    } else {
#pragma unroll
      for (int i = 0; i < VL; ++i) key[c * VL + i] = -INFINITY;
    }
  }
  float m = -INFINITY, inv_z = 1.f, smax = 1.f;
  const bool need_scores = biased || (grouped && p.gtop == 2);
  if (p.softmax && (need_scores || !p.renorm)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      key[i] = fmaxf(key[i], -INFINITY);  // NaN as masked
      m = fmaxf(m, key[i]);
    }
    m = warp_max(m);
    float z4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) z4[i & 3] += route_exp(key[i], m);
    const float z = warp_sum((z4[0] + z4[1]) + (z4[2] + z4[3]));
    inv_z = z > 0.f ? 1.0f / z : 0.f;
    smax = inv_z;
  }
  // keys: the logits themselves without a bias; score + bias (-inf where masked,
  // and a NaN never wins) to route_tol; or, for the plain case of sigmoid + bias,
  // to route_coarse_tol, which is enough to find the candidates
  const bool coarse = biased && !p.softmax && !grouped;
  if (coarse) {
    float least = INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) least = fminf(least, key[i]);
    uint32_t gone = 0u;  // masked values of the lane
    if (least == -INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i) gone |= key[i] == -INFINITY ? 1u << i : 0u;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * 32 + lane) * VL;
      if (e0 < E) {
        float b[VL];
        op_load_f32<VL>(p.bias + e0, b);
#pragma unroll
        for (int i = 0; i < VL; ++i) key[c * VL + i] = fmaf(0.5f, tanh_approx(0.5f * key[c * VL + i]), b[i]);
      }
    }
    if (gone != 0u) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((gone >> i) & 1u) key[i] = -INFINITY;
    }
  } else if (need_scores) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * 32 + lane) * VL;
      if (e0 < E) {
        float b[VL];
#pragma unroll
        for (int i = 0; i < VL; ++i) b[i] = 0.f;
        if (biased) op_load_f32<VL>(p.bias + e0, b);
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const float l = key[c * VL + i];
          const float s = p.softmax ? route_exp(l, m) * inv_z : __fdividef(1.0f, 1.0f + __expf(-l));
          float v = s + b[i];
          if (l == -INFINITY || v != v) v = -INFINITY;
          if (grouped) val[e0 + i] = v;
          if (biased) key[c * VL + i] = v;
        }
      }
    }
  } else if (grouped) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * 32 + lane) * VL;
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (e0 < E) val[e0 + i] = key[c * VL + i];
    }
  }

  double z64 = 0.0;  // route_sum64's, once it is needed
  uint32_t kept = 0xffffffffu;
  if (grouped) {
    __syncwarp();
    // 32 / P lanes per group, P the power of two at or above the group count
    const int lpg = 32 >> (32 - __clz(p.groups - 1));
    const int g = lane / lpg, sub = lane - g * lpg;
    float a = -INFINITY, b = -INFINITY;
    if (g < p.groups) {
      for (int j = sub; j < p.gsize; j += lpg) {
        const float v = val[g * p.gsize + j];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
      const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
      b = fmaxf(fmaxf(b, ob), fminf(a, oa));
      a = fmaxf(a, oa);
    }
    if (p.gtop == 1) b = -INFINITY;
    float score = b != -INFINITY ? a + b : a;
    score = __shfl_sync(0xffffffffu, score, (lane * lpg) & 31);
    if (lane >= p.groups) score = -INFINITY;
    kept = route_keep(score, p.groups, p.keep, lane);
    if (need_scores) {
      // the least that a kept group may have against the most of one left out
      const float tol = __shfl_sync(0xffffffffu, route_group_tol(p.softmax, smax, a, b), (lane * lpg) & 31);
      const bool mine = (kept >> lane) & 1u;
      const float lo = -warp_max(mine ? tol - score : -INFINITY);
      const float hi = warp_max(mine || score == -INFINITY ? -INFINITY : score + tol);
      if (hi != -INFINITY && !(lo > hi)) {
        if (p.softmax) z64 = route_sum64(row, E, m, lane);
        kept = route_keep64<T>(p, row, val, smax, m, z64, lane, lpg);
      }
    }
    const bool whole = VL == 1 || p.gsize % VL == 0;  // a load lies in one group
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const unsigned e0 = (c * 32 + lane) * VL;  // (past E: -inf already, any group will do)
      bool in = (kept >> (((e0 * p.gmagic) >> 20) & 31u)) & 1u;
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        if (!whole) in = (kept >> ((((e0 + i) * p.gmagic) >> 20) & 31u)) & 1u;
        if (!in) key[c * VL + i] = -INFINITY;
      }
    }
    __syncwarp();
  }

  // lower bound of the k-th largest key: the k-th largest of the lanes' maxima,
  // or, for k > 16, of two maxima a lane, over half its keys each (at k = 32 of
  // 1000 that leaves 43 candidates instead of 110)
  float lm = -INFINITY, lm2 = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; i += 2) {
    lm = fmaxf(lm, key[i]);
    lm2 = fmaxf(lm2, key[i + 1]);
  }
  float thr = -INFINITY;
  if (k <= 16) {
    // largest value by largest value (equal ones go together, which only lowers
    // the bound)
    lm = fmaxf(lm, lm2);
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      thr = warp_max(lm);
      if (lm == thr) lm = -INFINITY;
    }
  } else {
    lm = warp_sort_desc(lm, lane);
    lm2 = __shfl_sync(0xffffffffu, warp_sort_desc(lm2, lane), 31 - lane);
    lm = fmaxf(lm, lm2);
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) lm = cmpx(lm, lane, j, true);
    thr = __shfl_sync(0xffffffffu, lm, k - 1);
  }
  if (biased) thr -= 2.f * (coarse ? route_coarse_tol(thr) : route_tol(p.softmax, smax, thr));
  thr = fmaxf(thr, -FLT_MAX);  // never -inf (or inf - inf)
  // the keys at or above it, by number
  uint32_t hits = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) hits |= key[i] >= thr ? 1u << i : 0u;
  int cnt = 0;
  for (uint32_t has; (has = __ballot_sync(0xffffffffu, hits != 0u)) != 0u; cnt += __popc(has)) {
    if (hits != 0u) {
      const int i = __ffs(static_cast<int>(hits)) - 1;
      hits &= hits - 1u;
      cand[cnt + __popc(has & ((1u << lane) - 1u))] = static_cast<uint16_t>(((i / VL) * 32 + lane) * VL + i % VL);
    }
  }
  __syncwarp();
  // their keys, sorted; lane j then holds the j-th (0: none) with its logit and bias
  unsigned long long top = 0ull, drop = 0ull;
  float l = -INFINITY, b = 0.f;
  auto candidate = [&](int at) {
    const int e = cand[at];
    l = route_logit(op_f32(row[e]));
    float v = l;
    if (biased) {
      b = p.bias[e];
      v = (p.softmax ? route_exp(l, m) * inv_z : __fdividef(1.0f, 1.0f + __expf(-l))) + b;
      if (v != v) v = -INFINITY;
    }
    return route_pack(v, e);
  };
  if (cnt <= 32) {
    // the rank of each among them is its place
    const unsigned long long mine = lane < cnt ? candidate(lane) : 0ull;
    list[lane] = mine;
    __syncwarp();
    int rank = lane < cnt ? 0 : lane;
    const ulonglong2* l2 = reinterpret_cast<const ulonglong2*>(list);
#pragma unroll 4
    for (int j = 0; 2 * j < cnt; ++j) {
      const ulonglong2 o = l2[j];
      // (an empty entry's rank stays: nothing is above its own place)
      if (o.x > mine && mine != 0ull) ++rank;
      if (o.y > mine && mine != 0ull) ++rank;
    }
    list[32 + rank] = mine;
    list_lb[rank] = make_float2(l, b);
    __syncwarp();
    top = list[32 + lane];
    const float2 lb = list_lb[lane];
    l = lb.x;
    b = lb.y;
  } else {
    for (int at = 0; at < cnt; at += 32) {
      const unsigned long long mine = warp_sort_desc(at + lane < cnt ? candidate(at + lane) : 0ull, lane);
      top = at == 0 ? mine : route_merge(top, mine, lane, drop);
    }
    l = top != 0ull ? route_logit(op_f32(row[route_expert(top)])) : -INFINITY;
    b = biased && top != 0ull ? p.bias[route_expert(top)] : 0.f;
  }

  int e = top != 0ull ? route_expert(top) : 0;
  const float kk = f32_unorder(static_cast<uint32_t>(top >> 32));
  // chosen by key; the others by index.  (A candidate's key may be -inf: a NaN or
  // -inf bias under a coarse threshold.)
  const int nsel = min(k, __popc(__ballot_sync(0xffffffffu, top != 0ull && kk != -INFINITY)));
  if (biased) {
    const float k2 = __shfl_down_sync(0xffffffffu, kk, 1);
    const float l2 = __shfl_down_sync(0xffffffffu, l, 1);
    const float b2 = __shfl_down_sync(0xffffffffu, b, 1);
    // neighbours among the chosen: apart, or equal in logit and bias (then the
    // index has ordered them)
    bool bad = lane + 1 < nsel && !(kk - k2 > 2.f * route_tol(p.softmax, smax, kk)) && !(l == l2 && b == b2);
    // the last chosen against all that were left out
    const int last = nsel > 0 ? nsel - 1 : 0;
    const float kl = __shfl_sync(0xffffffffu, kk, last);
    const float ll = __shfl_sync(0xffffffffu, l, last);
    const float bl = __shfl_sync(0xffffffffu, b, last);
    const float tol = 2.f * route_tol(p.softmax, smax, kl);
    const bool beyond = nsel > 0 && drop != 0ull && !(kl - f32_unorder(static_cast<uint32_t>(drop >> 32)) > tol);
    bad |= beyond || (nsel > 0 && lane >= nsel && top != 0ull && !(kl - kk > tol) && !(l == ll && b == bl));
    if (__any_sync(0xffffffffu, bad)) {
      if (p.softmax && z64 == 0.0) z64 = route_sum64(row, E, m, lane);
      e = max(0, route_resolve<T>(p, row, cand, cnt, m, z64, lane));
      l = lane < k ? route_logit(op_f32(row[e])) : -INFINITY;
    }
  }
  if (nsel < k) {
    // masked experts of the kept groups fill up, in ascending order
    int have = nsel;
    for (int e0 = 0; e0 < E && have < k; e0 += 32) {
      const int x = e0 + lane;
      bool is = false;
      if (x < E && ((kept >> ((static_cast<unsigned>(x) * p.gmagic) >> 20)) & 1u)) {
        const float lx = route_logit(op_f32(row[x]));
        const float bx = biased ? p.bias[x] : 0.f;
        is = lx == -INFINITY || bx == -INFINITY || bx != bx;
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, is);
      const int want = lane - have;  // the lane's place among these
      if (lane >= have && want < __popc(mask)) e = e0 + static_cast<int>(__fns(mask, 0, want + 1));
      have += __popc(mask);
    }
    l = lane < k ? route_logit(op_f32(row[e])) : -INFINITY;
  }

  if (lane >= k) l = -INFINITY;
  const float out = (p.renorm ? route_share(l, p.softmax) : route_score(l, p.softmax, m, inv_z)) * p.scale;
  if (lane < k) {
    p.idx[t * k + lane] = e;
    p.w[t * k + lane] = out;
  }
}

// Gradient of the weights.  One warp per token.  Sigmoid scores and renormalised
// softmax scores reach the chosen logits only (the row is cleared and k values
// are put in); plain softmax scores reach every logit, and the row is read once,
// into registers.  16384 x 896 bf16, the first form 12 to 13 us, bound by the start of
// so many warps and the loads they wait for (40 % of the issue slots), the plain
// softmax 17 us, 21 out of memory: the exponentials of a whole row, 64 % of the issue
// slots with 29 of 64 warps.
template <typename T, int VL, int CH>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, 8)
    route_backward_kernel(const RouteParams p, const int32_t* __restrict__ idx, const float* __restrict__ dw,
                          T* __restrict__ dl_out) {
  constexpr int NV = VL * CH;
  pdl_next();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const T* row = static_cast<const T*>(p.logits) + t * E;
  T* out = dl_out + t * E;
  const bool dense = p.softmax && !p.renorm;
  float v[NV];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * 32 + lane) * VL;
#pragma unroll
    for (int i = 0; i < VL; ++i) v[c * VL + i] = dense ? -INFINITY : 0.f;
    if (dense && e0 < E) op_load<T, VL>(row + e0, v + c * VL);
  }
  int e = -1 - lane;  // distinct where there is none
  float d = 0.f, l = -INFINITY;
  if (lane < k) {
    const int x = idx[t * k + lane];
    if (x < 0 || x >= E) {
      record_fault(kFaultExpertRange);
    } else {
      e = x;
    }
  }
  const uint32_t same = __match_any_sync(0xffffffffu, e);
  if (__ffs(static_cast<int>(same)) - 1 < lane) {
    record_fault(kFaultDuplicateExpert);
    e = -1 - lane;
  }
  if (e >= 0) {
    l = route_logit(op_f32(row[e]));
    // a masked expert's weight is 0 whatever the logits: its dw counts for nothing
    if (l != -INFINITY) d = dw[t * k + lane] * p.scale;
  }
  float dl = 0.f;
  if (dense) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = fmaxf(v[i], -INFINITY);  // NaN as masked
      m = fmaxf(m, v[i]);
    }
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = route_exp(v[i], m);
      z += v[i];
    }
    z = warp_sum(z);
    const float inv_z = z > 0.f ? 1.0f / z : 0.f;
    const float s = e >= 0 ? route_score(l, 1, m, inv_z) : 0.f;
    const float dot = warp_sum(s * d);
    dl = s * (d - dot);
    const float f = -dot * inv_z;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] *= f;
  } else {
    float pj;
    if (p.renorm) {
      pj = route_share(l, p.softmax);
      d -= warp_sum(pj * d);
    } else {
      pj = route_score(l, 0, 0.f, 1.f);  // (sigmoid: softmax without renorm is dense)
    }
    // 1 - sigmoid(l) without cancellation
    dl = pj * d * (p.softmax ? 1.f : 1.0f / (1.0f + expf(l)));
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * 32 + lane) * VL;
    if (e0 < E) op_store<T, VL>(out + e0, v + c * VL);
  }
  __syncwarp();  // the row's stores come before the chosen experts'
  if (e >= 0) out[e] = op_from<T>(dl);
}

}  // namespace moe
