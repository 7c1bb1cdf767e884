// Routing from logits: scores (softmax or sigmoid), selection bias, groups,
// top-k in the exact order of the keys, weights; and the weights' gradient.
//
// Forward: one warp per token, its row of at most 1024 logits in registers.
// What bounds it is instruction issue next to the one read of the logits, so
// the top-k does not run k arg-max rounds over all keys: the k-th largest of
// the 32 lanes' own maxima (one 32-wide sort) is a lower bound of the k-th key,
// and only the few keys at or above it (22 of 896 at k = 16, on average) are
// compacted into shared memory and sorted, 32 at a time.
//
// Exact order from fp32 arithmetic: the fp32 keys carry an error of at most
// route_tol; where two neighbours in the sorted list (or the last chosen and
// the first left out) are nearer than twice that, and are not equal in both
// logit and bias, the warp selects again with fp64 keys (route_exact).  At
// k = 16 of 896 with normal logits about one row in a thousand does so.
#pragma once

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

// Bound of the error of an fp32 key: the score's (fast exponential and
// reciprocal; under 3e-7 of the largest score of the row, measured against
// 64 bits, with a margin of three) and the rounding of score + bias.
__device__ __forceinline__ float route_tol(float smax, float key) { return 1e-6f * smax + 1.5e-7f * fabsf(key); }

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

// Share of each lane's chosen logit (-inf: none) in the sum of the chosen scores,
// free of underflow: softmax scores relative to the largest chosen one; sigmoid
// scores as they are, or, where all are below 1e-18, as e^l (sigmoid(l) = e^l up
// to a relative e^l) relative to the largest.  0 everywhere where all are masked.
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

// Selection of one token in fp64, straight from the definition: lane j gets
// the j-th expert.  Called by whole warps, for the few rows whose fp32 keys are
// too near to be told apart.
template <typename T>
__device__ __noinline__ int route_exact(const RouteParams& p, const T* row, int lane) {
  const int E = p.E;
  double m = -INFINITY;
  for (int e = lane; e < E; e += 32) m = fmax(m, static_cast<double>(route_logit(op_f32(row[e]))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  double z = 0.0;
  if (p.softmax) {
    for (int e = lane; e < E; e += 32) {
      const double l = route_logit(op_f32(row[e]));
      z += isinf(m) ? (l == m && m > 0 ? 1.0 : 0.0) : exp(l - m);
    }
    z = warp_sum(z);
  }
  double key[32];   // keys of experts lane, lane + 32, ...
  uint32_t live = 0u;
  for (int i = 0; i < 32; ++i) {
    const int e = lane + 32 * i;
    key[i] = -INFINITY;
    if (e >= E) continue;
    const double l = route_logit(op_f32(row[e]));
    live |= 1u << i;
    if (isinf(l) && l < 0) continue;
    double s;
    if (p.softmax)
      s = (isinf(m) ? (l == m ? 1.0 : 0.0) : exp(l - m)) / z;
    else
      s = 1.0 / (1.0 + exp(-l));
    // without a bias the logits themselves order the experts
    const double kk = p.bias != nullptr ? s + static_cast<double>(p.bias[e]) : l;
    key[i] = kk == kk ? kk : -INFINITY;
  }
  uint32_t kept = 0xffffffffu;
  if (p.keep < p.groups) {
    double mine = -INFINITY;  // lane g: score of group g
    for (int g = 0; g < p.groups; ++g) {
      double a = -INFINITY, b = -INFINITY;
      for (int e = g * p.gsize + lane; e < (g + 1) * p.gsize; e += 32) {
        const double l = route_logit(op_f32(row[e]));
        if (isinf(l) && l < 0) continue;
        double s;
        if (p.softmax)
          s = (isinf(m) ? (l == m ? 1.0 : 0.0) : exp(l - m)) / z;
        else
          s = 1.0 / (1.0 + exp(-l));
        double v = s + (p.bias != nullptr ? static_cast<double>(p.bias[e]) : 0.0);
        if (p.bias == nullptr && p.gtop == 1) v = l;
        if (!(v == v)) continue;
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
        if (oa > a) {
          b = fmax(a, ob);
          a = oa;
        } else {
          b = fmax(b, oa);
        }
      }
      const double score = p.gtop == 2 && !(isinf(b) && b < 0) ? a + b : a;
      if (lane == g) mine = score;
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double o = __shfl_sync(0xffffffffu, mine, g);
      rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    kept = __ballot_sync(0xffffffffu, lane < p.groups && rank < p.keep);
    for (int i = 0; i < 32; ++i) {
      const unsigned e = lane + 32 * i;
      if (((live >> i) & 1u) && !((kept >> ((e * p.gmagic) >> 20)) & 1u)) live &= ~(1u << i);
    }
  }
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    double bk = -INFINITY;
    int be = 0x7fffffff;
    for (int i = 0; i < 32; ++i) {
      const int e = lane + 32 * i;
      if (((live >> i) & 1u) && (key[i] > bk || (key[i] == bk && e < be))) {
        bk = key[i];
        be = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ok = __shfl_xor_sync(0xffffffffu, bk, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (ok > bk || (ok == bk && oe < be)) {
        bk = ok;
        be = oe;
      }
    }
    if ((be & 31) == lane) live &= ~(1u << (be >> 5));
    if (lane == j) mine = be;
  }
  return mine;
}

// CH loads of VL elements per lane; expert of value (c, i): (c * 32 + lane) * VL + i.
template <typename T, int VL, int CH>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_kernel(const RouteParams p) {
  constexpr int NV = VL * CH;
  extern __shared__ unsigned long long route_smem[];  // per warp: E candidates (the group scores before them)
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * ROUTE_WARPS + warp;
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const T* row = static_cast<const T*>(p.logits) + t * E;
  unsigned long long* cand = route_smem + static_cast<size_t>(warp) * E;

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
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    key[i] = route_logit(key[i]);
    m = fmaxf(m, key[i]);
  }
  const bool biased = p.bias != nullptr;
  const bool grouped = p.keep < p.groups;
  float inv_z = 1.f;
  float smax = 1.f;
  if (p.softmax) {
    m = warp_max(m);
    if (biased || !p.renorm || (grouped && p.gtop == 2)) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) z += route_exp(key[i], m);
      z = warp_sum(z);
      inv_z = z > 0.f ? 1.0f / z : 0.f;
      smax = inv_z;
    }
  }
  // scores, then keys; a NaN key never wins over a number
  const bool need_scores = biased || (grouped && p.gtop == 2);
  float gval[NV];  // what the group scores add up (only read when grouped)
  if (need_scores) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * 32 + lane) * VL;
      float b[VL];
#pragma unroll
      for (int i = 0; i < VL; ++i) b[i] = 0.f;
      if (biased && e0 < E) op_load_f32<VL>(p.bias + e0, b);
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const float l = key[c * VL + i];
        const float s = p.softmax ? route_exp(l, m) * inv_z : __fdividef(1.0f, 1.0f + __expf(-l));
        float v = s + b[i];
        if (l == -INFINITY || v != v) v = -INFINITY;
        gval[c * VL + i] = v;
        if (biased) key[c * VL + i] = v;
      }
    }
  } else if (grouped) {
#pragma unroll
    for (int i = 0; i < NV; ++i) gval[i] = key[i];
  }

  bool near = false;
  uint32_t kept = 0xffffffffu;
  if (grouped) {
    float* val = reinterpret_cast<float*>(cand);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int e = (c * 32 + lane) * VL + i;
        if (e < E) val[e] = gval[c * VL + i];
      }
    __syncwarp();
    // 32 / P lanes per group, P the power of two at or above the group count
    int P = 1;
    while (P < p.groups) P <<= 1;
    const int lpg = 32 / P;
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
    float score = p.gtop == 2 && b != -INFINITY ? a + b : a;
    score = __shfl_sync(0xffffffffu, score, (lane * lpg) & 31);
    if (lane >= p.groups) score = -INFINITY;
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const float so = __shfl_sync(0xffffffffu, score, o);
      rank += (so > score || (so == score && o < lane)) ? 1 : 0;
    }
    const bool mine = lane < p.groups && rank < p.keep;
    kept = __ballot_sync(0xffffffffu, mine);
    if (need_scores) {
      const float lo = -warp_max(mine ? -score : -INFINITY);
      const float hi = warp_max(mine || lane >= p.groups ? -INFINITY : score);
      const float tol = p.gtop * (route_tol(smax, lo) + route_tol(smax, hi));
      near = hi != -INFINITY && !(lo - hi > tol);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const unsigned e = (c * 32 + lane) * VL + i;
        if (!((kept >> (((e * p.gmagic) >> 20) & 31u)) & 1u)) key[c * VL + i] = -INFINITY;  // (e >= E: -inf already)
      }
    __syncwarp();
  }

  // lower bound of the k-th largest key
  float lm = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) lm = fmaxf(lm, key[i]);
  lm = warp_sort_desc(lm, lane);
  float thr = __shfl_sync(0xffffffffu, lm, k - 1);
  if (biased) thr -= 2.f * route_tol(smax, thr);
  if (!(thr == thr)) thr = -INFINITY;
  int cnt = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const float v = key[c * VL + i];
      const bool in = v >= thr && v != -INFINITY;
      const uint32_t mask = __ballot_sync(0xffffffffu, in);
      if (in) cand[cnt + __popc(mask & ((1u << lane) - 1u))] = route_pack(v, (c * 32 + lane) * VL + i);
      cnt += __popc(mask);
    }
  __syncwarp();
  unsigned long long top = warp_sort_desc(lane < cnt ? cand[lane] : 0ull, lane);
  unsigned long long drop = 0ull;
  for (int at = 32; at < cnt; at += 32)
    top = route_merge(top, warp_sort_desc(at + lane < cnt ? cand[at + lane] : 0ull, lane), lane, drop);

  int e = top != 0ull ? route_expert(top) : 0;
  const int nsel = min(k, min(cnt, 32));  // chosen by key; the others by index
  float l = top != 0ull ? route_logit(op_f32(row[e])) : -INFINITY;
  if (biased) {
    // neighbours that fp32 cannot order
    const float kk = f32_unorder(static_cast<uint32_t>(top >> 32));
    const float b = top != 0ull ? p.bias[e] : 0.f;
    const float k2 = __shfl_down_sync(0xffffffffu, kk, 1);
    const float l2 = __shfl_down_sync(0xffffffffu, l, 1);
    const float b2 = __shfl_down_sync(0xffffffffu, b, 1);
    // neighbours among the chosen: apart, or equal in logit and bias (then the
    // index has ordered them)
    bool bad = lane + 1 < nsel && !(kk - k2 > 2.f * route_tol(smax, kk)) && !(l == l2 && b == b2);
    if (nsel > 0) {
      // the last chosen against all that were left out
      const float kl = __shfl_sync(0xffffffffu, kk, nsel - 1);
      const float ll = __shfl_sync(0xffffffffu, l, nsel - 1);
      const float bl = __shfl_sync(0xffffffffu, b, nsel - 1);
      const float tol = 2.f * route_tol(smax, kl);
      bad |= lane >= nsel && top != 0ull && !(kl - kk > tol) && !(l == ll && b == bl);
      bad |= drop != 0ull && !(kl - f32_unorder(static_cast<uint32_t>(drop >> 32)) > tol);
    }
    near = near || __any_sync(0xffffffffu, bad);
  }
  if (near) {
    e = route_exact<T>(p, row, lane);
    l = lane < k ? route_logit(op_f32(row[e])) : -INFINITY;
  } else if (nsel < k) {
    // masked experts of the kept groups fill up, in ascending order
    int have = nsel;
    for (int e0 = 0; e0 < E && have < k; e0 += 32) {
      const int x = e0 + lane;
      bool is = false;
      float lx = -INFINITY;
      if (x < E && ((kept >> ((static_cast<unsigned>(x) * p.gmagic) >> 20)) & 1u)) {
        lx = route_logit(op_f32(row[x]));
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
// are put in); plain softmax scores reach every logit, and the row is read.
// Bound by the write of dlogits.
template <typename T, int VL>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
    route_backward_kernel(const RouteParams p, const int32_t* __restrict__ idx, const float* __restrict__ dw,
                          T* __restrict__ dl_out) {
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const T* row = static_cast<const T*>(p.logits) + t * E;
  T* out = dl_out + t * E;
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
  if (p.softmax && !p.renorm) {
    // every lane's running maximum and sum, joined
    float m = -INFINITY, z = 0.f;
    for (int e0 = lane * VL; e0 < E; e0 += 32 * VL) {
      float v[VL];
      op_load<T, VL>(row + e0, v);
      float mm = m;
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        v[i] = route_logit(v[i]);
        mm = fmaxf(mm, v[i]);
      }
      z = m == mm ? z : z * route_exp(m, mm);
      m = mm;
#pragma unroll
      for (int i = 0; i < VL; ++i) z += route_exp(v[i], m);
    }
    const float mm = warp_max(m);
    z = warp_sum(m == mm ? z : z * route_exp(m, mm));
    m = mm;
    const float inv_z = z > 0.f ? 1.0f / z : 0.f;
    const float s = e >= 0 ? route_score(l, 1, m, inv_z) : 0.f;
    const float dot = warp_sum(s * d);
    dl = s * (d - dot);
    const float f = -dot * inv_z;
    for (int e0 = lane * VL; e0 < E; e0 += 32 * VL) {
      float v[VL];
      op_load<T, VL>(row + e0, v);
#pragma unroll
      for (int i = 0; i < VL; ++i) v[i] = f * route_exp(route_logit(v[i]), m);
      op_store<T, VL>(out + e0, v);
    }
  } else {
    float pj;
    if (p.renorm) {
      pj = route_share(l, p.softmax);
      d -= warp_sum(pj * d);
    } else {
      pj = route_score(l, 0, 0.f, 1.f);  // (sigmoid: softmax without renorm is above)
    }
    // 1 - sigmoid(l) without cancellation
    dl = pj * d * (p.softmax ? 1.f : 1.0f / (1.0f + expf(l)));
    float zero[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) zero[i] = 0.f;
    for (int e0 = lane * VL; e0 < E; e0 += 32 * VL) op_store<T, VL>(out + e0, zero);
  }
  __syncwarp();  // the row's stores come before the chosen experts'
  if (e >= 0) out[e] = op_from<T>(dl);
}

}  // namespace moe
