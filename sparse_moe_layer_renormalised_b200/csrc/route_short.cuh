// Routing of short rows: as route.cuh, with L lanes per token, 32 / L tokens a warp.
//
// What a token costs beside its logits (threshold, list, ranks, weights) is the same
// for every row length and is issued for whole warps; at 128 experts it was nearly
// all of the time (32767 x 128, top 8: 24 us with a warp a token).  L lanes (8 up to
// k = 8, else 16) share it among 4 or 2 tokens.  The lower bound of the k-th key is the
// k-th largest of two maxima a lane; the keys at or above it are listed with their
// numbers, and the place of each is the count of larger ones.
//
// Whatever a token needs seldom (near ties in fp64, masked experts to fill up with) is
// done by the whole warp, token by token.
#pragma once

#include "route.cuh"

namespace moe {

// Shared memory of a token: E + 2 sort keys (or, before them, the keys that the groups
// are ranked by and the bounds of the groups' scores), the numbers of the listed experts, and 144 bytes for 32 group scores
// or, after them, the chosen keys.  Tokens lie 16 bytes off a multiple of 128 apart:
// their lanes read different banks.
__host__ __device__ constexpr int route_short_cand(int E) { return ((E + 2) * 8 + 15) / 16 * 16; }
__host__ __device__ constexpr int route_short_tail(int E) { return route_short_cand(E) + (2 * E + 15) / 16 * 16; }
__host__ __device__ constexpr int route_short_token_bytes(int E) {
  return (route_short_tail(E) + 144 + 127) / 128 * 128 + 16;
}

// Reductions over each L neighbouring lanes, the same in all of them.
template <int L>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float part_sort_desc(float v, int lane) {
#pragma unroll
  for (int k = 2; k <= L; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) v = cmpx(v, lane, j, k == L || (lane & k) == 0);
  return v;
}

// route_share over each L lanes.
template <int L>
__device__ __forceinline__ float part_share(float l, int softmax) {
  float s = 0.f, total = 0.f;
  if (!softmax) {
    s = route_score(l, 0, 0.f, 1.f);
    total = part_sum<L>(s);
  }
  const bool tiny = total < 1e-18f;
  if (__any_sync(0xffffffffu, tiny)) {
    const float r = route_score(l, 1, part_max<L>(l), 1.f);
    const float all = part_sum<L>(r);
    if (tiny) {
      s = r;
      total = all;
    }
  }
  return total > 0.f ? s / total : 0.f;
}

// CH loads of VL elements per lane; expert of value (c, i): (c * L + s) * VL + i for
// the token's lane s.
template <typename T, int VL, int CH, int L>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, 7) route_short_kernel(const RouteParams p) {
  constexpr int NV = VL * CH, TOKENS = 32 / L;
  static_assert(NV % 2 == 0 && NV <= 32, "two maxima a lane");
  extern __shared__ __align__(16) uint8_t route_smem[];
  pdl_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = lane & (L - 1), sub = lane / L;
  const long long t0 = (static_cast<long long>(blockIdx.x) * ROUTE_WARPS + warp) * TOKENS;
  if (t0 >= p.T) return;
  const long long t = t0 + sub;
  const bool valid = t < p.T;
  const int E = p.E, k = p.k;
  const bool biased = p.bias != nullptr;
  const bool grouped = p.keep < p.groups;
  const T* const rows = static_cast<const T*>(p.logits) + t0 * E;
  const T* const row = rows + static_cast<long long>(valid ? sub : 0) * E;
  const int token_bytes = route_short_token_bytes(E);
  uint8_t* const smem = route_smem + warp * TOKENS * token_bytes;
  uint8_t* const mem = smem + sub * token_bytes;
  unsigned long long* const list = reinterpret_cast<unsigned long long*>(mem);
  float* const val = reinterpret_cast<float*>(mem);
  float* const gtol = val + E;  // (at most E groups)
  float* const gscore = reinterpret_cast<float*>(mem + route_short_tail(E));
  unsigned long long* const chosen = reinterpret_cast<unsigned long long*>(gscore);
  uint16_t* const cand = reinterpret_cast<uint16_t*>(mem + route_short_cand(E));

  // logits (a NaN is below every number in the comparisons and maxima below)
  float key[NV];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e0 = (c * L + s) * VL;
#pragma unroll
    for (int i = 0; i < VL; ++i) key[c * VL + i] = -INFINITY;
    if (valid && e0 < E) op_load<T, VL>(row + e0, key + c * VL);
  }
  float m = -INFINITY, inv_z = 1.f, smax = 1.f;
  const bool need_scores = biased || (grouped && p.gtop == 2);
  if (p.softmax && (need_scores || !p.renorm)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      key[i] = fmaxf(key[i], -INFINITY);  // NaN as masked
      m = fmaxf(m, key[i]);
    }
    m = part_max<L>(m);
    float z4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) z4[i & 3] += route_exp(key[i], m);
    const float z = part_sum<L>((z4[0] + z4[1]) + (z4[2] + z4[3]));
    inv_z = z > 0.f ? 1.0f / z : 0.f;
    smax = inv_z;
  }
  // keys as in route_kernel: to route_tol or, for sigmoid + bias without groups, to
  // route_coarse_tol
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
      const int e0 = (c * L + s) * VL;
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
      const int e0 = (c * L + s) * VL;
      if (e0 < E) {
        float b[VL];
#pragma unroll
        for (int i = 0; i < VL; ++i) b[i] = 0.f;
        if (biased) op_load_f32<VL>(p.bias + e0, b);
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const float l = key[c * VL + i];
          const float x = p.softmax ? route_exp(l, m) * inv_z : __fdividef(1.0f, 1.0f + __expf(-l));
          float v = x + b[i];
          if (l == -INFINITY || v != v) v = -INFINITY;
          if (grouped) val[e0 + i] = v;
          if (biased) key[c * VL + i] = v;
        }
      }
    }
  } else if (grouped) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e0 = (c * L + s) * VL;
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (e0 < E) val[e0 + i] = key[c * VL + i];
    }
  }

  uint32_t kept = 0xffffffffu;
  if (grouped) {
    __syncwarp();
    // a lane per group (lanes start at different values: groups often lie a multiple
    // of 32 banks apart)
    for (int g = s; g < p.groups; g += L) {
      float a = -INFINITY, b = -INFINITY;
      int j = s < p.gsize ? s : 0;
      for (int n = 0; n < p.gsize; ++n) {
        const float v = val[g * p.gsize + j];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
        if (++j == p.gsize) j = 0;
      }
      if (p.gtop == 1) b = -INFINITY;
      gscore[g] = b != -INFINITY ? a + b : a;
      gtol[g] = route_group_tol(p.softmax, smax, a, b);
    }
    __syncwarp();
    // equal scores go to the lower group
    uint32_t mine = 0u;
    float lo = INFINITY, hi = -INFINITY;
    for (int g = s; g < p.groups; g += L) {
      const float score = gscore[g];
      int rank = 0;
      for (int o = 0; o < p.groups; ++o) {
        const float so = gscore[o];
        rank += (so > score || (so == score && o < g)) ? 1 : 0;
      }
      // the least that a kept group may have, the most of one left out
      if (rank < p.keep) {
        mine |= 1u << g;
        lo = fminf(lo, score - gtol[g]);
      } else if (score != -INFINITY) {
        hi = fmaxf(hi, score + gtol[g]);
      }
    }
    __syncwarp();
    kept = mine;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) kept |= __shfl_xor_sync(0xffffffffu, kept, o);
    if (need_scores) {
      lo = -part_max<L>(-lo);
      hi = part_max<L>(hi);
      const uint32_t near = __ballot_sync(0xffffffffu, valid && hi != -INFINITY && !(lo > hi));
      if (near != 0u) {
        const int lpg = 32 >> (32 - __clz(p.groups - 1));
#pragma unroll 1
        for (int q = 0; q < TOKENS; ++q) {
          if (((near >> (q * L)) & 1u) == 0u) continue;
          const T* r = rows + static_cast<long long>(q) * E;
          const double mq = __shfl_sync(0xffffffffu, m, q * L);
          const float smaxq = __shfl_sync(0xffffffffu, smax, q * L);
          const double z = p.softmax ? route_sum64(r, E, mq, lane) : 0.0;
          const uint32_t exact =
              route_keep64<T>(p, r, reinterpret_cast<const float*>(smem + q * token_bytes), smaxq, mq, z, lane, lpg);
          if (sub == q) kept = exact;
        }
      }
    }
    const bool whole = VL == 1 || p.gsize % VL == 0;  // a load lies in one group
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const unsigned e0 = (c * L + s) * VL;  // (past E: -inf already, any group will do)
      bool in = (kept >> (((e0 * p.gmagic) >> 20) & 31u)) & 1u;
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        if (!whole) in = (kept >> ((((e0 + i) * p.gmagic) >> 20) & 31u)) & 1u;
        if (!in) key[c * VL + i] = -INFINITY;
      }
    }
    __syncwarp();
  }

  // lower bound of the k-th largest key: the k-th largest of two maxima a lane, over
  // half its keys each
  float lm = -INFINITY, lm2 = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; i += 2) {
    lm = fmaxf(lm, key[i]);
    lm2 = fmaxf(lm2, key[i + 1]);
  }
  lm = part_sort_desc<L>(lm, lane);
  lm2 = __shfl_xor_sync(0xffffffffu, part_sort_desc<L>(lm2, lane), L - 1);
  lm = fmaxf(lm, lm2);
#pragma unroll
  for (int j = L / 2; j > 0; j >>= 1) lm = cmpx(lm, lane, j, true);
  float thr = __shfl_sync(0xffffffffu, lm, (lane & ~(L - 1)) + k - 1);
  if (biased) thr -= 2.f * (coarse ? route_coarse_tol(thr) : route_tol(p.softmax, smax, thr));
  thr = fmaxf(thr, -FLT_MAX);  // never -inf (or inf - inf)
  // the keys at or above it, by number
  uint32_t hits = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) hits |= key[i] >= thr ? 1u << i : 0u;
  int at = __popc(hits);
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (s >= o) at += v;
  }
  const int cnt = __shfl_sync(0xffffffffu, at, lane | (L - 1));
  at -= __popc(hits);
  for (; hits != 0u; hits &= hits - 1u) {
    const int i = __ffs(static_cast<int>(hits)) - 1;
    cand[at++] = static_cast<uint16_t>(((i / VL) * L + s) * VL + i % VL);
  }
  __syncwarp();
  // their keys
  for (int q = s; q < cnt; q += L) {
    const int x = cand[q];
    const float lx = route_logit(op_f32(row[x]));
    float v = lx;
    if (biased) {
      v = (p.softmax ? route_exp(lx, m) * inv_z : __fdividef(1.0f, 1.0f + __expf(-lx))) + p.bias[x];
      if (v != v) v = -INFINITY;
    }
    list[q] = route_pack(v, x);
  }
  if (s == 0) list[cnt] = 0ull;
  __syncwarp();
  // the count of larger ones is the place of each
  for (int q = s; q < cnt; q += L) {
    const unsigned long long mine = list[q];
    int rank = 0;
    const ulonglong2* l2 = reinterpret_cast<const ulonglong2*>(list);
#pragma unroll 4
    for (int j = 0; 2 * j < cnt; ++j) {
      const ulonglong2 o = l2[j];
      if (o.x > mine) ++rank;
      if (o.y > mine) ++rank;
    }
    if (rank < k) chosen[rank] = mine;
  }
  __syncwarp();
  unsigned long long top = 0ull;
  int e = 0;
  float l = -INFINITY, b = 0.f;
  if (s < min(k, cnt)) {
    top = chosen[s];
    e = route_expert(top);
    l = route_logit(op_f32(row[e]));
    if (biased) b = p.bias[e];
  }
  __syncwarp();
  const float kk = top != 0ull ? f32_unorder(static_cast<uint32_t>(top >> 32)) : -INFINITY;
  // chosen by key; the others by index.  (A listed key may be -inf: a NaN or -inf bias
  // under a coarse threshold.)
  const int nsel = __popc(__ballot_sync(0xffffffffu, kk != -INFINITY) >> (sub * L) & ((1u << L) - 1u));
  if (biased) {
    const float k2 = __shfl_down_sync(0xffffffffu, kk, 1);
    const float l2 = __shfl_down_sync(0xffffffffu, l, 1);
    const float b2 = __shfl_down_sync(0xffffffffu, b, 1);
    // neighbours among the chosen: apart, or equal in logit and bias (then the
    // index has ordered them)
    bool bad = s + 1 < nsel && !(kk - k2 > 2.f * route_tol(p.softmax, smax, kk)) && !(l == l2 && b == b2);
    // the last chosen against all that were left out
    const int last = (lane & ~(L - 1)) + (nsel > 0 ? nsel - 1 : 0);
    const unsigned long long tl = __shfl_sync(0xffffffffu, top, last);
    const float ll = __shfl_sync(0xffffffffu, l, last);
    const float bl = __shfl_sync(0xffffffffu, b, last);
    const float kl = f32_unorder(static_cast<uint32_t>(tl >> 32));
    const float tol = 2.f * route_tol(p.softmax, smax, kl);
    for (int q = nsel > 0 ? s : cnt; q < cnt; q += L) {
      const unsigned long long o = list[q];
      if (o >= tl || kl - f32_unorder(static_cast<uint32_t>(o >> 32)) > tol) continue;
      const int x = route_expert(o);
      if (route_logit(op_f32(row[x])) != ll || p.bias[x] != bl) bad = true;
    }
    __syncwarp();
    const uint32_t near = __ballot_sync(0xffffffffu, bad);
    if (near != 0u) {
#pragma unroll 1
      for (int q = 0; q < TOKENS; ++q) {
        if (((near >> (q * L)) & ((1u << L) - 1u)) == 0u) continue;
        const T* r = rows + static_cast<long long>(q) * E;
        const double mq = __shfl_sync(0xffffffffu, m, q * L);
        const int cq = __shfl_sync(0xffffffffu, cnt, q * L);
        const uint16_t* of = reinterpret_cast<const uint16_t*>(smem + q * token_bytes + route_short_cand(E));
        const double z = p.softmax ? route_sum64(r, E, mq, lane) : 0.0;
        const int x = __shfl_sync(0xffffffffu, route_resolve<T>(p, r, of, cq, mq, z, lane), s);
        __syncwarp();
        if (sub == q && s < nsel) {
          e = max(0, x);
          l = route_logit(op_f32(row[e]));
        }
      }
    }
  }
  const uint32_t short_of = __ballot_sync(0xffffffffu, valid && nsel < k);
  if (short_of != 0u) {
    // masked experts of the kept groups fill up, in ascending order
#pragma unroll 1
    for (int q = 0; q < TOKENS; ++q) {
      if (((short_of >> (q * L)) & 1u) == 0u) continue;
      const T* r = rows + static_cast<long long>(q) * E;
      const uint32_t kq = __shfl_sync(0xffffffffu, kept, q * L);
      const int first = __shfl_sync(0xffffffffu, nsel, q * L);
      int have = first, mine = 0;
      for (int e0 = 0; e0 < E && have < k; e0 += 32) {
        const int x = e0 + lane;
        bool is = false;
        if (x < E && ((kq >> ((static_cast<unsigned>(x) * p.gmagic) >> 20)) & 1u)) {
          const float lx = route_logit(op_f32(r[x]));
          const float bx = biased ? p.bias[x] : 0.f;
          is = lx == -INFINITY || bx == -INFINITY || bx != bx;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, is);
        const int want = lane - have;  // the lane's place among these
        if (lane >= have && want < __popc(mask)) mine = e0 + static_cast<int>(__fns(mask, 0, want + 1));
        have += __popc(mask);
      }
      mine = __shfl_sync(0xffffffffu, mine, s);
      if (sub == q && s >= first && s < k) {
        e = mine;
        l = route_logit(op_f32(row[e]));
      }
    }
  }

  if (s >= k) l = -INFINITY;
  const float out = (p.renorm ? part_share<L>(l, p.softmax) : route_score(l, p.softmax, m, inv_z)) * p.scale;
  if (valid && s < k) {
    p.idx[t * k + s] = e;
    p.w[t * k + s] = out;
  }
}

}  // namespace moe
