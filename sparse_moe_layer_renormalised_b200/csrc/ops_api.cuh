// C-ABI entry points of the operators around the layer (see include/moe_ops.h):
// host-side validation, choice of the kernel variant and launches.  Included by
// moe_api.cu, whose helpers and device fault flag it shares.
#pragma once

#include "clip.cuh"
#include "linear.cuh"
#include "norm.cuh"
#include "route_short.cuh"
#include "../../include/moe_ops.h"

namespace moe {
namespace {

bool op_type_ok(int t) { return t == MOE_F32 || t == MOE_BF16 || t == MOE_F16; }
int op_type_bytes(int t) { return t == MOE_F32 ? 4 : 2; }
bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
bool ws_fits(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws != nullptr && (reinterpret_cast<uintptr_t>(ws) % kAlign) == 0 && have >= need);
}

// SMs of the current device, asked for once.
int op_sms() {
  static int cache[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return num_sms();
  if (cache[dev] == 0) cache[dev] = num_sms();
  return cache[dev];
}

// Allows a kernel `smem` bytes of dynamic shared memory (at every call: what was
// allowed goes with the device's context).
template <typename K>
cudaError_t op_allow_smem(K kern, size_t smem) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
}

// Launches a kernel so that it may be set up before the one ahead of it in the
// stream has ended (its pdl_wait() waits for that); `cluster` CTAs a cluster.
template <typename K, typename... A>
cudaError_t op_launch(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  ++g_last_launches;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Calls f with a value of the element type of dtype t.
template <typename F>
void with_type(int t, F f) {
  if (t == MOE_F32)
    f(float());
  else if (t == MOE_BF16)
    f(__nv_bfloat16());
  else
    f(__half());
}

template <int V>
struct Const {
  static constexpr int value = V;
};

// ------------------------------------------------------------------------------ routing
bool route_ok(const moe_route_desc* d) {
  if (d == nullptr || d->T < 0 || d->T > 0x7fffffffLL) return false;
  if (d->E < 1 || d->E > ROUTE_MAX_E || d->k < 1 || d->k > 32) return false;
  if (d->groups < 1 || d->groups > 32 || d->E % d->groups != 0) return false;
  if (d->keep_groups < 1 || d->keep_groups > d->groups) return false;
  const int gsize = d->E / d->groups;
  if (d->k > d->keep_groups * gsize) return false;
  if (d->group_top < 1 || d->group_top > 2 || d->group_top > gsize) return false;
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID) return false;
  return std::isfinite(d->scale) && op_type_ok(d->dtype);
}

RouteParams route_params(const moe_route_desc& d) {
  RouteParams p{};
  p.T = d.T;
  p.E = d.E;
  p.k = d.k;
  p.groups = d.groups;
  p.gsize = d.E / d.groups;
  p.keep = d.keep_groups;
  p.gtop = d.group_top;
  p.gmagic = ((1u << 20) + p.gsize - 1) / p.gsize;
  p.softmax = d.score == MOE_SCORE_SOFTMAX;
  p.renorm = d.renorm != 0;
  p.scale = d.scale;
  return p;
}

// Calls f(CH, VL as constants) with the fewest loads per lane that hold a row of E
// elements: 16-byte loads where the rows are made of whole ones, else one element
// a load.
template <typename T, typename F>
void route_dispatch(int E, F f) {
  constexpr int V = kVec<T>;
  if (E % V == 0) {
    switch (cdiv(E, 32 * V)) {
      case 1: return f(Const<V>(), Const<1>());
      case 2: return f(Const<V>(), Const<2>());
      case 3: return f(Const<V>(), Const<3>());
      case 4: return f(Const<V>(), Const<4>());
    }
    if constexpr (V == 4) {
      switch (cdiv(E, 32 * V)) {
        case 5: return f(Const<V>(), Const<5>());
        case 6: return f(Const<V>(), Const<6>());
        case 7: return f(Const<V>(), Const<7>());
        default: return f(Const<V>(), Const<8>());
      }
    }
  }
  if (E <= 128) return f(Const<1>(), Const<4>());
  if (E <= 256) return f(Const<1>(), Const<8>());
  if (E <= 512) return f(Const<1>(), Const<16>());
  return f(Const<1>(), Const<32>());
}

// Whether route_short_kernel takes the rows: up to 128 experts, and more rows than the
// GPU holds warps of route_kernel (32 a SM).  Top 8 of 128 softmax scores in bf16: 12.5 against
// 24.0 us for 32767 rows, with a bias 10.2 against 8.6 for 2048; top 8 of 256
// sigmoid scores plus bias, 16384 rows of fp32: 17.4 against 16.2.
bool route_is_short(const moe_route_desc& d) { return d.E <= 128 && d.k <= 16 && d.T > 32LL * op_sms(); }

template <typename T, int VL, int CH, int L>
cudaError_t route_launch_short(const RouteParams& p, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(cdiv(p.T, ROUTE_WARPS * (32 / L)));
  const size_t smem = static_cast<size_t>(ROUTE_WARPS) * (32 / L) * route_short_token_bytes(p.E);  // (below 48 KB)
  return op_launch(route_short_kernel<T, VL, CH, L>, blocks, ROUTE_WARPS * 32, smem, s, 0, p);
}
template <typename T>
cudaError_t route_short(const RouteParams& p, cudaStream_t s) {
  constexpr int V = kVec<T>;
  const bool whole = p.E % V == 0;
  if (p.k > 8) return whole ? route_launch_short<T, V, 8 / V, 16>(p, s) : route_launch_short<T, 1, 8, 16>(p, s);
  if (p.E <= 64) return whole ? route_launch_short<T, V, 8 / V, 8>(p, s) : route_launch_short<T, 1, 8, 8>(p, s);
  return whole ? route_launch_short<T, V, 16 / V, 8>(p, s) : route_launch_short<T, 1, 16, 8>(p, s);
}

// ------------------------------------------------------------------------------ norms
constexpr int kNormMaxH = 16384;

bool norm_ok(const moe_norm_desc* d) {
  return d != nullptr && d->T >= 0 && d->T <= 0x7fffffffLL && d->H >= 1 &&
         (d->kind == MOE_NORM_LAYER || d->kind == MOE_NORM_RMS) && std::isfinite(d->eps) && d->eps >= 0.f &&
         op_type_ok(d->dtype);
}

// Whether rows of H elements are whole 16-byte windows, and the most windows that
// a row of them touches.
bool norm_aligned(const moe_norm_desc& d) { return d.H % (16 / op_type_bytes(d.dtype)) == 0; }
int norm_windows(const moe_norm_desc& d) {
  const int vl = 16 / op_type_bytes(d.dtype);
  return static_cast<int>(norm_aligned(d) ? d.H / vl : cdiv(d.H + vl - 1, vl));
}

// How the kernels lay a row length out: nw windows a thread, tpg threads a group,
// as many groups as the block, the named barriers or the rows allow, and rings as
// deep as the shared memory is.
struct NormPlan {
  int nw, tpg, groups, stages, row_bytes, par_floats, blocks;
  size_t smem;
};
NormPlan norm_plan(const moe_norm_desc& d, bool backward) {
  const int vl = 16 / op_type_bytes(d.dtype), windows = norm_windows(d), ops = backward ? 2 : 1;
  NormPlan q{};
  const int threads = backward ? NORM_BWD_THREADS : NORM_FWD_THREADS;
  q.nw = windows <= 32 ? 1 : windows <= 64 ? 2 : windows <= 4 * threads ? 4 : static_cast<int>(cdiv(windows, threads));
  if (q.nw > 4 && vl == 4 && q.nw < 8) q.nw = 8;  // (fewer variants)
  q.tpg = static_cast<int>(cdiv(windows, 32 * q.nw) * 32);
  q.groups = std::max(1, std::min(q.tpg > 32 ? 14 : 32, threads / q.tpg));
  q.groups = static_cast<int>(std::max<long long>(1, std::min<long long>(q.groups, cdiv(d.T, op_sms()))));
  q.row_bytes = windows * 16;
  // gamma and beta in shared memory, unless rows of whole windows are so long that
  // they would leave less than two stages, or so few that no group takes a second one
  const size_t par_bytes = static_cast<size_t>(windows) * vl * (backward ? 4 : 8);
  if (!norm_aligned(d) || (par_bytes + 2 * static_cast<size_t>(ops) * q.row_bytes <= 224 * 1024 &&
                           d.T > static_cast<long long>(q.groups) * op_sms()))
    q.par_floats = windows * vl;
  // three stages at least are worth a group
  for (;; --q.groups) {
    const size_t head = norm_head(q.groups) + static_cast<size_t>(q.par_floats) * (backward ? 4 : 8);
    const size_t group = static_cast<size_t>(ops) * q.row_bytes * q.groups;
    q.stages = static_cast<int>(std::max<size_t>(1, std::min<size_t>(NORM_MAX_RING, (226 * 1024 - head) / group)));
    q.smem = head + std::max<size_t>(group * q.stages, backward && q.groups > 1 ? static_cast<size_t>(q.groups) * d.H * 8 : 0);
    if (q.stages >= 3 || q.groups <= 2) break;
  }
  q.blocks = static_cast<int>(std::max<long long>(1, std::min<long long>(cdiv(d.T, q.groups), op_sms())));
  // the rows of a block start at one offset in a window: they lie as many rows apart
  // as there are blocks, a multiple of a window's elements (or are one a block)
  if (!norm_aligned(d) && d.T > q.blocks) q.blocks = std::max(vl, q.blocks - q.blocks % vl);
  return q;
}

template <typename K>
moe_status norm_launch(K kern, const NormParams& p, const NormPlan& q, cudaStream_t s) {
  if (op_allow_smem(kern, q.smem) != cudaSuccess) return MOE_ERR_CUDA;
  return op_launch(kern, q.blocks, q.tpg * q.groups, q.smem, s, 0, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T, bool ALIGNED, bool PAR, bool BACKWARD>
moe_status norm_dispatch(const NormParams& p, const NormPlan& q, cudaStream_t s) {
  auto go = [&](auto nw) {
    constexpr int NW = decltype(nw)::value;
    if constexpr (BACKWARD) return norm_launch(norm_backward_kernel<T, NW, ALIGNED, PAR>, p, q, s);
    else return norm_launch(norm_kernel<T, NW, ALIGNED, PAR>, p, q, s);
  };
  // (16-bit rows have at most 2049 windows, fp32 ones 4097)
  if (q.nw == 1) return go(Const<1>());
  if (q.nw == 2) return go(Const<2>());
  if (q.nw == 4) return go(Const<4>());
  if constexpr (sizeof(T) == 4) {
    if (q.nw == 8) return go(Const<8>());
    if constexpr (BACKWARD)
      if (q.nw == 9) return go(Const<9>());
  } else if constexpr (BACKWARD) {
    if (q.nw == 5) return go(Const<5>());
  }
  return MOE_ERR_UNSUPPORTED;
}

template <bool BACKWARD>
moe_status norm_run(const moe_norm_desc& d, NormParams p, cudaStream_t s) {
  const NormPlan q = norm_plan(d, BACKWARD);
  p.T = d.T;
  p.H = d.H;
  p.eps = d.eps;
  p.inv_h = 1.0f / static_cast<float>(d.H);
  p.rms = d.kind == MOE_NORM_RMS;
  p.tpg = q.tpg;
  p.groups = q.groups;
  p.walkers = static_cast<long long>(q.blocks) * q.groups;
  p.stages = q.stages;
  p.row_bytes = q.row_bytes;
  p.par_floats = q.par_floats;
  moe_status st = MOE_OK;
  with_type(d.dtype, [&](auto v) {
    using T = decltype(v);
    st = !norm_aligned(d)      ? norm_dispatch<T, false, true, BACKWARD>(p, q, s)
         : q.par_floats != 0 ? norm_dispatch<T, true, true, BACKWARD>(p, q, s)
                             : norm_dispatch<T, true, false, BACKWARD>(p, q, s);
  });
  return st;
}

// Column sums of part[parts][width] (see column_sum_kernel).
moe_status column_sums(const float* part, int parts, int width, int H, float* a_out, float* b_out, cudaStream_t s) {
  const dim3 block(32, COLSUM_SLICES);
  const cudaError_t e =
      width % 4 == 0 ? op_launch(column_sum_kernel<4>, static_cast<unsigned>(cdiv(width, 128)), block, 0, s, 0, part, parts, width, H, a_out, b_out)
                     : op_launch(column_sum_kernel<1>, static_cast<unsigned>(cdiv(width, 32)), block, 0, s, 0, part, parts, width, H, a_out, b_out);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// ------------------------------------------------------------------------------ linear
bool lin_ok(const moe_linear_desc* d) {
  return d != nullptr && d->M >= 0 && d->M <= 0x7fffffffLL && d->N >= 1 && d->K >= 1 && d->act >= MOE_ACT_NONE &&
         d->act <= MOE_ACT_GELU_TANH && op_type_ok(d->dtype) && (d->y_out == MOE_F32 || d->y_out == d->dtype);
}
moe_status lin_check(const moe_linear_desc* d) {
  if (!lin_ok(d)) return MOE_ERR_INVALID_ARG;
  return d->dtype == MOE_F32 || d->N % 8 != 0 || d->K % 8 != 0 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// One product out[Q, P] = f(sum over R): operand p is [P, R] (or, MN-major, lies
// as [R, P]), operand q [Q, R] (or [R, Q]).
struct LinProblem {
  const void *p, *q;
  bool p_mn, q_mn;
  long long P, Q, R;
};

bool lin_map(CUtensorMap* m, const void* base, bool mn, long long rows, long long R, int box_rows) {
  return mn ? make_map(m, base, R, rows, rows, LIN_BK) : make_map(m, base, rows, R, R, box_rows);
}

// Boxes of 32 x 32 16-bit values of a [Q, P] matrix, 64-byte swizzle.
bool lin_box_map(CUtensorMap* m, const void* base, long long Q, long long P) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(P), static_cast<cuuint64_t>(Q)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(P) * 2};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles of the wide kernel: their width, how many are done whole, and in how many
// parts each of the others.
struct LinWidePlan {
  int bn, p_tiles, q_tiles, full, split;
  long long items() const { return full + (static_cast<long long>(p_tiles) * q_tiles - full) * split; }
};

// The width with the least time by this count: a tile's k-block costs about as the
// 256 + bn operand rows that are fetched for it (measured at 8192 x 7168 x 3584 and
// 4001 x 3584 x 7168 with widths of 160 to 256); full waves cost one tile each, a
// last one that is split into s parts 1 / s and a little more.
LinWidePlan lin_wide_plan(long long Q, long long P, int nkb, int pairs) {
  LinWidePlan best{};
  double cost = 0.0;
  for (int bn = 256; bn >= 128; bn -= 32) {
    LinWidePlan w{};
    w.bn = bn;
    w.q_tiles = static_cast<int>(cdiv(Q, 256));
    w.p_tiles = static_cast<int>(cdiv(P, bn));
    const long long tiles = static_cast<long long>(w.q_tiles) * w.p_tiles, waves = tiles / pairs, rest = tiles - waves * pairs;
    w.split = 1;
    // parts of eight k-blocks at least
    if (rest > 0) w.split = static_cast<int>(std::max<long long>(1, std::min<long long>(pairs / rest, nkb / 8)));
    w.full = static_cast<int>(w.split > 1 ? waves * pairs : tiles);
    const double c = (waves + (rest == 0 ? 0.0 : w.split > 1 ? 1.0 / w.split + 0.1 : 1.0)) * (256 + bn);
    if (best.bn == 0 || c < cost) {
      best = w;
      cost = c;
    }
  }
  return best;
}

// Bytes for the partial sums of a last wave, whatever the plan: one tile a pair.
size_t lin_wide_ws() { return static_cast<size_t>(op_sms() / 2) * 256 * 256 * 4; }

// The skinny kernel for few rows, one tile of them (bf16, skinny against wide: 32 x 7168 x
// 3584 13.4 and 22.7 us, 128 rows 17.0 and 23.5; two tiles fetch the weights twice: 160 rows
// 22.5 and 23.8, which is not worth a rule of its own, and 512 rows 36 and 28.6), and for
// outputs whose 128 x 128 tiles take half of the SMs at most: it splits their sums
// over several CTAs (1024 x 896 x 7168 20.7 and 22.5, 1024 x 1024 x 1024 10.6 and 13.3; 1024
// x 2048 x 2048, 128 tiles, 23.4 and 20.4).
bool lin_is_skinny(long long Q, long long P) {
  return Q <= 128 || cdiv(Q, 128) * cdiv(P, 128) <= op_sms() / 2;
}

template <typename OutT>
cudaError_t lin_launch_wide(const LinProblem& g, LinParams& p, cudaStream_t s) {
  auto kern = linear_wide_kernel<OutT>;
  cudaError_t e = op_allow_smem(kern, LW_SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(LW_THREADS);
  cfg.dynamicSmemBytes = LW_SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static int pairs_cache[128] = {};
  const int pairs = cluster_pairs(kern, cfg, pairs_cache);
  const LinWidePlan w = lin_wide_plan(g.Q, g.P, p.nkb, std::min(pairs, op_sms() / 2));
  p.bn = w.bn;
  p.q_tiles = w.q_tiles;
  p.p_tiles = w.p_tiles;
  p.full = w.full;
  p.split = w.split;
  LinMaps maps;
  std::memset(&maps, 0, sizeof maps);
  if (!lin_map(&maps.p, g.p, g.p_mn, g.P, g.R, p.bn / 2) || !lin_map(&maps.q, g.q, g.q_mn, g.Q, g.R, 128))
    return cudaErrorInvalidValue;
  if (sizeof(OutT) == 2) {
    if (!lin_box_map(&maps.out, p.out, g.Q, g.P) || (p.residual != nullptr && !lin_box_map(&maps.res, p.residual, g.Q, g.P)) ||
        (p.pre != nullptr && !lin_box_map(&maps.pre, p.pre, g.Q, g.P)))
      return cudaErrorInvalidValue;
  }
  e = op_launch(kern, 2 * static_cast<unsigned>(std::min<long long>(pairs, w.items())), LW_THREADS, LW_SMEM, s, 2, maps, p);
  const long long rest = static_cast<long long>(w.p_tiles) * w.q_tiles - w.full;
  if (e == cudaSuccess && rest > 0)
    e = op_launch(linear_fixup_kernel<OutT>, static_cast<unsigned>(rest * (w.bn / 4)), 256, 0, s, 0, p);
  return e;
}

template <typename OutT, int BN, bool QMN>
cudaError_t lin_launch_skinny_inst(const LinProblem& g, LinParams& p, cudaStream_t s) {
  using C = LsCfg<BN, QMN>;
  auto kern = linear_skinny_kernel<OutT, BN, QMN>;
  cudaError_t e = op_allow_smem(kern, C::kSmem);
  if (e != cudaSuccess) return e;
  p.bn = BN;
  p.p_tiles = static_cast<int>(cdiv(g.P, 128));
  p.q_tiles = static_cast<int>(cdiv(g.Q, BN));
  // as many CTAs on the sum as the SMs hold with certainty, two each (clusters have to
  // fit their part of the chip: at 1.9 a SM some waited for others, 16.9 instead of
  // 15.9 us at 4 x 7168 x 3584), each with a few blocks of it
  const long long tiles = static_cast<long long>(p.p_tiles) * p.q_tiles;
  const int split = static_cast<int>(
      std::max<long long>(1, std::min<long long>({LS_MAX_SPLIT, 16LL * op_sms() / 10 / tiles, p.nkb / 2})));
  LinMaps maps;
  std::memset(&maps, 0, sizeof maps);
  if (!lin_map(&maps.p, g.p, g.p_mn, g.P, g.R, 128) || !lin_map(&maps.q, g.q, g.q_mn, g.Q, g.R, BN))
    return cudaErrorInvalidValue;
  return op_launch(kern, dim3(static_cast<unsigned>(p.p_tiles * split), static_cast<unsigned>(p.q_tiles)), LS_THREADS,
                   C::kSmem, s, split, maps, p);
}

template <typename OutT, int BN>
cudaError_t lin_launch_skinny(const LinProblem& g, LinParams& p, cudaStream_t s) {
  return g.q_mn ? lin_launch_skinny_inst<OutT, BN, true>(g, p, s) : lin_launch_skinny_inst<OutT, BN, false>(g, p, s);
}

template <typename OutT>
moe_status lin_product(const LinProblem& g, LinParams p, cudaStream_t s) {
  p.P = static_cast<int>(g.P);
  p.Q = g.Q;
  p.nkb = static_cast<int>(cdiv(g.R, LIN_BK));
  p.p_mn = g.p_mn;
  p.q_mn = g.q_mn;
  if (cdiv(g.Q, 256) * cdiv(g.P, 128) > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  cudaError_t e;
  if (lin_is_skinny(g.Q, g.P)) {
    e = g.Q <= 16   ? lin_launch_skinny<OutT, 16>(g, p, s)
        : g.Q <= 32 ? lin_launch_skinny<OutT, 32>(g, p, s)
        : g.Q <= 64 ? lin_launch_skinny<OutT, 64>(g, p, s)
                    : lin_launch_skinny<OutT, 128>(g, p, s);
  } else {
    e = lin_launch_wide<OutT>(g, p, s);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status lin_product_of(int out_type, const LinProblem& g, const LinParams& p, cudaStream_t s) {
  if (out_type == MOE_F32) return lin_product<float>(g, p, s);
  return out_type == MOE_BF16 ? lin_product<__nv_bfloat16>(g, p, s) : lin_product<__half>(g, p, s);
}

// Blocks along the rows of the dp kernel: about eight a SM in all.
long long lin_dp_parts(const moe_linear_desc& d) {
  const long long across = cdiv(d.N, LIN_DP_THREADS * 8);
  return std::max<long long>(1, std::min<long long>({d.M, cdiv(8LL * op_sms(), across), 65535}));
}
size_t lin_dp_bytes(const moe_linear_desc& d) {
  return d.act == MOE_ACT_NONE ? 0 : round_up(static_cast<size_t>(d.M) * d.N * 2, kAlign);
}

// ------------------------------------------------------------------------------ clipping
constexpr int kClipMaxTensors = 65536;

bool clip_list_ok(const moe_grad_tensor* list, int32_t count) {
  if (count < 0 || count > kClipMaxTensors || (count > 0 && list == nullptr)) return false;
  for (int i = 0; i < count; ++i) {
    const moe_grad_tensor& t = list[i];
    if (t.n < 0 || t.n > (1LL << 44) || !op_type_ok(t.dtype)) return false;
    if (t.n == 0) continue;
    const uintptr_t mask = static_cast<uintptr_t>(op_type_bytes(t.dtype)) - 1;
    if (t.in == nullptr || t.out == nullptr || (reinterpret_cast<uintptr_t>(t.in) & mask) ||
        (reinterpret_cast<uintptr_t>(t.out) & mask))
      return false;
  }
  return true;
}

// Launches over the list, and the most blocks of each.
int clip_launches(int32_t count) { return std::max(1, static_cast<int>(cdiv(count, CLIP_MAX))); }
int clip_blocks() { return 8 * op_sms(); }

// 16-byte vectors that a tensor touches.
long long clip_vectors(const moe_grad_tensor& t) {
  const long long es = op_type_bytes(t.dtype), skew = static_cast<long long>(reinterpret_cast<uintptr_t>(t.in) & 15u) / es;
  return cdiv((t.n + skew) * es, 16);
}

// Vectors of a chunk: 64 KB, halved down to 8 KB while the whole list would not give
// every block one.
int clip_chunk_vectors(const moe_grad_tensor* list, int32_t count) {
  long long total = 0;
  for (int i = 0; i < count; ++i)
    if (list[i].n > 0) total += clip_vectors(list[i]);
  int chunk = 2 * CLIP_LOADS * CLIP_THREADS;
  while (chunk > 2 * CLIP_THREADS && total < static_cast<long long>(chunk) * clip_blocks()) chunk /= 2;
  return chunk;
}

template <int MAXT>
moe_status clip_run(const moe_grad_tensor* list, int32_t count, bool max_norm_kind, float max_norm, float* norm_out,
                    double* partial, cudaStream_t s) {
  const int nl = clip_launches(count);
  int parts = 0;  // partial sums written by the first pass
  const int chunk = clip_chunk_vectors(list, count);
  for (int pass = 0; pass < 2; ++pass) {
    for (int li = 0; li < nl; ++li) {
      ClipList<MAXT> l;
      l.count = 0;
      l.chunk = chunk;
      long long chunks = 0;
      for (int i = li * CLIP_MAX; i < std::min<long long>(count, (li + 1LL) * CLIP_MAX); ++i) {
        const moe_grad_tensor& t = list[i];
        if (t.n == 0) continue;
        const int k = l.count++;
        l.in[k] = t.in;
        l.out[k] = t.out;
        l.n[k] = t.n;
        l.first[k] = static_cast<int>(chunks);
        l.type[k] = t.dtype == MOE_F32 ? kClipF32 : t.dtype == MOE_BF16 ? kClipBF16 : kClipF16;
        chunks += cdiv(clip_vectors(t), chunk);
      }
      if (chunks > 0x3fffffffLL) return MOE_ERR_UNSUPPORTED;
      l.chunks = static_cast<int>(chunks);
      cudaError_t e;
      const int grid = std::max(1, std::min(clip_blocks(), l.chunks));
      if (pass == 0) {
        e = op_launch(max_norm_kind ? clip_norm_kernel<MAXT, true> : clip_norm_kernel<MAXT, false>, grid, CLIP_THREADS, 0, s,
                      0, l, partial + parts);
        parts += grid;
      } else {
        float* out = li == 0 ? norm_out : nullptr;
        e = op_launch(max_norm_kind ? clip_scale_kernel<MAXT, true> : clip_scale_kernel<MAXT, false>, grid, CLIP_THREADS, 0, s,
                      0, l, static_cast<const double*>(partial), parts, max_norm, out);
      }
      if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_route(const moe_route_desc* d, const void* logits, const float* bias, int32_t* idx, float* w,
                     moe_stream_t stream) {
  using namespace moe;
  if (!route_ok(d)) return MOE_ERR_INVALID_ARG;
  g_last_launches = 0;
  if (d->T == 0) return MOE_OK;
  if (!ptr_ok(logits) || !aligned16(bias) || !ptr_ok(idx) || !ptr_ok(w)) return MOE_ERR_INVALID_ARG;
  RouteParams p = route_params(*d);
  p.logits = logits;
  p.bias = bias;
  p.idx = idx;
  p.w = w;
  const unsigned blocks = static_cast<unsigned>(cdiv(d->T, ROUTE_WARPS));
  const size_t smem = static_cast<size_t>(ROUTE_WARPS) * route_warp_bytes(d->E, d->keep_groups < d->groups);
  cudaError_t e = cudaSuccess;
  with_type(d->dtype, [&](auto v) {
    using T = decltype(v);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (route_is_short(*d)) {
      e = route_short<T>(p, st);
      return;
    }
    route_dispatch<T>(d->E, [&](auto vl, auto ch) {
      e = op_launch(route_kernel<T, decltype(vl)::value, decltype(ch)::value>, blocks, ROUTE_WARPS * 32, smem, st, 0, p);
    });
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_route_backward(const moe_route_desc* d, const void* logits, const int32_t* idx, const float* dw,
                              void* dlogits, moe_stream_t stream) {
  using namespace moe;
  if (!route_ok(d)) return MOE_ERR_INVALID_ARG;
  g_last_launches = 0;
  if (d->T == 0) return MOE_OK;
  if (!ptr_ok(logits) || !ptr_ok(idx) || !ptr_ok(dw) || !ptr_ok(dlogits)) return MOE_ERR_INVALID_ARG;
  RouteParams p = route_params(*d);
  p.logits = logits;
  const unsigned blocks = static_cast<unsigned>(cdiv(d->T, ROUTE_WARPS));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  with_type(d->dtype, [&](auto v) {
    using T = decltype(v);
    route_dispatch<T>(d->E, [&](auto vl, auto ch) {
      e = op_launch(route_backward_kernel<T, decltype(vl)::value, decltype(ch)::value>, blocks, ROUTE_WARPS * 32, 0, s, 0,
                    p, idx, dw, static_cast<T*>(dlogits));
    });
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_norm(const moe_norm_desc* d, const void* x, const float* gamma, const float* beta, void* y, float* mean,
                    float* rstd, moe_stream_t stream) {
  using namespace moe;
  if (!norm_ok(d)) return MOE_ERR_INVALID_ARG;
  if (d->kind == MOE_NORM_RMS && mean != nullptr) return MOE_ERR_INVALID_ARG;
  if (d->H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
  g_last_launches = 0;
  if (d->T == 0) return MOE_OK;
  if (!ptr_ok(x) || !ptr_ok(y) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) || !aligned16(rstd))
    return MOE_ERR_INVALID_ARG;
  NormParams p{};
  p.x = x;
  p.gamma = gamma;
  p.beta = beta;
  p.out = y;
  p.mean = mean;
  p.rstd = rstd;
  return norm_run<false>(*d, p, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_norm_backward_workspace_size(const moe_norm_desc* d) {
  using namespace moe;
  if (!norm_ok(d) || d->H > kNormMaxH) return 0;
  return round_up(static_cast<size_t>(norm_plan(*d, true).blocks) * 2 * d->H * 4, kAlign);
}

moe_status moe_norm_backward(const moe_norm_desc* d, const void* dy, const void* x, const float* gamma,
                             const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta, void* ws,
                             size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!norm_ok(d)) return MOE_ERR_INVALID_ARG;
  if (d->H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
  const bool rms = d->kind == MOE_NORM_RMS;
  if (rms && mean != nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(gamma) || !aligned16(dgamma) || !aligned16(dbeta)) return MOE_ERR_INVALID_ARG;
  if (d->T > 0 && (!ptr_ok(dy) || !ptr_ok(x) || (!rms && !ptr_ok(mean)) || !ptr_ok(rstd) || !ptr_ok(dx)))
    return MOE_ERR_INVALID_ARG;
  if (!ws_fits(ws, ws_bytes, moe_norm_backward_workspace_size(d))) return MOE_ERR_INVALID_ARG;
  g_last_launches = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(ws);
  if (d->T > 0) {
    NormParams p{};
    p.x = x;
    p.dy = dy;
    p.gamma = gamma;
    p.out = dx;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.part = part;
    const moe_status st = norm_run<true>(*d, p, s);
    if (st != MOE_OK) return st;
  }
  if (dgamma != nullptr || dbeta != nullptr)
    return column_sums(part, d->T > 0 ? norm_plan(*d, true).blocks : 0, 2 * d->H, d->H, dgamma, dbeta, s);
  return MOE_OK;
}

size_t moe_linear_workspace_size(const moe_linear_desc* d) {
  using namespace moe;
  if (lin_check(d) != MOE_OK) return 0;
  return lin_is_skinny(d->M, d->N) ? 0 : lin_wide_ws();
}

moe_status moe_linear(const moe_linear_desc* d, const void* x, const void* weight, const float* bias,
                      const void* residual, void* pre, void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  moe_status st = lin_check(d);
  if (st != MOE_OK) return st;
  g_last_launches = 0;
  if (d->M == 0) return MOE_OK;
  if (!ptr_ok(x) || !ptr_ok(weight) || !ptr_ok(y) || !aligned16(bias) || !aligned16(residual) || !aligned16(pre))
    return MOE_ERR_INVALID_ARG;
  if (!ws_fits(ws, ws_bytes, moe_linear_workspace_size(d))) return MOE_ERR_INVALID_ARG;
  LinParams p{};
  p.bf16 = d->dtype == MOE_BF16;
  p.bias = bias;
  p.residual = residual;
  p.pre = pre;
  p.out = y;
  p.act = d->act;
  p.fault_site = 200;
  p.partial = static_cast<float*>(ws);
  const LinProblem g{weight, x, false, false, d->N, d->M, d->K};
  return lin_product_of(d->y_out, g, p, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_linear_backward_workspace_size(const moe_linear_desc* d) {
  using namespace moe;
  if (lin_check(d) != MOE_OK) return 0;
  return lin_dp_bytes(*d) + round_up(static_cast<size_t>(lin_dp_parts(*d)) * d->N * 4, kAlign) + lin_wide_ws();
}

moe_status moe_linear_backward(const moe_linear_desc* d, const void* dy, const void* pre, const void* x,
                               const void* weight, void* dx, void* dweight, float* dbias, void* ws, size_t ws_bytes,
                               moe_stream_t stream) {
  using namespace moe;
  moe_status st = lin_check(d);
  if (st != MOE_OK) return st;
  if (!aligned16(dx) || !aligned16(dweight) || !aligned16(dbias)) return MOE_ERR_INVALID_ARG;
  const bool act = d->act != MOE_ACT_NONE;
  if (d->M > 0 && (!ptr_ok(dy) || (act && !ptr_ok(pre)) || (dweight != nullptr && !ptr_ok(x)) ||
                   (dx != nullptr && !ptr_ok(weight))))
    return MOE_ERR_INVALID_ARG;
  if (!ws_fits(ws, ws_bytes, moe_linear_backward_workspace_size(d))) return MOE_ERR_INVALID_ARG;
  g_last_launches = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->M == 0) {
    if (dweight != nullptr && cudaMemsetAsync(dweight, 0, static_cast<size_t>(d->N) * d->K * 2, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dbias != nullptr && cudaMemsetAsync(dbias, 0, static_cast<size_t>(d->N) * 4, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const void* dp = dy;
  if (act || dbias != nullptr) {
    void* to = act ? ws : nullptr;
    float* part = dbias != nullptr ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + lin_dp_bytes(*d)) : nullptr;
    const long long parts = lin_dp_parts(*d), rows = cdiv(d->M, parts);
    const dim3 grid(static_cast<unsigned>(cdiv(d->N, LIN_DP_THREADS * 8)), static_cast<unsigned>(cdiv(d->M, rows)));
    auto run = [&](auto v) {
      using T = decltype(v);
      return op_launch(linear_dp_kernel<T>, grid, LIN_DP_THREADS, 0, s, 0, static_cast<const T*>(dy), static_cast<const T*>(pre),
                       static_cast<T*>(to), part, static_cast<long long>(d->M), d->N, rows, static_cast<int>(d->act));
    };
    if ((d->dtype == MOE_BF16 ? run(__nv_bfloat16()) : run(__half())) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias != nullptr && (st = column_sums(part, static_cast<int>(grid.y), d->N, d->N, dbias, nullptr, s)) != MOE_OK) return st;
    if (act) dp = to;
  }
  LinParams p{};
  p.bf16 = d->dtype == MOE_BF16;
  p.act = kActNone;
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + moe_linear_backward_workspace_size(d) - lin_wide_ws());
  if (dx != nullptr) {
    p.out = dx;
    p.fault_site = 210;
    if ((st = lin_product_of(d->dtype, {weight, dp, true, false, d->K, d->M, d->N}, p, s)) != MOE_OK) return st;
  }
  if (dweight != nullptr) {
    p.out = dweight;
    p.fault_site = 220;
    if ((st = lin_product_of(d->dtype, {x, dp, true, true, d->K, d->N, d->M}, p, s)) != MOE_OK) return st;
  }
  return MOE_OK;
}

size_t moe_clip_grads_workspace_size(const moe_grad_tensor* list, int32_t count) {
  using namespace moe;
  if (!clip_list_ok(list, count)) return 0;
  return round_up(static_cast<size_t>(clip_launches(count)) * clip_blocks() * 8, kAlign);
}

moe_status moe_clip_grads(const moe_grad_tensor* list, int32_t count, moe_clip_norm kind, float max_norm,
                          float* norm_out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!clip_list_ok(list, count) || (kind != MOE_CLIP_L2 && kind != MOE_CLIP_MAX)) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(max_norm) || max_norm < 0.f) return MOE_ERR_INVALID_ARG;
  if (norm_out == nullptr || (reinterpret_cast<uintptr_t>(norm_out) & 3u)) return MOE_ERR_INVALID_ARG;
  if (!ws_fits(ws, ws_bytes, moe_clip_grads_workspace_size(list, count))) return MOE_ERR_INVALID_ARG;
  g_last_launches = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(ws);
  // few tensors: a small parameter block (the launch copies all of it)
  return count <= 64 ? clip_run<64>(list, count, kind == MOE_CLIP_MAX, max_norm, norm_out, partial, s)
                     : clip_run<CLIP_MAX>(list, count, kind == MOE_CLIP_MAX, max_norm, norm_out, partial, s);
}

}  // extern "C"
