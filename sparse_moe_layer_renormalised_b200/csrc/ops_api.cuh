// C-ABI entry points of the operators around the layer (see include/moe_ops.h):
// host-side validation, choice of the kernel variant and launches.  Included by
// moe_api.cu, whose helpers and device fault flag it shares.
#pragma once

#include "clip.cuh"
#include "norm.cuh"
#include "route.cuh"
#include "../../include/moe_ops.h"

namespace moe {
namespace {

bool op_type_ok(int t) { return t == MOE_F32 || t == MOE_BF16 || t == MOE_F16; }
int op_type_bytes(int t) { return t == MOE_F32 ? 4 : 2; }
bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
bool ws_fits(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws != nullptr && (reinterpret_cast<uintptr_t>(ws) % kAlign) == 0 && have >= need);
}
moe_status launched() { return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

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

template <typename T, int VL, int CH>
void route_launch(const RouteParams& p, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(cdiv(p.T, ROUTE_WARPS));
  route_kernel<T, VL, CH><<<blocks, ROUTE_WARPS * 32, static_cast<size_t>(ROUTE_WARPS) * p.E * 8, s>>>(p);
}

// The fewest loads per lane that hold the row; 16-byte loads where the rows
// are made of whole ones, else one element a load.
template <typename T>
void route_dispatch(const RouteParams& p, cudaStream_t s) {
  constexpr int V = kVec<T>;
  if (p.E % V == 0) {
    switch (cdiv(p.E, 32 * V)) {
      case 1: return route_launch<T, V, 1>(p, s);
      case 2: return route_launch<T, V, 2>(p, s);
      case 3: return route_launch<T, V, 3>(p, s);
      case 4: return route_launch<T, V, 4>(p, s);
    }
    if constexpr (V == 4) {
      switch (cdiv(p.E, 32 * V)) {
        case 5: return route_launch<T, V, 5>(p, s);
        case 6: return route_launch<T, V, 6>(p, s);
        case 7: return route_launch<T, V, 7>(p, s);
        default: return route_launch<T, V, 8>(p, s);
      }
    }
  }
  if (p.E <= 128) return route_launch<T, 1, 4>(p, s);
  if (p.E <= 256) return route_launch<T, 1, 8>(p, s);
  if (p.E <= 512) return route_launch<T, 1, 16>(p, s);
  return route_launch<T, 1, 32>(p, s);
}

// ------------------------------------------------------------------------------ norms
constexpr int kNormMaxH = 16384;

bool norm_ok(const moe_norm_desc* d) {
  return d != nullptr && d->T >= 0 && d->T <= 0x7fffffffLL && d->H >= 1 &&
         (d->kind == MOE_NORM_LAYER || d->kind == MOE_NORM_RMS) && std::isfinite(d->eps) && d->eps >= 0.f &&
         op_type_ok(d->dtype);
}

// Whether rows of H elements are whole 16-byte vectors.
bool norm_vec(const moe_norm_desc& d) { return d.H % (16 / op_type_bytes(d.dtype)) == 0; }

template <typename T, int VL>
void norm_dispatch(const NormParams& p, cudaStream_t s) {
  const int nvec = p.H / VL;
  if (nvec <= 128) {
    const unsigned blocks = static_cast<unsigned>(cdiv(p.T, NORM_WARP_ROWS));
    const int threads = 32 * NORM_WARP_ROWS;
    if (nvec <= 32)
      norm_kernel<T, VL, 1, true><<<blocks, threads, 0, s>>>(p);
    else if (nvec <= 64)
      norm_kernel<T, VL, 2, true><<<blocks, threads, 0, s>>>(p);
    else
      norm_kernel<T, VL, 4, true><<<blocks, threads, 0, s>>>(p);
    return;
  }
  const unsigned blocks = static_cast<unsigned>(p.T);
  auto threads = [&](int nv) { return static_cast<int>(cdiv(cdiv(nvec, nv), 32) * 32); };
  if (nvec <= 1024)
    norm_kernel<T, VL, 4, false><<<blocks, threads(4), 0, s>>>(p);
  else if (nvec <= 8192)
    norm_kernel<T, VL, 8, false><<<blocks, threads(8), 0, s>>>(p);
  else if constexpr (VL == 1)
    norm_kernel<T, VL, 16, false><<<blocks, threads(16), 0, s>>>(p);
}

// Blocks of the backward pass: what the parts in the workspace are laid out for.
int norm_bwd_blocks(const moe_norm_desc& d) {
  const int vl = norm_vec(d) ? 16 / op_type_bytes(d.dtype) : 1;
  const long long groups = d.H / vl <= 128 ? 8 : 1;
  return static_cast<int>(std::max<long long>(1, std::min<long long>(cdiv(d.T, groups), 2LL * num_sms())));
}

template <typename T, int VL>
void norm_bwd_dispatch(const NormBwdParams& p, int blocks, cudaStream_t s) {
  const int nvec = p.H / VL;
  if (nvec <= 128) {
    const size_t smem = static_cast<size_t>(p.H) * 8;
    if (nvec <= 32)
      norm_backward_kernel<T, VL, 1, true><<<blocks, 256, smem, s>>>(p);
    else if (nvec <= 64)
      norm_backward_kernel<T, VL, 2, true><<<blocks, 256, smem, s>>>(p);
    else
      norm_backward_kernel<T, VL, 4, true><<<blocks, 256, smem, s>>>(p);
    return;
  }
  auto threads = [&](int nv) { return static_cast<int>(cdiv(cdiv(nvec, nv), 32) * 32); };
  if (nvec <= 1024)
    norm_backward_kernel<T, VL, 1, false><<<blocks, threads(1), 0, s>>>(p);
  else if (nvec <= 2048)
    norm_backward_kernel<T, VL, 2, false><<<blocks, threads(2), 0, s>>>(p);
  else if constexpr (VL <= 4) {
    if (nvec <= 4096)
      norm_backward_kernel<T, VL, 4, false><<<blocks, threads(4), 0, s>>>(p);
    else if constexpr (VL == 1)
      norm_backward_kernel<T, VL, 16, false><<<blocks, threads(16), 0, s>>>(p);
  }
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

// Launches over the list and blocks of each.
int clip_launches(int32_t count) { return std::max(1, static_cast<int>(cdiv(count, CLIP_MAX))); }
int clip_blocks() { return 4 * num_sms(); }

// Elements of a chunk: about eight chunks a block over the whole list, so that
// the blocks' shares are even, and at least 4096, so that a chunk's start-up is
// small beside it.
int clip_chunk(const moe_grad_tensor* list, int32_t count) {
  long long total = 0;
  for (int i = 0; i < count; ++i) total += list[i].n;
  long long c = total / (8LL * clip_blocks());
  c = std::max<long long>(4096, std::min<long long>(c, 65536));
  return static_cast<int>(c / 64 * 64);
}

template <int MAXT>
moe_status clip_run(const moe_grad_tensor* list, int32_t count, bool max_norm_kind, float max_norm, float* norm_out,
                    double* partial, cudaStream_t s) {
  const int nl = clip_launches(count), blocks = clip_blocks();
  const int chunk = clip_chunk(list, count);
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
        chunks += cdiv(t.n, chunk);
      }
      if (chunks > 0x3fffffffLL) return MOE_ERR_UNSUPPORTED;
      l.chunks = static_cast<int>(chunks);
      if (pass == 0) {
        if (max_norm_kind)
          clip_norm_kernel<MAXT, true><<<blocks, CLIP_THREADS, 0, s>>>(l, partial + li * blocks);
        else
          clip_norm_kernel<MAXT, false><<<blocks, CLIP_THREADS, 0, s>>>(l, partial + li * blocks);
      } else {
        float* out = li == 0 ? norm_out : nullptr;
        const int grid = std::max(1, std::min(blocks, l.chunks));
        if (max_norm_kind)
          clip_scale_kernel<MAXT, true><<<grid, CLIP_THREADS, 0, s>>>(l, partial, nl * blocks, max_norm, out);
        else
          clip_scale_kernel<MAXT, false><<<grid, CLIP_THREADS, 0, s>>>(l, partial, nl * blocks, max_norm, out);
      }
      ++g_last_launches;
      if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
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
  with_type(d->dtype, [&](auto v) { route_dispatch<decltype(v)>(p, reinterpret_cast<cudaStream_t>(stream)); });
  g_last_launches = 1;
  return launched();
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
  with_type(d->dtype, [&](auto v) {
    using T = decltype(v);
    if (d->E % kVec<T> == 0)
      route_backward_kernel<T, kVec<T>><<<blocks, ROUTE_WARPS * 32, 0, s>>>(p, idx, dw, static_cast<T*>(dlogits));
    else
      route_backward_kernel<T, 1><<<blocks, ROUTE_WARPS * 32, 0, s>>>(p, idx, dw, static_cast<T*>(dlogits));
  });
  g_last_launches = 1;
  return launched();
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
  const NormParams p{x, gamma, beta, y, mean, rstd, d->T, d->H, d->eps, 1.0f / d->H, d->kind == MOE_NORM_RMS};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  with_type(d->dtype, [&](auto v) {
    using T = decltype(v);
    if (norm_vec(*d))
      norm_dispatch<T, kVec<T>>(p, s);
    else
      norm_dispatch<T, 1>(p, s);
  });
  g_last_launches = 1;
  return launched();
}

size_t moe_norm_backward_workspace_size(const moe_norm_desc* d) {
  using namespace moe;
  if (!norm_ok(d) || d->H > kNormMaxH) return 0;
  return round_up(static_cast<size_t>(norm_bwd_blocks(*d)) * 2 * d->H * 4, kAlign);
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
  const int blocks = norm_bwd_blocks(*d);
  float* part = static_cast<float*>(ws);
  if (d->T > 0) {
    const NormBwdParams p{dy, x, gamma, mean, rstd, dx, part, d->T, d->H, 1.0f / d->H};
    with_type(d->dtype, [&](auto v) {
      using T = decltype(v);
      if (norm_vec(*d))
        norm_bwd_dispatch<T, kVec<T>>(p, blocks, s);
      else
        norm_bwd_dispatch<T, 1>(p, blocks, s);
    });
    ++g_last_launches;
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (dgamma != nullptr || dbeta != nullptr) {
    column_sum_kernel<<<static_cast<unsigned>(cdiv(2LL * d->H, 32)), dim3(32, 32), 0, s>>>(
        part, d->T > 0 ? blocks : 0, d->H, dgamma, dbeta);
    ++g_last_launches;
  }
  return launched();
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
