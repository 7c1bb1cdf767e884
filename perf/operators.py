"""Measured cases of the operators around the MoE layer: routing from logits (moe_route), layer and RMS norm
(moe_norm), the dense product with an epilogue (moe_linear), each with its gradients, and gradient clipping
(moe_clip_grads).

With `own` false, run() computes an operator in elementary torch operations (fp32, fp64 for the routing keys and the
long sum of squares, one rounding at the end); with `own` true it makes the library's calls.  exact() restates each
definition in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6  # of the norms, and beside the gradients' norm


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a serving step, sigmoid scores limited to the best groups of experts: pure latency
        {"name": "route one token, groups", "op": "route", "T": 1, "E": 256, "k": 8, "groups": 8, "keep": 4,
         "group_top": 2, "score": "sigmoid", "bias": True, "renorm": True, "scale": 2.5, "masked": False, "dtype": "f32"},
        # a 16384-token prompt through the 896-expert router, fp32 logits
        {"name": "route prompt, 896 experts", "op": "route", "T": 16384, "E": 896, "k": 16, "groups": 1, "keep": 1,
         "group_top": 1, "score": "sigmoid", "bias": True, "renorm": True, "scale": 1.0, "masked": False, "dtype": "f32"},
        # a training batch with bf16 logits, softmax scores and no bias; some experts (and some whole rows) masked
        {"name": "route softmax batch, masked", "op": "route", "T": 32767, "E": 128, "k": 8, "groups": 1, "keep": 1,
         "group_top": 1, "score": "softmax", "bias": False, "renorm": True, "scale": 1.0, "masked": True, "dtype": "bf16"},
        # the router's gradient in training where the weights are plain softmax scores: every logit gets one
        {"name": "route gradients, softmax", "op": "route_bwd", "T": 16384, "E": 896, "k": 16, "score": "softmax",
         "renorm": False, "scale": 1.0, "masked": False, "dtype": "bf16"},
        # the pre-norm of a 256-sequence decode step
        {"name": "norm decode step", "op": "norm", "kind": "layer", "T": 256, "H": 7168, "stats": False, "dtype": "bf16"},
        # RMS norm of a ragged prompt with an odd row length
        {"name": "norm prompt, odd rows", "op": "norm", "kind": "rms", "T": 4097, "H": 5001, "stats": True, "dtype": "f16"},
        # the pre-norm's gradients over a 16384-token training batch
        {"name": "norm gradients", "op": "norm_bwd", "kind": "layer", "T": 16384, "H": 7168, "dtype": "bf16"},
        # a 4-sequence decode step through a dense projection: the weights' bytes count
        {"name": "linear 4 tokens", "op": "linear", "M": 4, "N": 7168, "K": 3584, "act": "silu", "bias": True,
         "residual": True, "dtype": "bf16"},
        # a prompt through the same projection
        {"name": "linear prompt", "op": "linear", "M": 8192, "N": 7168, "K": 3584, "act": "gelu", "bias": True,
         "residual": True, "dtype": "bf16"},
        # its gradients in training, ragged rows
        {"name": "linear gradients", "op": "linear_bwd", "M": 4001, "N": 3584, "K": 7168, "act": "silu", "bias": True,
         "dtype": "bf16"},
        # the gradients of a small model's buckets: views at odd offsets of one flat bf16 buffer
        {"name": "clip small buckets", "op": "clip", "tensors": 40, "elements": 3000001, "max_norm": 1.0, "dtype": "bf16"},
        # the fp32 gradients of a 128-expert layer (expert weights and the dense ones)
        {"name": "clip a layer's gradients", "op": "clip", "tensors": 393, "elements": 322000003, "max_norm": 1.0,
         "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "norm", "norm_bwd", "linear", "linear_bwd", "clip"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        size = max(2, _log_int(rng, 8, 1024) // groups)
        E = groups * size
        T = min(_log_int(rng, 1, 32768), 16384 * 896 // E)
        k = rng.randint(1, min(32, E))
        c = {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["sigmoid", "softmax"]),
             "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.3,
             "dtype": rng.choice(["f32", "bf16", "f16"])}
        if op == "route":
            c.update(groups=groups, keep=rng.randint(-(-k // size), groups), group_top=rng.choice([1, 2]),
                     bias=rng.random() < 0.6)
        return c
    if op in ("norm", "norm_bwd"):
        H = _log_int(rng, 32, 16384)
        T = min(_log_int(rng, 1, 16384), 16384 * 7168 // H)
        c = {"op": op, "kind": rng.choice(["layer", "rms"]), "T": T, "H": H, "dtype": rng.choice(["f32", "bf16", "f16"])}
        if op == "norm":
            c["stats"] = rng.random() < 0.5
        elif c["dtype"] == "f32":
            c["T"] = max(1, T // 2)
        return c
    if op in ("linear", "linear_bwd"):
        M = _log_int(rng, 1, 8192)
        N, K = (8 * _log_int(rng, 8, 1024) for _ in range(2))
        most = 8192 * 7168 * 3584 if op == "linear" else 4001 * 7168 * 3584
        c = {"op": op, "M": max(1, min(M, most // (N * K))), "N": N, "K": K,
             "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.7,
             "dtype": rng.choice(["bf16", "f16"])}
        if op == "linear":
            c["residual"] = rng.random() < 0.5
        return c
    dtype = rng.choice(["f32", "bf16", "f16"])
    return {"op": "clip", "tensors": _log_int(rng, 1, 400), "elements": _log_int(rng, 1000, 300000000),
            "max_norm": rng.choice([0.1, 1.0, 10.0]), "dtype": dtype}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def _lengths(case):
    """Ragged tensor lengths that add up to the case's elements: log-uniform shares, some of them nothing."""
    r = random.Random(case["tensors"] * 7919 + case["elements"])
    share = [math.exp(r.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    total = sum(share)
    lens = [int(case["elements"] * s / total) for s in share]
    if len(lens) > 8:
        lens[3] = 0
    lens[-1] += case["elements"] - sum(lens)
    return lens


def _logits(case, g):
    logits = _randn(g, (case["T"], case["E"]), torch.float32, 1.5)
    if case["masked"]:
        gone = torch.rand((case["T"], case["E"]), generator=g, device=DEV) < 0.1
        gone[96::97] = True  # rows with nothing left
        logits.masked_fill_(gone, -math.inf)
    return logits.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], {"case": case}
    dt = DTYPES[case["dtype"]]
    if op == "route":
        s["logits"] = _logits(case, g)
        s["bias"] = _randn(g, (case["E"],), torch.float32, 0.05) if case["bias"] else None
        s["idx"] = torch.empty(case["T"], case["k"], dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(case["T"], case["k"], dtype=torch.float32, device=DEV)
    elif op == "route_bwd":
        s["logits"] = _logits(case, g)
        # the forward pass's selection (any k distinct experts are valid here)
        s["idx"] = torch.topk(s["logits"].float(), case["k"], dim=1).indices.to(torch.int32)
        s["dw"] = _randn(g, (case["T"], case["k"]), torch.float32)
        s["dlogits"] = torch.empty_like(s["logits"])
    elif op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        s["x"] = torch.randn((T, H), generator=g, device=DEV).mul_(1.3).add_(0.2).to(dt)
        s["gamma"] = 1.0 + _randn(g, (H,), torch.float32, 0.1)
        s["beta"] = _randn(g, (H,), torch.float32, 0.1) if case["kind"] == "layer" else None
        s["mean"] = torch.empty(T, dtype=torch.float32, device=DEV)
        s["rstd"] = torch.empty(T, dtype=torch.float32, device=DEV)
        if op == "norm":
            s["y"] = torch.empty_like(s["x"])
        else:
            # the statistics that the forward pass kept
            x = s["x"].double()
            mu = x.mean(1) if case["kind"] == "layer" else torch.zeros(T, dtype=torch.float64, device=DEV)
            s["mean"].copy_(mu)
            s["rstd"].copy_(((x - mu[:, None]).square().mean(1) + EPS).rsqrt())
            s["dy"] = _randn(g, (T, H), dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(H, dtype=torch.float32, device=DEV)
            s["dbeta"] = torch.empty(H, dtype=torch.float32, device=DEV) if case["kind"] == "layer" else None
    elif op in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _randn(g, (M, K), dt)
        s["weight"] = _randn(g, (N, K), dt, K ** -0.5)
        if op == "linear":
            s["bias"] = _randn(g, (N,), torch.float32, 0.1) if case["bias"] else None
            s["residual"] = _randn(g, (M, N), dt) if case["residual"] else None
            s["y"] = torch.empty(M, N, dtype=dt, device=DEV)
        else:
            s["pre"] = _randn(g, (M, N), dt)
            s["dy"] = _randn(g, (M, N), dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty_like(s["weight"])
            s["dbias"] = torch.empty(N, dtype=torch.float32, device=DEV) if case["bias"] else None
    else:
        s["flat"], lens = _flat(case, g)
        s["out_flat"] = torch.empty_like(s["flat"])
        s["grads"], s["out"] = s["flat"].split(lens), s["out_flat"].split(lens)
        s["norm"] = torch.empty(1, dtype=torch.float32, device=DEV)
    return s


def _flat(case, g):
    lens = _lengths(case)
    flat = torch.empty(case["elements"], dtype=DTYPES[case["dtype"]], device=DEV)
    for part, std in zip(flat.split(lens), torch.rand(len(lens), generator=g, device=DEV).mul_(4.0).sub_(6.0).exp_().tolist()):
        part.normal_(0.0, std, generator=g)
    return flat, lens


# ------------------------------------------------------------------------------------------------ run
def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# plain forms
def _plain_route(s):
    c, logits, bias = s["case"], s["logits"], s["bias"]
    T, E, G = c["T"], c["E"], c["groups"]
    l64 = logits.double()
    gone = (l64 == -math.inf) | l64.isnan()
    l64 = l64.masked_fill(gone, -math.inf)
    score = _scores(l64, c["score"])
    key = score if bias is None else score + bias.double()
    order = l64 if bias is None else key.masked_fill(gone, -math.inf)
    if G > 1:
        best = key.masked_fill(gone, -math.inf).view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        rank = best.masked_fill(best == -math.inf, 0.0).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        kept = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        out = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, False)
        # masked experts of kept groups still come before those of other groups
        order = order.clamp_min(-1e300).masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    idx = order.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, idx).float()
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return idx.to(torch.int32), w * c["scale"]


def _scores(logits, kind):
    if kind == "sigmoid":
        return torch.sigmoid(logits)
    top = logits.max(1, keepdim=True).values
    e = torch.where(logits == -math.inf, torch.zeros_like(logits), torch.exp(logits - top))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _plain_route_bwd(s):
    c, idx, dw = s["case"], s["idx"].long(), s["dw"]
    score = _scores(s["logits"].float(), c["score"])
    chosen = score.gather(1, idx)
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        p = torch.where(total > 0, chosen / total, torch.zeros_like(chosen))
        inner = dw - (p * dw).sum(1, keepdim=True)
        if c["score"] == "sigmoid":
            d = p * inner * (1.0 - chosen)
        else:
            d = p * inner
        dl = torch.zeros_like(score).scatter_(1, idx, d * c["scale"])
    else:
        ds = torch.zeros_like(score).scatter_(1, idx, dw * c["scale"])
        if c["score"] == "sigmoid":
            dl = ds * score * (1.0 - score)
        else:
            dl = score * (ds - (score * ds).sum(1, keepdim=True))
    return dl.to(s["logits"].dtype)


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    if c["kind"] == "layer":
        mean = x.mean(1, keepdim=True)
        x = x - mean
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    y = y.to(s["x"].dtype)
    if not c["stats"]:
        return y
    return (y, mean[:, 0], rstd[:, 0]) if c["kind"] == "layer" else (y, rstd[:, 0])


def _plain_norm_bwd(s):
    layer = s["case"]["kind"] == "layer"
    dy, r = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * r if layer else s["x"].float() * r
    g = dy * s["gamma"]
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        dx = dx - g.mean(1, keepdim=True)
    dx = (dx * r).to(s["x"].dtype)
    dgamma = (dy * xh).sum(0)
    return (dx, dgamma, dy.sum(0)) if layer else (dx, dgamma)


def _act(x, kind):
    if kind == "relu":
        return x.clamp_min(0.0)
    if kind == "silu":
        return x * torch.sigmoid(x)
    if kind == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.5 ** 0.5))
    if kind == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))
    return x


def _act_grad(x, kind):
    if kind == "relu":
        return (x > 0).to(x.dtype)
    if kind == "silu":
        sg = torch.sigmoid(x)
        return sg * (1.0 + x * (1.0 - sg))
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (2.0 * math.pi) ** -0.5
    if kind == "gelu_tanh":
        a = (2.0 / math.pi) ** 0.5
        t = torch.tanh(a * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _plain_linear(s):
    y = s["x"].float() @ s["weight"].float().T
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _plain_linear_bwd(s):
    c = s["case"]
    dp = s["dy"].float() * _act_grad(s["pre"].float(), c["act"])
    dx = (dp @ s["weight"].float()).to(s["x"].dtype)
    dweight = (dp.T @ s["x"].float()).to(s["x"].dtype)
    return (dx, dweight, dp.sum(0)) if c["bias"] else (dx, dweight)


def _plain_clip(s):
    x = s["flat"].float()
    norm = x.square().sum(dtype=torch.float64).sqrt().float()
    coef = (s["case"]["max_norm"] / (norm + EPS)).clamp_max(1.0)
    return norm.view(1), (x * coef).to(s["flat"].dtype)


PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
         "linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "clip": _plain_clip}


# the library's calls; descriptors and workspaces are made once per state, as a program keeps them
def _moe():
    import sparse_moe_layer_renormalised_b200 as moe

    return moe


def _workspace(nbytes):
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=DEV)


def _route_desc(s):
    c = s["case"]
    return _moe().route_desc(T=c["T"], E=c["E"], k=c["k"], groups=c.get("groups", 1), keep_groups=c.get("keep", 1),
                             group_top=c.get("group_top", 1), score=c["score"], renorm=c["renorm"], scale=c["scale"],
                             dtype=c["dtype"])


def _own_route(s):
    moe = _moe()
    if "desc" not in s:
        s["desc"] = _route_desc(s)
    moe.check(moe.moe_route(s["desc"], s["logits"], s["bias"], s["idx"], s["w"]))
    return s["idx"], s["w"]


def _own_route_bwd(s):
    moe = _moe()
    if "desc" not in s:
        s["desc"] = _route_desc(s)
    moe.check(moe.moe_route_backward(s["desc"], s["logits"], s["idx"], s["dw"], s["dlogits"]))
    return s["dlogits"]


def _norm_desc(s):
    c = s["case"]
    return _moe().norm_desc(T=c["T"], H=c["H"], kind=c["kind"], eps=EPS, dtype=c["dtype"])


def _own_norm(s):
    moe, c = _moe(), s["case"]
    if "desc" not in s:
        s["desc"] = _norm_desc(s)
    layer = c["kind"] == "layer"
    mean, rstd = (s["mean"] if layer else None, s["rstd"]) if c["stats"] else (None, None)
    moe.check(moe.moe_norm(s["desc"], s["x"], s["gamma"], s["beta"], s["y"], mean, rstd))
    if not c["stats"]:
        return s["y"]
    return (s["y"], mean, rstd) if layer else (s["y"], rstd)


def _own_norm_bwd(s):
    moe = _moe()
    if "desc" not in s:
        s["desc"] = _norm_desc(s)
        s["ws"] = _workspace(moe.moe_norm_backward_workspace_size(s["desc"]))
    layer = s["case"]["kind"] == "layer"
    moe.check(moe.moe_norm_backward(s["desc"], s["dy"], s["x"], s["gamma"], s["mean"] if layer else None, s["rstd"],
                                    s["dx"], s["dgamma"], s["dbeta"], s["ws"]))
    return (s["dx"], s["dgamma"], s["dbeta"]) if layer else (s["dx"], s["dgamma"])


def _linear_desc(s):
    c = s["case"]
    return _moe().linear_desc(M=c["M"], N=c["N"], K=c["K"], act=c["act"], dtype=c["dtype"])


def _own_linear(s):
    moe = _moe()
    if "desc" not in s:
        s["desc"] = _linear_desc(s)
        s["ws"] = _workspace(moe.moe_linear_workspace_size(s["desc"]))
    moe.check(moe.moe_linear(s["desc"], s["x"], s["weight"], s["bias"], s["residual"], None, s["y"], s["ws"]))
    return s["y"]


def _own_linear_bwd(s):
    moe = _moe()
    if "desc" not in s:
        s["desc"] = _linear_desc(s)
        s["ws"] = _workspace(moe.moe_linear_backward_workspace_size(s["desc"]))
    moe.check(moe.moe_linear_backward(s["desc"], s["dy"], s["pre"], s["x"], s["weight"], s["dx"], s["dweight"],
                                      s["dbias"], s["ws"]))
    return (s["dx"], s["dweight"], s["dbias"]) if s["case"]["bias"] else (s["dx"], s["dweight"])


def _own_clip(s):
    moe = _moe()
    if "list" not in s:
        s["list"] = moe.tensor_list(s["grads"], s["out"])
        s["ws"] = _workspace(moe.moe_clip_grads_workspace_size(s["list"]))
    moe.check(moe.moe_clip_grads(s["list"], "l2", s["case"]["max_norm"], s["norm"], s["ws"]))
    return s["norm"], s["out_flat"]


OWN = {"route": _own_route, "route_bwd": _own_route_bwd, "norm": _own_norm, "norm_bwd": _own_norm_bwd,
       "linear": _own_linear, "linear_bwd": _own_linear_bwd, "clip": _own_clip}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * e + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    if op == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["score"] == "softmax" and not case["renorm"]  # every logit counts, else the chosen ones
        return {"bytes": T * E * e * (2 if dense else 1) + T * k * (8 if dense else 8 + e), "flops": T * (8 * E if dense else 12 * k)}
    if op == "norm":
        T, H = case["T"], case["H"]
        return {"bytes": 2 * T * H * e + 8 * H + (8 * T if case["stats"] else 0), "flops": 8 * T * H}
    if op == "norm_bwd":
        T, H = case["T"], case["H"]
        return {"bytes": 3 * T * H * e + 12 * H + 8 * T, "flops": 16 * T * H}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M * K + N * K + M * N * (2 if case["residual"] else 1)) * e + 4 * N, "flops": 2 * M * N * K}
    if op == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (2 * M * N + 2 * M * K + 2 * N * K) * e + 4 * N, "flops": 4 * M * N * K}
    return {"bytes": 2 * case["elements"] * e, "flops": 3 * case["elements"]}


# ------------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))


def _exact_scores(logits, kind):
    l = logits.double()
    l = torch.where(l.isnan(), torch.full_like(l, -math.inf), l)
    if kind == "sigmoid":
        return l, 1.0 / (1.0 + torch.exp(-l))
    lse = torch.logsumexp(l, 1, keepdim=True)
    return l, torch.where(l > -math.inf, torch.exp(l - torch.where(lse > -math.inf, lse, 0.0)), torch.zeros_like(l))


def _ranks(key):
    """How many come before each value of its row: the larger ones, and the equal ones at a lower place."""
    n = key.shape[1]
    lower = torch.ones(n, n, dtype=torch.bool, device=DEV).tril(-1)  # [i, j]: j < i
    rows = max(1, (1 << 28) // (n * n))
    parts = [((p[:, None, :] > p[:, :, None]) | ((p[:, None, :] == p[:, :, None]) & lower)).sum(2) for p in key.split(rows)]
    return torch.cat(parts)


def _exact_route(c, s):
    l, score = _exact_scores(s["logits"], c["score"])
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    gone = l == -math.inf
    b = torch.zeros(E, dtype=torch.float64, device=DEV) if s["bias"] is None else s["bias"].double()
    low = torch.finfo(torch.float64).min
    key = torch.where(gone, torch.full_like(l, low), l if s["bias"] is None else score + b)
    if G > 1:
        part = torch.where(gone, torch.full_like(l, -math.inf), score + b).view(T, G, -1)
        top = part.topk(min(c["group_top"], E // G), dim=2).values
        rank = torch.where(top > -math.inf, top, 0.0).sum(2)
        rank = torch.where((part > -math.inf).any(2), rank, torch.full_like(rank, -math.inf))
        kept = _ranks(rank) < c["keep"]
        key = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), key, torch.full_like(key, -math.inf))
    place = _ranks(key)
    at = torch.arange(E, device=DEV).expand(T, E)
    idx = torch.zeros(T, k + 1, dtype=torch.int64, device=DEV).scatter_(1, place.clamp_max(k), at)[:, :k]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
    return idx.to(torch.int32), c["scale"] * w


def _exact_route_bwd(c, s):
    """By automatic differentiation of the weights with the selection held fixed."""
    l = s["logits"].double()
    fine = (l > -math.inf)
    z = torch.where(fine, l, torch.zeros_like(l)).requires_grad_(True)
    with torch.enable_grad():
        if c["score"] == "sigmoid":
            score = torch.where(fine, torch.sigmoid(z), torch.zeros_like(z))
        else:
            some = fine.any(1, keepdim=True)
            score = torch.where(fine, torch.softmax(torch.where(fine | ~some, z, torch.full_like(z, -math.inf)), 1), torch.zeros_like(z))
        w = score.gather(1, s["idx"].long())
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total > 0, total, torch.ones_like(total))
        loss = (c["scale"] * w * s["dw"].double()).sum()
        return torch.autograd.grad(loss, z)[0]


def _exact_norm(c, s):
    x = s["x"].double()
    mu = x.mean(1) if c["kind"] == "layer" else torch.zeros(c["T"], dtype=torch.float64, device=DEV)
    rstd = 1.0 / torch.sqrt((x - mu[:, None]).pow(2).sum(1) / c["H"] + EPS)
    y = (x - mu[:, None]) * rstd[:, None] * s["gamma"].double()
    y = y if s["beta"] is None else y + s["beta"].double()
    if not c["stats"]:
        return y
    return (y, mu, rstd) if c["kind"] == "layer" else (y, rstd)


def _exact_norm_bwd(c, s):
    """From the saved statistics, term by term of the definition's derivative."""
    layer = c["kind"] == "layer"
    x, dy, r, H = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None], c["H"]
    u = (x - s["mean"].double()[:, None]) * r if layer else x * r
    g = dy * s["gamma"].double()
    along = torch.einsum("th,th->t", g, u)[:, None] / H
    dx = r * (g - u * along - (g.sum(1, keepdim=True) / H if layer else 0.0))
    dgamma = torch.einsum("th,th->h", dy, u)
    return (dx, dgamma, dy.sum(0)) if layer else (dx, dgamma)


def _exact_act(x, kind):
    if kind == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if kind == "silu":
        return x / (1.0 + torch.exp(-x))
    if kind == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def _exact_linear(c, s):
    pre = torch.mm(s["x"].double(), s["weight"].double().t())
    pre = pre if s["bias"] is None else pre + s["bias"].double()
    y = _exact_act(pre, c["act"])
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_linear_bwd(c, s):
    pre = s["pre"].double().requires_grad_(True)
    with torch.enable_grad():
        dp, = torch.autograd.grad((_exact_act(pre, c["act"]) * s["dy"].double()).sum(), pre)
    dx, dweight = torch.mm(dp, s["weight"].double()), torch.mm(dp.t(), s["x"].double())
    return (dx, dweight, dp.sum(0)) if c["bias"] else (dx, dweight)


def _exact_clip(c, s):
    norm = torch.linalg.vector_norm(s["flat"].double())
    return norm.view(1), s["flat"].double() * torch.clamp(c["max_norm"] / (norm + EPS), max=1.0)


EXACT = {"route": _exact_route, "route_bwd": _exact_route_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd,
         "linear": _exact_linear, "linear_bwd": _exact_linear_bwd, "clip": _exact_clip}
