"""The operators as they are used together: a block's pre-norm, router product,
routing and the layer's own dispatch, experts, combine and output, forward; the
router's gradients back through routing, product and norm, and clipping.  Then the
same under a captured graph, and on two streams at once."""
import pytest
import torch

import gen
import oracle
import sparse_moe_layer_renormalised_b200 as moe
from harness import dims_for, parity
from ops_util import HALF, within, workspace
from oracle import inputs as oin
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
F64 = torch.float64


class Block:
    """Buffers and calls of one step at the "mid" layer's shape."""

    def __init__(self, T, seed=0):
        self.cfg = cfg = gen.CONFIGS["mid"].with_(T=T, k=8)
        self.T, dev = T, "cuda"
        w = gen.device_layer(cfg, dev)
        self.x = w.pop("x")
        self.w = w
        self.layer = moe.MoeLayer(dims_for(cfg), w)
        E, H, L, k = cfg.E, cfg.H, cfg.L, cfg.k
        g = torch.Generator(device=dev).manual_seed(seed)
        self.gamma = 1.0 + 0.1 * torch.randn(H, generator=g, device=dev)
        new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        bf = torch.bfloat16
        self.nd = moe.norm_desc(T, H, "rms")
        self.ld = moe.linear_desc(T, E, H, "none", "bf16", "f32")
        self.rd = moe.route_desc(T, E, k, groups=8, keep_groups=4, group_top=2, scale=1.5)
        self.xn, self.rstd, self.logits = new(T, H, dt=bf), new(T), new(T, E)
        self.idx, self.p = new(T, k, dt=torch.int32), new(T, k)
        self.z, self.h_s = new(T, L, dt=bf), new(T, cfg.S * cfg.Is, dt=bf)
        self.offsets, self.perm, self.inv = new(E + 1, dt=torch.int32), new(T * k, dt=torch.int32), new(T * k, dt=torch.int32)
        self.z_perm, self.y_perm = new(T * k, L, dt=bf), new(T * k, L)
        self.u, self.n, self.y = new(T, L), new(T, L, dt=bf), new(T, H)
        self.ws = workspace(moe.moe_workspace_size(dims_for(cfg)))
        self.lws = workspace(moe.moe_linear_workspace_size(self.ld))
        # backward
        self.dw = torch.randn(T, k, generator=g, device=dev)
        self.dlogits, self.dl16 = new(T, E), new(T, E, dt=bf)
        self.dxn, self.dWr, self.dx, self.dgamma = new(T, H, dt=bf), new(E, H, dt=bf), new(T, H, dt=bf), new(H)
        self.ld16 = moe.linear_desc(T, E, H, "none")
        self.bws = workspace(moe.moe_linear_backward_workspace_size(self.ld16))
        self.nws = workspace(moe.moe_norm_backward_workspace_size(self.nd))
        self.norm, self.cWr, self.cgamma = new(1), new(E, H, dt=bf), new(H)
        self.grads = moe.tensor_list([self.dWr, self.dgamma], [self.cWr, self.cgamma])
        self.cws = workspace(moe.moe_clip_grads_workspace_size(self.grads))

    def forward(self):
        d, w, c = dims_for(self.cfg), self.layer._w, moe.check
        c(moe.moe_norm(self.nd, self.x, self.gamma, None, self.xn, None, self.rstd))
        c(moe.moe_linear(self.ld, self.xn, self.w["Wr"], None, None, None, self.logits, self.lws))
        c(moe.moe_route(self.rd, self.logits, self.w["bias"], self.idx, self.p))
        c(moe.moe_latent_shared(d, w, self.xn, self.z, self.h_s))
        c(moe.moe_permute(d, self.idx, self.z, self.offsets, self.perm, self.inv, self.z_perm, self.ws))
        c(moe.moe_expert_ffn(d, w, self.z_perm, self.offsets, self.y_perm, self.ws))
        c(moe.moe_combine(d, self.y_perm, self.inv, self.p, self.w["gamma"], self.u, self.n))
        c(moe.moe_output(d, w, self.h_s, self.n, self.y))

    def backward(self):
        c = moe.check
        c(moe.moe_route_backward(self.rd, self.logits, self.idx, self.dw, self.dlogits))
        self.dl16.copy_(self.dlogits)
        c(moe.moe_linear_backward(self.ld16, self.dl16, None, self.xn, self.w["Wr"], self.dxn, self.dWr, None, self.bws))
        c(moe.moe_norm_backward(self.nd, self.dxn, self.x, self.gamma, None, self.rstd, self.dx, self.dgamma, None, self.nws))
        c(moe.moe_clip_grads(self.grads, "l2", 0.5, self.norm, self.cws))

    def outputs(self):
        return {n: getattr(self, n).clone() for n in ("xn", "logits", "idx", "p", "u", "y", "dlogits", "dxn", "dWr", "dx",
                                                      "dgamma", "norm", "cWr", "cgamma")}


def test_step_against_the_oracle():
    b = Block(300)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    assert moe.moe_device_error() == (moe.MOE_OK, 0)
    cfg, cpu = b.cfg, lambda t: t.cpu()  # noqa: E731
    # each step from the device's own inputs of it
    xn, _, rstd = oo.norm(cpu(b.x), cpu(b.gamma), None, 1e-6, "rms")
    within(b.xn, xn, xn.abs() * (HALF["bf16"] + 1e-5) + 1e-6, "pre-norm")
    pre, _ = oo.linear(cpu(b.xn), cpu(b.w["Wr"]), None, None, "none")
    within(b.logits, pre, (cfg.H / 16 + 32) * 2.0 ** -23 * (cpu(b.xn).double().abs() @ cpu(b.w["Wr"]).double().abs().T), "logits")
    idx, p = oo.route(cpu(b.logits), cpu(b.w["bias"]), cfg.k, 8, 4, 2, "sigmoid", True, 1.5)
    assert torch.equal(cpu(b.idx).long(), idx)
    within(b.p, p, p * 1e-5, "weights")
    # the layer with this routing: the combine of the experts' rows, and the output of it
    ref_u = torch.zeros(b.T, cfg.L, dtype=F64)
    inv, y_perm = cpu(b.inv).long().view(b.T, cfg.k), cpu(b.y_perm).double()
    for j in range(cfg.k):
        ref_u += cpu(b.p)[:, j:j + 1].double() * y_perm[inv[:, j]]
    assert parity(b.u, ref_u) <= 1e-5
    # experts from the oracle, for some tokens
    z = cpu(b.z).double()
    for t in (0, 17, 299):
        for j in (0, 7):
            e = int(idx[t, j])
            y = oracle.expert_forward(z[t:t + 1], *oin.expert_weights(cfg, e), cfg.situ_c, oracle.bf16_round)
            got = y_perm[inv[t, j]]
            assert parity(got, y[0]) <= 1e-2
    # backward, step by step
    dl = oo.route_backward(cpu(b.logits), idx, cpu(b.dw), "sigmoid", True, 1.5)
    within(b.dlogits, dl, dl.abs() * 1e-4 + 1e-5, "dlogits")
    _, dxn, dWr, _ = oo.linear_backward(cpu(b.dl16), None, cpu(b.xn), cpu(b.w["Wr"]), "none")
    assert parity(b.dxn, dxn) <= 2e-2 and float((cpu(b.dxn).double() - dxn).norm() / dxn.norm()) <= HALF["bf16"]
    assert float((cpu(b.dWr).double() - dWr).norm() / dWr.norm()) <= HALF["bf16"]
    dx, dgamma, _ = oo.norm_backward(cpu(b.dxn), cpu(b.x), cpu(b.gamma), None, cpu(b.rstd), "rms")
    assert float((cpu(b.dx).double() - dx).norm() / dx.norm()) <= HALF["bf16"]
    assert float((cpu(b.dgamma).double() - dgamma).norm() / dgamma.norm()) <= 1e-5
    norm, (cWr, cgamma) = oo.clip([cpu(b.dWr), cpu(b.dgamma)], 0.5)
    assert abs(float(b.norm) - norm) <= 1e-6 * norm and norm > 0.5
    within(b.cWr.view(-1), cWr, cWr.abs() * (HALF["bf16"] + 1e-6) + 1e-38)
    within(b.cgamma, cgamma, cgamma.abs() * 1e-6 + 1e-38)


def test_router_gradient_of_the_whole_chain():
    """x -> norm -> logits -> weights as one fp64 function with the selection held
    fixed: its gradient along x and W_r against the chain of the operators."""
    b = Block(64)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    x = b.x.cpu().double().requires_grad_(True)
    Wr = b.w["Wr"].cpu().double().requires_grad_(True)
    gamma = b.gamma.cpu().double().requires_grad_(True)
    xn = x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + 1e-6) * gamma
    p = oo.route_weights(xn @ Wr.T, b.idx.cpu().long(), "sigmoid", True, 1.5)
    dx, dWr, dgamma = torch.autograd.grad((p * b.dw.cpu().double()).sum(), (x, Wr, gamma))
    # three bf16 roundings on the way (xn, dlogits, dxn) and one of the result, each of rms HALF / sqrt 3, the
    # norm's and the product's sums on top: within 3 HALF
    for got, want in ((b.dx, dx), (b.dWr, dWr), (b.dgamma, dgamma)):
        rel = float((got.cpu().double() - want).norm() / want.norm())
        assert rel <= 3 * HALF["bf16"], rel


def test_captured_step_replays_on_new_inputs():
    a, b = Block(200), Block(200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.forward()
        a.backward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward()
        a.backward()
    for seed in (3, 4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(a.x.shape, generator=g, device="cuda").bfloat16()
        a.x.copy_(x)
        b.x.copy_(x)
        graph.replay()
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        for n, v in a.outputs().items():
            assert torch.equal(v, getattr(b, n)), n
    assert moe.moe_device_error() == (moe.MOE_OK, 0)


def test_two_streams_at_once():
    ref = Block(256)
    ref.forward()
    ref.backward()
    torch.cuda.synchronize()
    want = ref.outputs()
    blocks, streams = [Block(256), Block(256)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.forward()
                b.backward()
    torch.cuda.synchronize()
    for b in blocks:
        for n, v in b.outputs().items():
            assert torch.equal(v, want[n]), n
    assert moe.moe_device_error() == (moe.MOE_OK, 0)


def test_streams_that_fork_and_join_captured_and_not():
    """A step over two streams that wait for one another several times, as it is and as a captured graph: the
    same bits as on one stream."""
    T, H, E, bf = 700, 1536, 256, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, W, Wr = randn(T, H).to(bf), (randn(H, H) * H ** -0.5).to(bf), (randn(E, H) * H ** -0.5).to(bf)
    nd, ld, lr = moe.norm_desc(T, H, "rms"), moe.linear_desc(T, H, H, "silu"), moe.linear_desc(T, E, H, "none", "bf16", "f32")
    rd = moe.route_desc(T, E, 8, groups=8, keep_groups=4, group_top=2)
    xn, a, b, ca, cb = (torch.empty(T, H, dtype=bf, device="cuda") for _ in range(5))
    logits, idx, w = torch.empty(T, E, device="cuda"), torch.empty(T, 8, dtype=torch.int32, device="cuda"), torch.empty(T, 8, device="cuda")
    norm, grads = torch.empty(1, device="cuda"), moe.tensor_list([a, b], [ca, cb])
    size = max(moe.moe_linear_workspace_size(ld), moe.moe_linear_workspace_size(lr))
    ws1, ws2, cws = workspace(size), workspace(size), workspace(moe.moe_clip_grads_workspace_size(grads))

    def step(side):
        main, c, cur = torch.cuda.current_stream(), moe.check, x
        for _ in range(6):
            c(moe.moe_norm(nd, cur, None, None, xn))
            side.wait_stream(main)
            c(moe.moe_linear(ld, xn, W, None, None, None, a, ws1))
            with torch.cuda.stream(side):
                c(moe.moe_linear(lr, xn, Wr, None, None, None, logits, ws2))
                c(moe.moe_route(rd, logits, None, idx, w))
                c(moe.moe_linear(ld, xn, W, None, xn, None, b, ws2))
            main.wait_stream(side)
            c(moe.moe_clip_grads(grads, "l2", 100.0, norm, cws))
            cur = cb

    results = lambda: [t.clone() for t in (a, b, ca, cb, logits, idx, w, norm)]  # noqa: E731
    step(torch.cuda.current_stream())
    want = results()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.Stream())
    for run in (lambda: step(side), graph.replay):
        for _ in range(4):
            for t in (xn, a, b, ca, cb, logits):
                t.fill_(float("nan"))
            run()
            torch.cuda.synchronize()
            for p, q in zip(results(), want):
                assert torch.equal(p, q)
    assert moe.moe_device_error() == (moe.MOE_OK, 0)


def test_calls_after_one_another_without_waiting():
    """Many calls in a row on one stream, outputs of one the inputs of the next, as
    launches that overlap would break them."""
    H, T = 2048, 96
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = (torch.randn(H, H, generator=torch.Generator().manual_seed(2)) * H ** -0.5).bfloat16().cuda()
    nd, ld = moe.norm_desc(T, H, "rms"), moe.linear_desc(T, H, H, "silu")
    lws = workspace(moe.moe_linear_workspace_size(ld))

    def run(wait):
        a, b = x.clone(), torch.empty_like(x)
        for _ in range(30):
            moe.check(moe.moe_norm(nd, a, None, None, b))
            if wait:
                torch.cuda.synchronize()
            moe.check(moe.moe_linear(ld, b, w, None, a, None, a, lws))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return a
    slow = run(True)
    for _ in range(4):
        assert torch.equal(run(False), slow)
