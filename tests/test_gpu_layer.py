"""The operators around dispatch and combine run together, as an MoE layer uses them: forward and backward against
the same layer in 64 bits, captured and replayed, on other streams, two calls at once, and refused buffers.

The layer: h = x + residual, y = norm(h), each token's experts apply a SwiGLU product and a down product with a bias,
combine weighs and adds them, a dense product that every token sees is added as a residual. Outputs and gradients are
compared in norm: every step rounds to bf16 (2^-9 relative on average, at most 2^-8), there are six in the forward
and eleven in the backward pass, and errors of different rows are independent, so an output is off by under
6 * 2^-8 and a gradient by under 17 * 2^-8 of the largest tensor norm on its way, which the layer keeps near 1."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, F8, Dense, Routed, activate, ids, norm

pytestmark = pytest.mark.gpu
N, T, E, R, H, F = 2, 24, 8, 2, 256, 128
EPS = 1e-5


def randn(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


class Layer:
    """Weights and inputs of one layer on the GPU, with every buffer that its steps need."""

    def __init__(self, seed=0, cap=0):
        g = torch.Generator().manual_seed(seed)
        dev = "cuda"
        self.idx = ids(N, T, E, R, seed)
        self.d = ep.make_desc(N, T, H, E, R, cap_rows=cap)
        self.b = ep.Buffers(self.d)
        self.b.idx.copy_(self.idx)
        self.weights = torch.softmax(torch.randn((N, T, R), generator=g), -1)
        self.x, self.res = randn(g, N, T, H), randn(g, N, T, H)
        self.gamma = (1 + 0.1 * torch.randn(H, generator=g)).to(BF)
        self.up, self.down = randn(g, E, 2 * F, H, scale=H**-0.5), randn(g, E, H, F, scale=F**-0.5)
        self.up_bias, self.down_bias = randn(g, E, 2 * F, scale=0.1), randn(g, E, H, scale=0.1)
        self.dense_w = randn(g, 1, H, H, scale=H**-0.5)
        self.dout = randn(g, N, T, H)
        self.dd = Dense(1, N * T).desc
        cuda = {k: getattr(self, k).to(dev) for k in ("x", "res", "gamma", "up", "down", "up_bias", "down_bias", "dense_w",
                                                      "dout", "weights")}
        self.c = cuda
        self.p_up = ep.make_product(cuda["up"], ep.EP_ACT_SWIGLU, bias=cuda["up_bias"])
        self.p_down = ep.make_product(cuda["down"], bias=cuda["down_bias"])
        self.p_dense = ep.make_product(cuda["dense_w"])
        rows = N * self.b.cap

        def e(*shape, dtype=BF):
            return torch.zeros(shape, dtype=dtype, device=dev)
        self.h, self.y = e(N, T, H), e(N, T, H)
        self.pre, self.mid, self.eout = e(rows, 2 * F), e(rows, F), e(rows, H)
        self.comb, self.out = e(N, T, H), e(N, T, H)
        self.deout, self.dmid, self.dgrouped = e(rows, H), e(rows, F), e(rows, H)
        self.dweights, self.dy, self.dx = e(N, T, R, dtype=torch.float32), e(N, T, H), e(N, T, H)
        self.ddense = e(N, T, H)
        self.dgamma = e(H, dtype=torch.float32)
        self.dup, self.ddown, self.ddense_w = e(E, 2 * F, H), e(E, H, F), e(1, H, H)
        self.dup_b, self.ddown_b = e(E, 2 * F, dtype=torch.float32), e(E, H, dtype=torch.float32)
        self.ws = [torch.zeros(n, dtype=torch.uint8, device=dev) for n in (
            ep.expert_product_grad_bytes(self.d, self.p_up), ep.expert_product_grad_bytes(self.d, self.p_down),
            ep.expert_product_grad_bytes(self.dd, self.p_dense), ep.rms_norm_grad_bytes(N * T, H))]

    def forward(self, stream=None):
        b, c = self.b, self.c
        ep.rms_norm(c["x"], c["gamma"], EPS, residual=c["res"], sum=self.h, y=self.y, stream=stream)
        ep.dispatch(self.d, b.idx, [self.y], b.plan_ws, b.send, b.grouped, b.status, stream=stream)
        ep.expert_product(self.d, self.p_up, b.grouped, b.plan_ws, self.mid, pre=self.pre, stream=stream)
        ep.expert_product(self.d, self.p_down, [self.mid], b.plan_ws, self.eout, stream=stream)
        ep.combine(self.d, self.eout, c["weights"], b.plan_ws, self.comb, stream=stream)
        ep.expert_product(self.dd, self.p_dense, [self.y.view(N * T, H)], None, self.out, residual=self.comb, stream=stream)

    def backward(self, stream=None):
        b, c, ws = self.b, self.c, self.ws
        ep.expert_product_grad(self.dd, self.p_dense, c["dout"], self.y, None, None, ws[2], dx=self.ddense,
                               dw=self.ddense_w, stream=stream)
        ep.combine_grad(self.d, c["dout"], self.eout, c["weights"], b.plan_ws, self.deout, self.dweights, stream=stream)
        ep.expert_product_grad(self.d, self.p_down, self.deout, self.mid, None, b.plan_ws, ws[1], dx=self.dmid,
                               dw=self.ddown, dbias=self.ddown_b, stream=stream)
        ep.expert_product_grad(self.d, self.p_up, self.dmid, b.grouped[0], self.pre, b.plan_ws, ws[0], dx=self.dgrouped,
                               dw=self.dup, dbias=self.dup_b, stream=stream)
        ep.dispatch_grad(self.d, self.dgrouped, b.plan_ws, self.dy, add=self.ddense, stream=stream)
        ep.rms_norm_grad(self.dy, self.h, c["gamma"], EPS, self.dx, self.dgamma, ws[3], dsum=c["dout"], stream=stream)

    def results(self):
        return {k: getattr(self, k) for k in ("h", "y", "out", "dx", "dgamma", "dweights", "dup", "ddown", "dup_b",
                                              "ddown_b", "ddense_w")}

    def reference(self):
        """Out, and gradients of sum(out dout) + sum(h dout), by differentiating the definition in 64 bits."""
        leaf = {k: getattr(self, k).double().requires_grad_() for k in (
            "x", "gamma", "weights", "up", "down", "up_bias", "down_bias", "dense_w")}
        h = leaf["x"] + self.res.double()
        y = norm(h, leaf["gamma"], EPS).view(N * T, H)
        where = Routed(N, T, E, R, self.idx, hidden=H, cap=self.d.cap_rows)
        rows = where.row.view(N * T, R)
        out = y @ leaf["dense_w"][0].T
        for s in range(N * T):
            for k in range(R):
                if rows[s, k] < 0:
                    continue
                e = int(self.idx.view(-1, R)[s, k])
                m = activate(leaf["up"][e] @ y[s] + leaf["up_bias"][e], ep.EP_ACT_SWIGLU)
                add = torch.zeros_like(out)
                add[s] = leaf["weights"].view(-1, R)[s, k] * (leaf["down"][e] @ m + leaf["down_bias"][e])
                out = out + add
        d = self.dout.double()
        ((out.view_as(h) * d).sum() + (h * d).sum()).backward()
        names = dict(dx="x", dgamma="gamma", dweights="weights", dup="up", ddown="down", dup_b="up_bias",
                     ddown_b="down_bias", ddense_w="dense_w")
        want = {k: leaf[v].grad for k, v in names.items()}
        want.update(h=h.detach(), y=y.detach().view_as(h), out=out.detach().view_as(h))
        return want


def near(got, want, most):
    err = (got.double().cpu().view_as(want) - want).norm() / want.norm()
    assert err < most, float(err)


@pytest.mark.parametrize("cap", [0, 40])
def test_layer_against_64_bits(cap):
    note(f"layer {cap}")
    layer = Layer(cap=cap)
    layer.forward()
    layer.backward()
    torch.cuda.synchronize()
    assert int(layer.b.status.item()) == (ep.EP_STATUS_CAPACITY if cap else 0)
    want = layer.reference()
    for name, got in layer.results().items():
        near(got, want[name], (6 if name in ("h", "y", "out") else 17) * 2.0**-8)


def test_layer_captured_and_replayed():
    """A step captured into a graph and replayed between eager steps of another layer: always the eager bytes."""
    note("layer graph")
    layer, other = Layer(1), Layer(2)
    layer.forward()
    layer.backward()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in layer.results().items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.forward()
        layer.backward()
    for rep in range(4):
        for v in layer.results().values():
            v.fill_(rep)
        for w in layer.ws:
            w.fill_(255)
        other.forward()
        other.backward()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, v in layer.results().items():
            assert torch.equal(v, want[k]), (rep, k)


def test_two_layers_at_once_on_two_streams():
    note("layers on two streams")
    layers = [Layer(3), Layer(4)]
    want = []
    for x in layers:
        x.forward()
        x.backward()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in x.results().items()})
    streams = [torch.cuda.Stream() for _ in layers]
    for x in layers:
        for v in x.results().values():
            v.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s in zip(layers, streams):
            x.forward(s)
            x.backward(s)
    torch.cuda.synchronize()
    for x, w in zip(layers, want):
        for k, v in x.results().items():
            assert torch.equal(v, w[k]), k


def test_block_fp8_layer():
    """The norm's planes through the plain dispatch into a product of codes: against the products of the bf16 rows'
    own quantisation, which differs by one rounding of y, and against 64 bits on the codes themselves."""
    note("fp8 layer")
    g = torch.Generator().manual_seed(5)
    n, t, e, r, h, f = 2, 20, 4, 2, 256, 128
    x = randn(g, n, t, h).cuda()
    gamma = torch.ones(h, dtype=BF, device="cuda")
    codes, scales = torch.zeros((n, t, h), dtype=F8, device="cuda"), torch.zeros((n, t, h // 128), device="cuda")
    ep.rms_norm(x, gamma, EPS, codes=codes, scales=scales)
    where = Routed(n, t, e, r, ids(n, t, e, r, 6), hidden=h, payload=ep.EP_PAYLOAD_FP8_B128)
    b = ep.Buffers(where.desc)
    b.idx.copy_(ids(n, t, e, r, 6))
    ep.dispatch(where.desc, b.idx, [codes, scales], b.plan_ws, b.send, b.grouped, b.status)
    w = (torch.randn((e, 2 * f, h), generator=g) * 100).clamp(-448, 448).to(F8)
    ws = (torch.rand((e, 2 * f // 128, h // 128), generator=g) + 0.5) / 1600
    p = ep.make_product(w.cuda(), ep.EP_ACT_SWIGLU, w_scale=ws.cuda())
    out = torch.zeros((n * b.cap, f), dtype=BF, device="cuda")
    ep.expert_product(where.desc, p, b.grouped, b.plan_ws, out)
    torch.cuda.synchronize()
    rows = (codes.cpu().double().view(n * t, -1, 128) * scales.cpu().double().view(n * t, -1, 1)).view(n * t, h)
    w64 = w.double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    token = torch.arange(n * t * r) // r
    for j, (a, m) in enumerate(where.groups):
        slots = [int((where.row == a + i).nonzero()) for i in range(m)]
        want = activate(rows[token[slots]] @ w64[j].T, ep.EP_ACT_SWIGLU)
        near(out[a:a + m], want, 2.0**-8)


def test_refused_buffers():
    """Buffers that overlap, lie on the host, are misaligned or too small are refused before anything runs."""
    note("refused buffers")
    x = torch.randn(8, 256, device="cuda").to(BF)
    w = torch.ones(256, dtype=BF, device="cuda")
    y = torch.empty_like(x)
    big = torch.zeros(16, 256, dtype=BF, device="cuda")

    def refused(f, *a, **kw):
        with pytest.raises((ep.EPError, ValueError)):
            f(*a, **kw)
    refused(ep.rms_norm, x, w, 1e-6, y=x)
    refused(ep.rms_norm, big[:8], w, 1e-6, y=big[4:12])
    refused(ep.rms_norm, x, w, 1e-6, residual=y, sum=x, y=big[:8])
    refused(ep.rms_norm, x, w, 1e-6, residual=big[:8], sum=big[:8], y=big[1:9])
    refused(ep.rms_norm, x.cpu(), w, 1e-6, y=y)
    refused(ep.rms_norm, x, w.cpu(), 1e-6, y=y)
    flat = torch.zeros(8 * 256 + 4, dtype=BF, device="cuda")
    refused(ep.rms_norm, x, w, 1e-6, y=flat[4:].view(8, 256))               # 8 bytes off
    refused(ep.rms_norm_grad, x, x, w, 1e-6, x)
    refused(ep.rms_norm_grad, x, y, w, 1e-6, big[:8], torch.empty(256, device="cuda"), None)
    where = Routed(1, 8, 2, 2, ids(1, 8, 2, 2, 0), hidden=64)
    rows = where.rows
    p = ep.make_product(torch.zeros(2, 64, 64, dtype=BF, device="cuda"))
    a, o = torch.zeros(rows, 64, dtype=BF, device="cuda"), torch.zeros(rows, 64, dtype=BF, device="cuda")
    refused(ep.expert_product, where.desc, p, [a], where.plan, a)
    refused(ep.expert_product, where.desc, p, [a], where.plan, o, pre=o)
    refused(ep.expert_product, where.desc, p, [a], where.plan, o, residual=o)
    refused(ep.expert_product, where.desc, p, [a], None, o)                 # two experts on one rank, no plan
    refused(ep.expert_product, where.desc, p, [a.cpu()], where.plan, o)
    ws = torch.zeros(ep.expert_product_grad_bytes(where.desc, p), dtype=torch.uint8, device="cuda")
    refused(ep.expert_product_grad, where.desc, p, o, a, None, where.plan, ws, dx=o)
    refused(ep.expert_product_grad, where.desc, p, o, a, a, where.plan, ws, dx=torch.empty_like(a))
    refused(ep.expert_product_grad, where.desc, p, o, None, None, where.plan, ws, dw=torch.zeros_like(p.tensors[0]))
    d64 = torch.zeros(1, 8, 64, dtype=BF, device="cuda")
    wt = torch.zeros(1, 8, 2, device="cuda")
    refused(ep.combine_grad, where.desc, d64, a, wt, where.plan)
    refused(ep.combine_grad, where.desc, d64, a, wt, where.plan, dy=a, dweights=wt.clone())
    refused(ep.combine_grad, where.desc, d64, None, wt, where.plan, dweights=wt.clone())
    refused(ep.dispatch_grad, where.desc, a, where.plan, None)
    ep.expert_product_grad(where.desc, p, o, None, None, where.plan, ws, dx=torch.empty_like(a))   # x not needed
    torch.cuda.synchronize()


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
def test_no_tokens(act):
    """No tokens and no capacity: every operator returns, sums over nothing are zero."""
    note(f"no tokens {act}")
    dev = "cuda"
    where = Routed(2, 0, 4, 2, torch.zeros(2, 0, 2, dtype=torch.int32), hidden=64)
    assert where.rows == 0
    none = torch.empty(0, 64, dtype=BF, device=dev)
    w = torch.ones(64, dtype=BF, device=dev)
    dweight = torch.full((64,), 7.0, device=dev)
    ep.rms_norm(none, w, EPS, y=none)
    ep.rms_norm_grad(none, none, w, EPS, none, dweight, torch.empty(0, dtype=torch.uint8, device=dev))
    wrows = 80 if act == ep.EP_ACT_SWIGLU else 40
    m = torch.ones(4, wrows, 64, dtype=BF, device=dev)
    p = ep.make_product(m, act)
    out = torch.empty(0, 40, dtype=BF, device=dev)
    pre = None if act == ep.EP_ACT_NONE else torch.empty(0, wrows, dtype=BF, device=dev)
    ep.expert_product(where.desc, p, [none], where.plan, out, pre=pre)
    ws = torch.empty(ep.expert_product_grad_bytes(where.desc, p), dtype=torch.uint8, device=dev)
    dw, dbias = torch.full_like(m, 7.0), torch.full((4, wrows), 7.0, device=dev)
    ep.expert_product_grad(where.desc, p, out, none, pre, where.plan, ws, none, dw, dbias)
    ep.expert_product_grad(where.desc, p, out, none, pre, where.plan, ws, dx=none)
    d, wt = torch.empty(2, 0, 64, dtype=BF, device=dev), torch.empty(2, 0, 2, device=dev)
    ep.combine_grad(where.desc, d, none, wt, where.plan, none, wt.clone())
    ep.dispatch_grad(where.desc, none, where.plan, d)
    torch.cuda.synchronize()
    assert (dweight == 0).all() and (dw == 0).all() and (dbias == 0).all()
