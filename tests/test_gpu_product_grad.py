"""Backward pass of the experts' product on the GPU against the formula in 64 bits and against differences.

Tolerances, from the arithmetic. dz = dout act'(pre) is off by 2^-16 relative to
the sum of the absolute terms of act' (under 1.6 |dout|, times |up| for SwiGLU)
and rounded to bf16 before it meets a matrix: half a step, 2^-8 relative (not
without an activation: dz is dout). Sums of n products in 32 bits: (n + 8) 2^-23
of the absolute terms, then half a step of bf16. dbias: sums of the unrounded
dz, (rows + 8) 2^-24."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, HALF, NAMES, TINY, Dense, Routed, activate, activate_grad, check, ids

pytestmark = pytest.mark.gpu
ACTS = [ep.EP_ACT_NONE, ep.EP_ACT_SILU, ep.EP_ACT_GELU, ep.EP_ACT_SWIGLU]


class Case:
    def __init__(self, where, experts, k, n, act, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.where, self.e, self.k, self.n, self.act = where, experts, k, n, act
        self.wrows = 2 * n if act == ep.EP_ACT_SWIGLU else n
        self.x = torch.randn((where.rows, k), generator=g).to(BF)
        self.w = (torch.randn((experts, self.wrows, k), generator=g) * k**-0.5).to(BF)
        self.dout = torch.randn((where.rows, n), generator=g).to(BF)
        self.pre = (2 * torch.randn((where.rows, self.wrows), generator=g)).to(BF) if act != ep.EP_ACT_NONE else None
        self.clean = [None if t is None else t.double() for t in (self.x, self.dout, self.pre)]
        for t in (self.x, self.dout, self.pre):
            if t is not None:
                t[~where.owned] = float("nan")

    def run(self, dx=True, dw=True, dbias=True):
        c, dev = self.where, "cuda"
        p = ep.make_product(self.w.to(dev), self.act)
        ws = torch.full((ep.expert_product_grad_bytes(c.desc, p),), 255, dtype=torch.uint8, device=dev)
        gx = torch.full((c.rows + 2, self.k), 7.0, dtype=BF, device=dev) if dx else None
        gw = torch.full((self.e + 1, self.wrows, self.k), 7.0, dtype=BF, device=dev) if dw else None
        gb = torch.full((self.e + 1, self.wrows), 7.0, device=dev) if dbias else None
        ep.expert_product_grad(c.desc, p, self.dout.to(dev), self.x.to(dev),
                               None if self.pre is None else self.pre.to(dev), c.plan, ws,
                               dx=gx[1:-1] if dx else None, dw=gw[:-1] if dw else None, dbias=gb[:-1] if dbias else None)
        torch.cuda.synchronize()
        if dx:
            assert (gx[0] == 7).all() and (gx[-1] == 7).all() and (gx[1:-1][~c.owned.to(dev)] == 7).all()
        for t in (gw, gb):
            assert t is None or (t[-1] == 7).all()
        return (gx[1:-1].cpu() if dx else None, gw[:-1].cpu() if dw else None, gb[:-1].cpu() if dbias else None)

    def check(self, got=None):
        gx, gw, gb = got or self.run()
        x, dout, pre = self.clean
        half = 0.0 if self.act == ep.EP_ACT_NONE else 2.0**-8
        for e, (a, m) in enumerate(self.where.groups):
            r, w = slice(a, a + m), self.w[e].double()
            dz = dout[r] if pre is None else activate_grad(pre[r], dout[r], self.act)
            slack = torch.zeros_like(dz)
            if self.act in (ep.EP_ACT_SILU, ep.EP_ACT_GELU):
                slack = 1.6 * dout[r].abs() * 2.0**-16
            elif self.act == ep.EP_ACT_SWIGLU:
                gate, up = pre[r].chunk(2, -1)
                slack = torch.cat([1.6 * dout[r].abs() * up.abs(), dout[r].abs() * gate.abs()], -1) * 2.0**-16
            off = dz.abs() * half + slack
            if gx is not None and m:
                want, terms = dz @ w, (dz.abs() + off) @ w.abs()
                check(gx[r], want, off @ w.abs() + terms * (self.wrows + 8) * 2.0**-23 + HALF[BF] * want.abs() * 1.01 +
                      TINY[BF], f"dx of {e}")
            if gw is not None:
                want, terms = dz.T @ x[r], (dz.abs() + off).T @ x[r].abs()
                check(gw[e], want, off.T @ x[r].abs() + terms * (m + 8) * 2.0**-23 + HALF[BF] * want.abs() * 1.01 +
                      TINY[BF], f"dw of {e}")
            if gb is not None:
                check(gb[e], dz.sum(0), slack.sum(0) + dz.abs().sum(0) * (m + 8) * 2.0**-24, f"dbias of {e}")


def routed(n, t, e, r, seed=0, cap=0, only=None):
    return Routed(n, t, e, r, ids(n, t, e, r, seed, only), cap=cap)


@pytest.mark.parametrize("act", ACTS, ids=NAMES.get)
@pytest.mark.parametrize("n,t,e,r,k,m", [
    (1, 1, 4, 1, 8, 8),
    (1, 1, 8, 3, 72, 40),
    (4, 16, 16, 2, 256, 512),
    (2, 37, 6, 2, 520, 264),
    (1, 515, 3, 2, 200, 104),
    (1, 64, 1, 1, 264, 136),      # a step of k exactly full of rows
    (1, 700, 2, 1, 40, 304),
])
def test_product_grad(n, t, e, r, k, m, act):
    note(f"product grad {n} {t} {e} {r} {k} {m} {NAMES[act]}")
    Case(routed(n, t, e, r), e, k, m, act).check()


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU], ids=NAMES.get)
def test_product_grad_parts(act):
    """Each output alone is what all of them together give; twice the same bytes."""
    c = Case(routed(1, 130, 5, 2), 5, 136, 72, act)
    gx, gw, gb = c.run()
    for again in (c.run(), c.run(dw=False, dbias=False), c.run(dx=False, dbias=False), c.run(dx=False, dw=False)):
        for a, b in zip(again, (gx, gw, gb)):
            assert a is None or torch.equal(a, b)
    c.check((gx, gw, gb))


def test_product_grad_empty_experts_and_capacity():
    note("product grad empty experts")
    c = Case(routed(1, 50, 12, 2, only=[3, 4, 9]), 12, 72, 40, ep.EP_ACT_SILU)
    gx, gw, gb = c.run()
    c.check((gx, gw, gb))
    for e in (0, 2, 5, 11):
        assert (gw[e] == 0).all() and (gb[e] == 0).all()
    Case(routed(2, 64, 4, 2, cap=50), 4, 72, 40, ep.EP_ACT_SWIGLU).check()
    idx = ids(2, 0, 4, 2, 0)
    c = Case(Routed(2, 0, 4, 2, idx, cap=3), 4, 72, 40, ep.EP_ACT_GELU)
    gx, gw, gb = c.run()
    assert (gw == 0).all() and (gb == 0).all()


@pytest.mark.parametrize("n,rows,k,m,act", [(1, 1, 520, 264, ep.EP_ACT_GELU), (3, 70, 264, 40, ep.EP_ACT_SWIGLU),
                                            (2, 300, 128, 136, ep.EP_ACT_NONE)])
def test_dense_product_grad(n, rows, k, m, act):
    note(f"dense grad {n} {rows} {k} {m}")
    Case(Dense(n, rows), n, k, m, act).check()


@pytest.mark.parametrize("act", ACTS, ids=NAMES.get)
def test_product_grad_against_differences(act):
    """Directional derivative of sum(act(x w^T + b) dout) by central differences in 64 bits, at the pre-activations
    that the forward call stored."""
    note(f"product grad differences {NAMES[act]}")
    g = torch.Generator().manual_seed(9)
    where = routed(1, 24, 3, 2)
    c = Case(where, 3, 40, 24, act, seed=4)
    bias = torch.randn((3, c.wrows), generator=g).to(BF)
    x64, w64, b64, d64 = c.clean[0], c.w.double(), bias.double(), c.clean[1]
    if act != ep.EP_ACT_NONE:
        dev = "cuda"
        p = ep.make_product(c.w.to(dev), act, bias=bias.to(dev))
        pre = torch.zeros((where.rows, c.wrows), dtype=BF, device=dev)
        ep.expert_product(where.desc, p, [c.x.to(dev)], where.plan, torch.empty((where.rows, c.n), dtype=BF, device=dev),
                          pre=pre)
        c.pre = pre.cpu()
    gx, gw, gb = c.run()

    def loss(x, w, b):
        return sum(float((activate(x[a:a + m] @ w[e].T + b[e], act) * d64[a:a + m]).sum())
                   for e, (a, m) in enumerate(where.groups))
    u, v, b = (torch.randn(t.shape, generator=g).double() for t in (x64, w64, b64))
    u[~where.owned] = 0
    e = 2.0**-14
    slope = (loss(x64 + e * u, w64 + e * v, b64 + e * b) - loss(x64 - e * u, w64 - e * v, b64 - e * b)) / (2 * e)
    o = where.owned
    got = float((gx[o].double() * u[o]).sum() + (gw.double() * v).sum() + (gb.double() * b).sum())
    # The stored pre-activation is off by half a step of bf16 (|z| < 6 here: under 2^-6 absolute) and act'' is under
    # 1.1: each dz by 2^-6 |dout| and, for SwiGLU, by 2^-6 |dout| (1 + |up|); then dz, dx and dw by half a step each.
    z = torch.zeros((where.rows, c.wrows), dtype=torch.float64)
    for i, (a, m) in enumerate(where.groups):
        z[a:a + m] = x64[a:a + m] @ w64[i].T + b64[i]
    dz = activate_grad(z, d64, act)
    wide = torch.cat([d64, d64], -1) if act == ep.EP_ACT_SWIGLU else d64
    grow = 1 + z.abs().max() if act == ep.EP_ACT_SWIGLU else 1.0
    off = dz.abs() * 2.0**-8 + (0 if act == ep.EP_ACT_NONE else 2.0**-6 * 1.1 * grow * wide.abs())
    tol = 0.0
    for i, (a, m) in enumerate(where.groups):
        r = slice(a, a + m)
        tol += float(((off[r] @ w64[i].abs()) * u[r].abs()).sum() + ((off[r].T @ x64[r].abs()) * v[i].abs()).sum() +
                     (off[r].sum(0) * b[i].abs()).sum())
    tol += float((gx[o].double() * u[o]).abs().sum() + (gw.double() * v).abs().sum()) * 2.0**-8
    assert abs(got - slope) <= tol, (got, slope, tol)
    assert tol < 0.5 * float((gx[o].double() * u[o]).abs().sum() + (gw.double() * v).abs().sum())


def test_product_grad_special_values():
    """NaN in one row's gradient reaches that row of dx, its expert's dw and dbias, and no other expert."""
    note("product grad special values")
    c = Case(routed(1, 70, 4, 1), 4, 72, 40, ep.EP_ACT_SILU)
    gx, gw, gb = c.run()
    a, m = c.where.groups[1]
    assert m > 2
    c.dout[a + 1, 5] = float("nan")
    hx, hw, hb = c.run()
    keep = c.where.owned.clone()
    keep[a + 1] = False
    assert torch.equal(hx[keep], gx[keep]) and hx[a + 1].isnan().all()
    for e in (0, 2, 3):
        assert torch.equal(hw[e], gw[e]) and torch.equal(hb[e], gb[e])
    cols = torch.arange(40) != 5
    assert torch.equal(hw[1][cols], gw[1][cols]) and hw[1][5].isnan().all()
    assert torch.equal(hb[1][cols], gb[1][cols]) and hb[1][5].isnan()


def sorted_rows(sizes):
    idx = torch.cat([torch.full((m,), e, dtype=torch.int32) for e, m in enumerate(sizes)])
    idx = idx[torch.randperm(len(idx), generator=torch.Generator().manual_seed(1))]
    return Routed(1, len(idx), len(sizes), 1, idx.view(1, -1, 1))


@pytest.mark.parametrize("sizes,k,n,act", [
    ([256, 0, 257, 64, 65, 1, 128, 129, 192, 193, 512, 30, 250, 3, 700, 31] * 2, 1920, 136, ep.EP_ACT_NONE),
    ([4113], 4096, 72, ep.EP_ACT_SILU),          # rows in tiles of 256
    ([100, 0, 260, 64], 2088, 2048, ep.EP_ACT_NONE),   # weights in tiles of 256, several each
    ([900, 124], 1160, 1032, ep.EP_ACT_SWIGLU),
    ([20] * 10, 3840, 72, ep.EP_ACT_GELU),
    ([2100, 40], 64, 72, ep.EP_ACT_SILU),        # more row blocks of one expert than a group of lanes takes at once
])
def test_product_grad_large(sizes, k, n, act):
    note(f"product grad large {sizes[:4]} {k} {n} {act}")
    Case(sorted_rows(sizes), len(sizes), k, n, act).check()


def test_product_grad_of_a_plan_that_was_never_made():
    """Offsets of any value: nothing outside the rank's rows and the workspace is touched."""
    note("product grad broken plan")
    for fill in (0, 127, 255):
        where = sorted_rows([50, 60, 70])
        c = Case(where, 3, 72, 40, ep.EP_ACT_SWIGLU)
        where.plan.fill_(fill)
        where.owned[:] = True
        c.run()
