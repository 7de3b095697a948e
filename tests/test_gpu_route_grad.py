"""Backward passes of combine and dispatch on the GPU against the definition in 64 bits.

Tolerances: dy = w dout is a 32-bit product rounded to bf16: half a step and
2^-24. dweights is a 32-bit sum of H exact products: (H / threads + 24) adds
in a row, at most H: H 2^-24 of the absolute terms. dx sums k + 1 terms in 32
bits (k 2^-24 of the absolute terms), then half a step."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, HALF, TINY, Routed, check, ids

pytestmark = pytest.mark.gpu


def case(n, t, e, r, h, cap=0, idx=None, seed=0):
    where = Routed(n, t, e, r, ids(n, t, e, r, seed) if idx is None else idx, hidden=h, cap=cap)
    g = torch.Generator().manual_seed(seed + 1)
    dout = torch.randn((n, t, h), generator=g).to(BF)
    y, dg = (torch.randn((where.rows, h), generator=g).to(BF) for _ in range(2))
    y[~where.owned] = float("nan")
    dg[~where.owned] = float("nan")
    return where, dout, y, dg, torch.rand((n, t, r), generator=g), torch.randn((n, t, h), generator=g).to(BF)


def combine_grad(where, dout, y, w, dy=True, dweights=True):
    n, t, h = dout.shape
    gy = torch.full((where.rows + 2, h), 7.0, dtype=BF, device="cuda") if dy else None
    gw = torch.full((n * t + 1, w.shape[2]), 7.0, device="cuda") if dweights else None
    ep.combine_grad(where.desc, dout.cuda(), y.cuda(), w.cuda(), where.plan, gy[1:-1] if dy else None,
                    gw[:-1] if dweights else None)
    torch.cuda.synchronize()
    if dy:
        assert (gy[0] == 7).all() and (gy[-1] == 7).all() and (gy[1:-1][~where.owned.cuda()] == 7).all()
    assert gw is None or (gw[-1] == 7).all()
    return gy[1:-1].cpu() if dy else None, gw[:-1].cpu() if dweights else None


SHAPES = [(1, 1, 1, 1, 8, 0), (4, 16, 16, 2, 256, 0), (2, 33, 6, 3, 1000, 0), (3, 20, 9, 9, 72, 0), (2, 40, 4, 2, 264, 30),
          (1, 5, 64, 64, 128, 0), (1, 3, 4, 2, 7168, 0), (1, 3, 4, 4, 16392, 0), (2, 2, 4, 2, 40000, 0)]


@pytest.mark.parametrize("n,t,e,r,h,cap", SHAPES)
def test_combine_grad(n, t, e, r, h, cap):
    note(f"combine grad {n} {t} {e} {r} {h} {cap}")
    where, dout, y, _, w, _ = case(n, t, e, r, h, cap)
    gy, gw = combine_grad(where, dout, y, w)
    d = dout.double().view(n * t, 1, h).expand(-1, r, -1).reshape(-1, h)
    there = where.row >= 0
    rows = where.row[there]
    want = w.double().view(-1, 1)[there] * d[there]
    check(gy[rows], want, want.abs() * (HALF[BF] + 2.0**-23) + TINY[BF], "dy")
    want, terms = torch.zeros(n * t * r, dtype=torch.float64), torch.zeros(n * t * r, dtype=torch.float64)
    want[there] = (y.double()[rows] * d[there]).sum(1)
    terms[there] = (y.double()[rows] * d[there]).abs().sum(1)
    check(gw.view(-1), want, terms * h * 2.0**-24, "dweights")
    assert (gw.view(-1)[~there] == 0).all()
    for parts in ((True, False), (False, True), (True, True)):
        a, b = combine_grad(where, dout, y, w, *parts)
        assert (a is None or torch.equal(a[rows], gy[rows])) and (b is None or torch.equal(b, gw))


@pytest.mark.parametrize("n,t,e,r,h,cap", SHAPES)
@pytest.mark.parametrize("past", [False, True])
def test_dispatch_grad(n, t, e, r, h, cap, past):
    note(f"dispatch grad {n} {t} {e} {r} {h} {cap} {past}")
    where, _, _, dg, _, add = case(n, t, e, r, h, cap)
    dx = torch.full((n * t + 1, h), 7.0, dtype=BF, device="cuda")
    ep.dispatch_grad(where.desc, dg.cuda(), where.plan, dx[:-1], add=add.cuda() if past else None)
    torch.cuda.synchronize()
    assert (dx[-1] == 7).all()
    parts = torch.zeros((n * t * r, h), dtype=torch.float64)
    there = where.row >= 0
    parts[there] = dg.double()[where.row[there]]
    parts = parts.view(n * t, r, h)
    base = add.double().view(n * t, h) if past else torch.zeros((n * t, h), dtype=torch.float64)
    want = parts.sum(1) + base
    terms = parts.abs().sum(1) + base.abs()
    check(dx[:-1], want, want.abs() * HALF[BF] + terms * r * 2.0**-23 + TINY[BF], "dx")
    if past:   # in place
        here = add.cuda()
        ep.dispatch_grad(where.desc, dg.cuda(), where.plan, here, add=here)
        assert torch.equal(here.view(n * t, h), dx[:-1])


def test_repeated_and_bad_ids():
    """A token that names an expert twice has two rows of it; ids outside the range have none."""
    idx = torch.tensor([[[1, 1, 3], [-1, 4, 0]], [[2, 2, 2], [9, 9, 9]]], dtype=torch.int32)
    where, dout, y, dg, w, _ = case(2, 2, 4, 3, 64, idx=idx)
    gy, gw = combine_grad(where, dout, y, w)
    there = where.row >= 0
    assert there.sum() == 7 and (gw.view(-1)[~there] == 0).all()
    d = dout.double().view(4, 1, 64).expand(-1, 3, -1).reshape(-1, 64)
    want = w.double().view(-1, 1)[there] * d[there]
    check(gy[where.row[there]], want, want.abs() * (HALF[BF] + 2.0**-23) + TINY[BF], "dy")
    dx = torch.empty((2, 2, 64), dtype=BF, device="cuda")
    ep.dispatch_grad(where.desc, dg.cuda(), where.plan, dx)
    parts = torch.zeros((12, 64), dtype=torch.float64)
    parts[there] = dg.double()[where.row[there]]
    want, terms = parts.view(4, 3, 64).sum(1), parts.view(4, 3, 64).abs().sum(1)
    check(dx.view(4, 64), want, want.abs() * HALF[BF] + terms * 2.0**-21 + TINY[BF], "dx")
    assert (dx.view(4, 64)[3] == 0).all()


def test_combine_grad_against_differences():
    """The directional derivative of sum(out dout), out = sum_k w_k y_k, by differences (it is linear in each)."""
    where, dout, y, _, w, _ = case(2, 12, 4, 2, 64)
    gy, gw = combine_grad(where, dout, y, w)
    g = torch.Generator().manual_seed(8)
    o = where.owned
    u, v = torch.randn(y.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
    y64 = torch.where(o[:, None], y.double(), 0.0)

    def loss(y, w):
        out = (w.view(-1, 1) * y[where.row]).view(24, 2, 64).sum(1)
        return float((out * dout.double().view(24, 64)).sum())
    e = 2.0**-10
    slope = (loss(y64 + e * u, w.double() + e * v) - loss(y64 - e * u, w.double() - e * v)) / (2 * e)
    parts = (gy[o].double() * u[o]).sum() + (gw.view_as(w).double() * v).sum()
    tol = float((gy[o].double() * u[o]).abs().sum()) * 2.0**-7.9 + float((gw.view_as(w).double() * v).abs().sum()) * 2.0**-16
    assert abs(float(parts) - slope) <= tol
