"""Workspaces of the backward passes, exactly as large as the size functions say, between guards: nothing outside is
written, nothing in them is read before it is written (they hold NaN), whatever share of their room a call needs.

Tolerances: dweight and dbias are sums of n 32-bit terms, each off by 2^-17 for the norm and 2^-16 (times 1.6 |dout|,
by |up| for SwiGLU's gates) for an activation: (n + 32) 2^-24 of the absolute terms and that."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, NAMES, activate_grad, check, guarded, norm_grad

pytestmark = pytest.mark.gpu


def workspace(nbytes):
    ws, whole = guarded((nbytes,), torch.uint8, 255)
    return ws, whole


@pytest.mark.parametrize("rows,hidden", [(1, 8), (1, 7168), (7, 512), (8, 1024), (9, 1024), (255, 8200), (257, 8200),
                                         (300, 32768), (511, 7168), (512, 7168), (513, 7168), (2047, 1024), (4104, 40)])
def test_norm_grad_workspace(rows, hidden):
    note(f"norm grad workspace {rows} {hidden}")
    g = torch.Generator().manual_seed(rows + hidden)
    h, dy, w = (torch.randn(s, generator=g).to(BF) for s in ((rows, hidden), (rows, hidden), (hidden,)))
    ws, whole = workspace(ep.rms_norm_grad_bytes(rows, hidden))
    (dx, a), (dw, b) = guarded((rows, hidden), BF), guarded((hidden,), torch.float32)
    ep.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), 1e-5, dx, dw, ws)
    torch.cuda.synchronize()
    for f in (whole, a, b):
        f()
    h64, dy64 = h.double(), dy.double()
    _, want = norm_grad(dy64, h64, w.double(), torch.zeros_like(h64), 1e-5)
    terms = (dy64 * h64 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt()).abs().sum(0)
    check(dw, want, terms * ((rows + 32) * 2.0**-24 + 2.0**-17), "dweight")


def routed(sizes):
    """Plan of one rank whose experts get these numbers of rows, and their first rows."""
    idx = torch.cat([torch.full((m,), e, dtype=torch.int32) for e, m in enumerate(sizes)])
    d = ep.make_desc(1, len(idx), 8, len(sizes), 1)
    plan = torch.zeros(ep.plan_bytes(d), dtype=torch.uint8, device="cuda")
    ep.plan(d, idx.view(1, -1, 1).cuda(), plan, torch.zeros(1, dtype=torch.int32, device="cuda"))
    first = torch.tensor([0] + list(sizes)).cumsum(0)
    return d, plan, [(int(a), m) for a, m in zip(first, sizes)]


def dense(n, rows):
    d = ep.make_desc(n, 1, 8, n, 1, cap_rows=rows)
    return d, None, [(e * rows, rows) for e in range(n)]


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_GELU, ep.EP_ACT_SWIGLU], ids=NAMES.get)
@pytest.mark.parametrize("make,arg", [
    (routed, (([1] * 256),)),                  # a row block for every row
    (routed, (([33] * 64),)),                  # two for 33 rows
    (routed, (([1, 0, 0, 33] * 40),)),
    (routed, (([31, 32, 33, 64, 65] * 8),)),
    (dense, (40, 33)), (dense, (1, 1)), (dense, (3, 257)),
])
def test_product_grad_workspace(make, arg, act):
    d, plan, groups = make(*arg)
    note(f"product grad workspace {len(groups)} {groups[:4]} {NAMES[act]}")
    e, k, m = d.n_experts, 72, 264
    wrows = 2 * m if act == ep.EP_ACT_SWIGLU else m
    rows = d.n_ranks * ep.capacity(d)
    g = torch.Generator().manual_seed(5)
    x, dout = torch.randn((rows, k), generator=g).to(BF), torch.randn((rows, m), generator=g).to(BF)
    pre = torch.randn((rows, wrows), generator=g).to(BF) if act != ep.EP_ACT_NONE else None
    p = ep.make_product(torch.randn((e, wrows, k), generator=g).to(BF).cuda(), act)
    ws, whole = workspace(ep.expert_product_grad_bytes(d, p))
    outs = [guarded(s, t) for s, t in (((rows, k), BF), ((e, wrows, k), BF), ((e, wrows), torch.float32))]
    (dx, _), (dw, _), (db, _) = outs
    ep.expert_product_grad(d, p, dout.cuda(), x.cuda(), None if pre is None else pre.cuda(), plan, ws, dx, dw, db)
    torch.cuda.synchronize()
    whole()
    for _, f in outs:
        f()
    for j, (a, n) in enumerate(groups):
        r = slice(a, a + n)
        dz = dout[r].double() if pre is None else activate_grad(pre[r].double(), dout[r].double(), act)
        slack = 0.0 if pre is None else 1.6 * 2.0**-16 * dout[r].double().abs()
        if act == ep.EP_ACT_SWIGLU:
            gate, up = pre[r].double().chunk(2, -1)
            slack = torch.cat([slack * up.abs(), slack * gate.abs()], -1)
        if pre is not None:
            slack = slack.sum(0)
        check(db[j], dz.sum(0), slack + dz.abs().sum(0) * (n + 32) * 2.0**-24, f"dbias of {j}")
        assert n == 0 or (not dx[r].isnan().any() and not dw[j].isnan().any())
