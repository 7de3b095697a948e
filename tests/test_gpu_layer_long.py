"""Batches of more rows or tokens than one launch holds (2^21), against the definition in 64 bits. Tolerances as in
test_gpu_norm.py and test_gpu_route_grad.py."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, F8, HALF, TINY, check, guarded, norm, norm_grad

pytestmark = pytest.mark.gpu
ROWS = (1 << 21) + 5


def test_long_norm():
    note("long norm")
    g = torch.Generator().manual_seed(1)
    x, r, dy = (torch.randn((ROWS, 8), generator=g).to(BF) for _ in range(3))
    w = (1 + 0.2 * torch.randn(8, generator=g)).to(BF)
    (total, a), (y, b), (dx, c) = (guarded((ROWS, 8), BF) for _ in range(3))
    dw = torch.empty(8, device="cuda")
    ep.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=r.cuda(), sum=total, y=y)
    ws = torch.empty(ep.rms_norm_grad_bytes(ROWS, 8), dtype=torch.uint8, device="cuda")
    ep.rms_norm_grad(dy.cuda(), total, w.cuda(), 1e-5, dx, dw, ws)
    torch.cuda.synchronize()
    for f in (a, b, c):
        f()
    h = (x.float() + r.float()).to(BF)
    assert torch.equal(total.cpu(), h)
    h64, dy64, w64 = h.double(), dy.double(), w.double()
    want = norm(h64, w64, 1e-5)
    check(y, want, want.abs() * (HALF[BF] + 2.0**-18) + TINY[BF], "y")
    want, want_w = norm_grad(dy64, h64, w64, torch.zeros_like(h64), 1e-5)
    rs = 1 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt()
    gr = (dy64 * w64).abs()
    terms = rs * (gr + h64.abs() * rs * rs * (gr * h64.abs()).mean(1, keepdim=True))
    check(dx, want, HALF[BF] * want.abs() + 2.0**-17 * terms + TINY[BF], "dx")
    # 512 workgroups of eight waves: 513 terms one after another, then 7 waves' sums, then 512 parts in 32 lines of 16.
    check(dw, want_w, (dy64 * h64 * rs).abs().sum(0) * (640 * 2.0**-24 + 2.0**-17), "dweight")


def test_long_norm_codes():
    """Codes and scales behind the first launch's rows: the same bytes as those rows get by themselves."""
    note("long norm codes")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((ROWS, 128), dtype=BF, device="cuda").normal_(generator=g)
    w = torch.ones(128, dtype=BF, device="cuda")
    (codes, a), (scales, b) = guarded((ROWS, 128), F8, 7.0), guarded((ROWS, 1), torch.float32)
    ep.rms_norm(x, w, 1e-5, codes=codes, scales=scales)
    last = x[-700:].contiguous()
    c, s = torch.empty((700, 128), dtype=F8, device="cuda"), torch.empty((700, 1), device="cuda")
    ep.rms_norm(last, w, 1e-5, codes=c, scales=s)
    torch.cuda.synchronize()
    a()
    b()
    assert torch.equal(codes[-700:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-700:], s)
    top = x.float().abs().amax(1) * torch.rsqrt(x.float().square().mean(1) + 1e-5) / 448
    assert ((scales[:, 0] - top).abs() <= top * 2.0**-17).all()


def test_long_route_gradients():
    """2^21 + 5 tokens of one rank, each with two slots of three experts, some dropped for want of room."""
    note("long route gradients")
    t, e, r, h = ROWS, 3, 2, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.rand((t, e), generator=g, device="cuda").argsort(1)[:, :r].to(torch.int32).view(1, t, r)
    cap = 2 * t - 1000
    d = ep.make_desc(1, t, h, e, r, cap_rows=cap)
    plan, status = torch.zeros(ep.plan_bytes(d), dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.plan(d, idx, plan, status)
    flat = idx.flatten().long()
    count = torch.bincount(flat, minlength=e)
    order = torch.sort(flat, stable=True)[1]
    row = torch.empty_like(flat)
    row[order] = torch.arange(t * r, device="cuda")
    there = row < cap
    assert int(count.sum()) == t * r and int((~there).sum()) == 1000
    dout = torch.empty((1, t, h), dtype=BF, device="cuda").normal_(generator=g)
    y, dg = (torch.empty((cap, h), dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))
    wt = torch.rand((1, t, r), device="cuda", generator=g)
    (dy, a), (dwt, b), (dx, c) = guarded((cap, h), BF), guarded((1, t, r), torch.float32), guarded((1, t, h), BF)
    ep.combine_grad(d, dout, y, wt, plan, dy, dwt)
    ep.dispatch_grad(d, dg, plan, dx)
    torch.cuda.synchronize()
    for f in (a, b, c):
        f()
    assert int(status) == ep.EP_STATUS_CAPACITY
    do = dout.double().view(t, 1, h).expand(-1, r, -1).reshape(-1, h)
    at = row[there]
    want = wt.double().view(-1, 1)[there] * do[there]
    assert ((dy[at].double() - want).abs() <= want.abs() * (HALF[BF] + 2.0**-23) + TINY[BF]).all()
    want, terms = (torch.zeros(t * r, dtype=torch.float64, device="cuda") for _ in range(2))
    want[there], terms[there] = (y[at].double() * do[there]).sum(1), (y[at].double() * do[there]).abs().sum(1)
    assert ((dwt.view(-1).double() - want).abs() <= terms * h * 2.0**-24).all()
    parts = torch.zeros((t * r, h), dtype=torch.float64, device="cuda")
    parts[there] = dg[at].double()
    want, terms = parts.view(t, r, h).sum(1), parts.view(t, r, h).abs().sum(1)
    assert ((dx.view(t, h).double() - want).abs() <= want.abs() * HALF[BF] + terms * r * 2.0**-23 + TINY[BF]).all()
