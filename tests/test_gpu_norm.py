"""RMS norm and its backward pass on the GPU against the definition in 64 bits.

Tolerances, from the arithmetic. The sum of squares is a 32-bit sum of at most
32 fused terms per thread, 6 adds in the wave and 16 of waves, all positive:
off by under 64 2^-24 relative, the root of it by half that and an ulp or two,
and two products follow: under 2^-18 in all. Then y is rounded to its type:
half a step. The sums h are rounded 32-bit sums of two 16-bit values: exact,
bit for bit. A code is off by half a step of e4m3 (2^-4 relative, 2^-10 of the
scale under the normal range), the scale by the 2^-18 above.
Backward: dx = dsum + r (g - h r^2 mean(g h)); mean(g h) is off by 64 2^-24 of
mean |g h| and r by 2^-18, so the bracket by 2^-17 of its absolute terms.
dweight sums 32-bit terms over the rows: (rows + 32) 2^-24 of the absolute
terms, each off by 2^-17."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, F8, HALF, HF, TINY, check, norm, norm_grad

pytestmark = pytest.mark.gpu


def rows_of(rows, hidden, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, hidden), generator=g) * scale).to(dtype)


def weight_of(hidden, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.2 * torch.randn(hidden, generator=g)).to(dtype)


def check_codes(codes, scales, y, what):
    """Codes and scales against the 64-bit rows y."""
    blocks = y.view(y.shape[0], -1, 128)
    top = blocks.abs().amax(-1)
    scale = torch.where(top > 0, top / 448, 1.0)
    check(scales, scale, scale * 2.0**-17, what + " scales")
    value = codes.cpu().double().view_as(blocks) * scales.cpu().double()[..., None]
    check(value, blocks, blocks.abs() * (2.0**-4 + 2.0**-16) + scale[..., None] * 2.0**-10, what + " codes")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 56), (1, 7168), (5, 128), (7, 1000), (2, 1024), (3, 4096), (2, 8192),
                                         (2, 8200), (3, 16384), (2, 16392), (2, 32768), (300, 520)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, hidden, dtype, residual):
    note(f"norm {rows} {hidden} {dtype} {residual}")
    x, w = rows_of(rows, hidden, dtype, 1), weight_of(hidden, dtype, 2)
    r = rows_of(rows, hidden, dtype, 3, 4.0) if residual else None
    h = (x.float() + r.float()).to(dtype) if residual else x
    y = torch.full((rows + 1, hidden), 7.0, dtype=dtype, device="cuda")
    total = torch.full((rows + 1, hidden), 7.0, dtype=dtype, device="cuda") if residual else None
    quant = hidden % 128 == 0
    codes = torch.zeros((rows, hidden), dtype=F8, device="cuda") if quant else None
    scales = torch.full((rows, hidden // 128), 7.0, device="cuda") if quant else None
    ep.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(),
                sum=None if total is None else total[:rows], y=y[:rows], codes=codes, scales=scales)
    torch.cuda.synchronize()
    want = norm(h.double(), w.double(), 1e-5)
    check(y[:rows], want, want.abs() * (HALF[dtype] + 2.0**-18) + TINY[dtype], "y")
    assert (y[rows] == 7).all()
    if residual:
        assert torch.equal(total[:rows].cpu(), h) and (total[rows] == 7).all()
    if quant:
        check_codes(codes, scales, want, "both")
        only, fine = torch.zeros_like(codes), torch.zeros_like(scales)
        ep.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(), sum=total, codes=only,
                    scales=fine)
        assert torch.equal(only.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(fine, scales)


def test_norm_in_place():
    x, r, w = rows_of(9, 256, BF, 1).cuda(), rows_of(9, 256, BF, 2).cuda(), weight_of(256, BF, 3).cuda()
    total, y, here, z = torch.empty_like(x), torch.empty_like(x), r.clone(), torch.empty_like(x)
    ep.rms_norm(x, w, 1e-6, residual=r, sum=total, y=y)
    ep.rms_norm(x, w, 1e-6, residual=here, sum=here, y=z)
    assert torch.equal(here, total) and torch.equal(z, y)


def test_norm_special_rows():
    """A row of zeros, one with an infinity, one with NaN, one of tiny values: no other row changes."""
    note("norm special rows")
    x = rows_of(8, 256, BF, 5)
    w = weight_of(256, BF, 6)
    plain = torch.empty_like(x, device="cuda")
    ep.rms_norm(x.cuda(), w.cuda(), 1e-6, y=plain)
    x[1] = 0
    x[3, 77] = float("inf")
    x[5, 200] = float("nan")
    x[6] = rows_of(1, 256, BF, 7, 2.0**-60)[0]
    y = torch.empty_like(plain)
    codes, scales = torch.zeros((8, 256), dtype=F8, device="cuda"), torch.zeros((8, 2), device="cuda")
    ep.rms_norm(x.cuda(), w.cuda(), 1e-6, y=y, codes=codes, scales=scales)
    for i in (0, 2, 4, 7):
        assert torch.equal(y[i], plain[i])
    assert (y[1] == 0).all() and (codes[1].view(torch.uint8) & 127 == 0).all() and (scales[1] == 1).all()
    # inf / inf is NaN and the row's other values are 0; a NaN makes its whole row NaN.
    assert y[3, 77].isnan() and (y[3, :77] == 0).all() and (y[3, 78:] == 0).all()
    assert codes[3].view(torch.uint8)[77] == 0x7F
    assert y[5].isnan().all() and (codes[5].view(torch.uint8) == 0x7F).all()
    want = norm(x[6:7].double(), w.double(), 1e-6)
    check(y[6:7], want, want.abs() * (2.0**-8 + 2.0**-18), "tiny")


def test_norm_codes_are_the_dispatch_planes():
    """Codes of a bf16 value are the quantising sender's: rows whose normed values bf16 holds exactly."""
    note("norm codes against the quantising sender")
    n, t, h = 1, 16, 512
    g = torch.Generator().manual_seed(3)
    x = torch.where(torch.rand((t, h), generator=g) < 0.5, -1.0, 1.0).to(BF).cuda()   # rms 1, eps 0: y = x weight
    w = (torch.randn(h, generator=g).to(BF) * 8).cuda()
    codes, scales = torch.zeros((t, h), dtype=F8, device="cuda"), torch.zeros((t, h // 128), device="cuda")
    y = torch.empty_like(x)
    ep.rms_norm(x, w, 0.0, y=y, codes=codes, scales=scales)
    assert torch.equal(y, x * w)
    d = ep.make_desc(n, t, h, 1, 1, ep.EP_PAYLOAD_FP8_B128)
    b = ep.Buffers(d)
    b.idx.zero_()
    ep.dispatch_quant(d, b.idx, y.view(n, t, h), b.plan_ws, b.send, b.grouped, b.status)
    assert torch.equal(b.grouped[0].view(-1)[:t * h], codes.view(torch.uint8).view(-1))
    assert torch.equal(b.grouped[1].view(torch.float32).view(-1)[:t * h // 128], scales.view(-1))


def grad_case(rows, hidden, dtype, dsum, seed=0):
    h, dy = rows_of(rows, hidden, dtype, seed, 2.0), rows_of(rows, hidden, dtype, seed + 1)
    w = weight_of(hidden, dtype, seed + 2)
    s = rows_of(rows, hidden, dtype, seed + 3) if dsum else None
    return h, dy, w, s


def run_grad(h, dy, w, s, eps, want_weight=True):
    rows, hidden = h.shape
    dx = torch.full((rows + 1, hidden), 7.0, dtype=h.dtype, device="cuda")
    dw = torch.full((hidden + 8,), 7.0, device="cuda") if want_weight else None
    ws = torch.full((ep.rms_norm_grad_bytes(rows, hidden),), 255, dtype=torch.uint8, device="cuda")
    ep.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), eps, dx[:rows], None if dw is None else dw[:hidden], ws,
                     dsum=None if s is None else s.cuda())
    torch.cuda.synchronize()
    assert (dx[rows] == 7).all() and (dw is None or (dw[hidden:] == 7).all())
    return dx[:rows], None if dw is None else dw[:hidden]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,hidden,dsum", [(1, 8, False), (2, 56, True), (1, 7168, True), (5, 128, False), (700, 1000, True),
                                              (1500, 264, True), (3, 4096, True), (2, 8200, True), (3, 16384, False),
                                              (2, 16392, True), (3, 32768, True), (600, 7168, True)])
def test_norm_grad(rows, hidden, dsum, dtype):
    note(f"norm grad {rows} {hidden} {dsum} {dtype}")
    h, dy, w, s = grad_case(rows, hidden, dtype, dsum)
    dx, dw = run_grad(h, dy, w, s, 1e-5)
    h64, dy64, w64 = h.double(), dy.double(), w.double()
    s64 = s.double() if dsum else torch.zeros_like(h64)
    want, want_w = norm_grad(dy64, h64, w64, s64, 1e-5)
    r = 1 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt()
    g = (dy64 * w64).abs()
    terms = r * (g + h64.abs() * r * r * (g * h64.abs()).mean(1, keepdim=True)) + s64.abs() * 2.0**-7
    check(dx, want, HALF[dtype] * want.abs() + 2.0**-17 * terms + TINY[dtype], "dx")
    terms = (dy64 * h64 * r).abs().sum(0)
    check(dw, want_w, terms * ((rows + 32) * 2.0**-24 + 2.0**-17), "dweight")
    again, same = run_grad(h, dy, w, s, 1e-5)
    assert torch.equal(again, dx) and torch.equal(same, dw)
    only, _ = run_grad(h, dy, w, s, 1e-5, want_weight=False)
    assert torch.equal(only, dx)


def test_norm_grad_against_differences():
    """The directional derivative of sum(y dy) + sum(h dsum) by central differences in 64 bits."""
    h, dy, w, s = grad_case(6, 72, BF, True, seed=11)
    dx, dw = run_grad(h, dy, w, s, 1e-3)
    h64, dy64, w64, s64 = h.double(), dy.double(), w.double(), s.double()

    def loss(a, b):
        return float((norm(a, b, 1e-3) * dy64).sum() + (a * s64).sum())
    g = torch.Generator().manual_seed(5)
    for _ in range(4):
        u, v = torch.randn(h64.shape, generator=g).double(), torch.randn(w64.shape, generator=g).double()
        e = 2.0**-16
        slope = (loss(h64 + e * u, w64 + e * v) - loss(h64 - e * u, w64 - e * v)) / (2 * e)
        got = float((dx.cpu().double() * u).sum() + (dw.cpu().double() * v).sum())
        # Each dx is off by half a bf16 step and 2^-17 of its terms, which are under 16 times it here;
        # the differences by e^2 times third derivatives, under 2^-20 of the terms.
        tol = float((dx.cpu().double().abs() * u.abs()).sum()) * 2.0**-7.9 + float((dw.cpu().double() * v).abs().sum()) * 2.0**-12
        assert abs(got - slope) <= tol, (got, slope, tol)


def test_norm_grad_in_place_and_no_rows():
    h, dy, w, s = (t.cuda() for t in grad_case(40, 264, BF, True))
    ws = torch.empty(ep.rms_norm_grad_bytes(40, 264), dtype=torch.uint8, device="cuda")
    dx, dw, here, dw2 = torch.empty_like(h), torch.empty(264, device="cuda"), s.clone(), torch.empty(264, device="cuda")
    ep.rms_norm_grad(dy, h, w, 1e-6, dx, dw, ws, dsum=s)
    ep.rms_norm_grad(dy, h, w, 1e-6, here, dw2, ws, dsum=here)
    assert torch.equal(here, dx) and torch.equal(dw, dw2)
    none = h[:0]
    ep.rms_norm(none, w, 1e-6, y=none.clone())
    dw.fill_(7)
    ep.rms_norm_grad(none, none, w, 1e-6, none.clone(), dw, ws)
    assert (dw == 0).all()
