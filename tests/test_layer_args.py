"""Refusals of the operators around dispatch and combine (no GPU): the checks that come before the
device is looked up, the binding's own, and the sizes of workspaces."""
import ctypes

import pytest
import torch

import combine_ep_plan_amd as ep

FAKE = 0x10000
BAD, TOO_LARGE = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def norm(**kw):
    a = dict(weight=FAKE, rows=4, hidden=256, dtype=ep.EP_DTYPE_BF16, eps=1e-6, reserved=0)
    a.update(kw)
    return ep.Norm(**a)


def call_norm(n, x=FAKE, residual=None, total=None, y=FAKE, codes=None, scales=None):
    return ep.lib().ep_rms_norm(ctypes.byref(n), x, residual, total, y, codes, scales, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=ep.EP_DTYPE_E4M3), BAD), (dict(dtype=-1), BAD), (dict(reserved=1), BAD), (dict(rows=-1), BAD),
    (dict(hidden=0), BAD), (dict(hidden=12), BAD), (dict(hidden=-8), BAD), (dict(eps=-1e-6), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(hidden=ep.EP_NORM_MAX_HIDDEN + 8), TOO_LARGE), (dict(rows=1 << 31), TOO_LARGE),
])
def test_norms_are_checked_before_the_device(kw, code):
    assert call_norm(norm(**kw)) == code and ep.last_error() != ""
    assert ep.lib().ep_rms_norm_grad(ctypes.byref(norm(**kw)), FAKE, FAKE, None, FAKE, FAKE, FAKE, None) == code
    assert ep.lib().ep_rms_norm_grad_bytes(ctypes.byref(norm(**kw))) == 0


def test_norm_outputs_are_checked_before_the_device():
    assert call_norm(norm(), residual=FAKE) == BAD
    assert call_norm(norm(), total=FAKE) == BAD
    assert call_norm(norm(), codes=FAKE) == BAD and call_norm(norm(), scales=FAKE) == BAD
    assert call_norm(norm(), y=None) == BAD
    assert call_norm(norm(hidden=264), codes=FAKE, scales=FAKE) == BAD       # no whole blocks of 128
    assert ep.lib().ep_rms_norm_grad(ctypes.byref(norm()), FAKE, FAKE, None, None, FAKE, FAKE, None) == BAD
    assert ep.lib().ep_rms_norm(None, FAKE, None, None, FAKE, None, None, None) == BAD
    assert call_norm(norm(rows=0), x=None) == ep.EP_OK                      # nothing to do


def test_norm_workspace_holds_a_row_per_part():
    assert ep.rms_norm_grad_bytes(0, 256) == 0
    assert ep.rms_norm_grad_bytes(1, 256) == 4 * 256
    for rows in (1 << 20, 1 << 24):
        assert ep.rms_norm_grad_bytes(rows, 7168) == 512 * 4 * 7168
    assert ep.rms_norm_grad_bytes(1 << 20, 32768) == 256 * 4 * 32768


def desc(**kw):
    a = dict(n_ranks=2, tokens=8, hidden=64, n_experts=4, topk=2, payload=0, cap_rows=16)
    a.update(kw)
    return ep.make_desc(**a)


def product(**kw):
    a = dict(w=FAKE, w_scale=None, bias=None, inn=64, out=32, act=ep.EP_ACT_NONE, dtype=ep.EP_DTYPE_BF16)
    a.update(kw)
    return ep.Product(**a)


def call_product(p, d=None, x=(FAKE, None), plan=FAKE):
    return ep.lib().ep_expert_product(ctypes.byref(d or desc()), ctypes.byref(p), (ctypes.c_void_p * 2)(*x), plan,
                                      None, None, FAKE, None)


def call_grad(p, d=None, pre=None, dx=FAKE, dw=FAKE, dbias=FAKE):
    return ep.lib().ep_expert_product_grad(ctypes.byref(d or desc()), ctypes.byref(p), FAKE, FAKE, pre, FAKE, FAKE, dx,
                                           dw, dbias, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=ep.EP_DTYPE_F16), BAD), (dict(act=4), BAD), (dict(act=-1), BAD), (dict(inn=0), BAD), (dict(out=0), BAD),
    (dict(inn=60), BAD), (dict(out=-8), BAD), (dict(w_scale=FAKE), BAD),
    (dict(dtype=ep.EP_DTYPE_E4M3, w_scale=FAKE, inn=64, out=128), BAD),      # blocks of 128
    (dict(dtype=ep.EP_DTYPE_E4M3, w_scale=FAKE, inn=128, out=64), BAD),
    (dict(inn=1 << 15, out=1 << 15), TOO_LARGE), (dict(inn=1 << 15, out=1 << 14, act=ep.EP_ACT_SWIGLU), TOO_LARGE),
    (dict(inn=1 << 20, out=8), TOO_LARGE), (dict(inn=8, out=1 << 20), TOO_LARGE),
    (dict(out=2**31 - 8, act=ep.EP_ACT_SWIGLU), TOO_LARGE),
])
def test_products_are_checked_before_the_device(kw, code):
    assert call_product(product(**kw)) == code and ep.last_error() != ""
    assert call_grad(product(**kw)) == code
    assert ep.lib().ep_expert_product_grad_bytes(ctypes.byref(desc()), ctypes.byref(product(**kw))) == 0


def test_other_product_arguments_are_checked_before_the_device():
    lib = ep.lib()
    assert call_product(product(), d=desc(n_experts=3)) == BAD
    assert call_product(product(), x=(FAKE, FAKE)) == BAD                    # scales of bf16 rows
    assert lib.ep_expert_product(ctypes.byref(desc()), ctypes.byref(product()), None, FAKE, None, None, FAKE, None) == BAD
    assert lib.ep_expert_product(ctypes.byref(desc()), None, (ctypes.c_void_p * 2)(FAKE, None), FAKE, None, None, FAKE,
                                 None) == BAD
    big = desc(n_ranks=1, tokens=1 << 21, n_experts=8, topk=8, hidden=8, cap_rows=0)
    assert call_product(product(inn=8, out=8192), d=big) == TOO_LARGE        # more tiles than a launch holds
    assert call_grad(product(inn=8, out=8192), d=big) == TOO_LARGE
    assert call_grad(product(dtype=ep.EP_DTYPE_E4M3, w_scale=FAKE, inn=128, out=128)) == TOO_LARGE
    assert call_grad(product(), pre=FAKE) == BAD                             # no activation, no pre
    assert call_grad(product(act=ep.EP_ACT_SILU)) == BAD
    assert call_grad(product(), dx=None, dw=None, dbias=None) == BAD


def test_product_workspace_holds_dz_and_parts():
    for act, wide in ((ep.EP_ACT_NONE, 0), (ep.EP_ACT_GELU, 32), (ep.EP_ACT_SWIGLU, 64)):
        d, p = desc(), product(act=act)
        w = 64 if act == ep.EP_ACT_SWIGLU else 32
        got = ep.lib().ep_expert_product_grad_bytes(ctypes.byref(d), ctypes.byref(p))
        assert got >= 2 * 2 * 16 * wide + 4 * w * 4                          # dz, a part per expert at least


def test_route_gradients_are_checked_before_the_device():
    lib, d = ep.lib(), ctypes.byref(desc(n_experts=3))
    assert lib.ep_combine_grad(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == BAD
    assert lib.ep_dispatch_grad(d, FAKE, None, FAKE, FAKE, None) == BAD


def test_binding_checks_tensors():
    x, w = torch.zeros(4, 256, dtype=BF), torch.ones(256, dtype=BF)
    with pytest.raises(ValueError, match="weight"):
        ep.rms_norm(x, w[:128], 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="weight"):
        ep.rms_norm(x, w.float(), 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="dtype"):
        ep.rms_norm(x.float(), w.float(), 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="contiguous"):
        ep.rms_norm(x.t(), torch.ones(4, dtype=BF), 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="y holds"):
        ep.rms_norm(x, w, 1e-6, y=torch.empty(3, 256, dtype=BF))
    with pytest.raises(ValueError, match="y has dtype"):
        ep.rms_norm(x, w, 1e-6, y=torch.empty(4, 256))
    with pytest.raises(ValueError, match="scales"):
        ep.rms_norm(x, w, 1e-6, codes=torch.empty(4, 256, dtype=F8), scales=torch.empty(4, 1))
    with pytest.raises(ValueError, match="residual"):
        ep.rms_norm(x, w, 1e-6, residual=x.half(), sum=x, y=x)
    with pytest.raises(ValueError, match="ws holds"):
        ep.rms_norm_grad(x, x, w, 1e-6, torch.empty_like(x), torch.empty(256), torch.empty(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dweight"):
        ep.rms_norm_grad(x, x, w, 1e-6, torch.empty_like(x), torch.empty(255), torch.empty(1 << 16, dtype=torch.uint8))


def test_binding_checks_products():
    w = torch.zeros(4, 32, 64, dtype=BF)
    with pytest.raises(ValueError, match="taken"):
        ep.make_product(w.half())
    with pytest.raises(ValueError, match="taken"):
        ep.make_product(w[0])
    with pytest.raises(ValueError, match="even"):
        ep.make_product(w[:, :31].contiguous(), ep.EP_ACT_SWIGLU)
    with pytest.raises(ValueError, match="contiguous"):
        ep.make_product(w.transpose(1, 2))
    with pytest.raises(ValueError, match="w_scale"):
        ep.make_product(w, w_scale=torch.zeros(4, 1, 1))
    with pytest.raises(ValueError, match="w_scale"):
        ep.make_product(torch.zeros(4, 128, 128, dtype=F8))
    with pytest.raises(ValueError, match="w_scale"):
        ep.make_product(torch.zeros(4, 128, 256, dtype=F8), w_scale=torch.zeros(4, 1, 1))
    with pytest.raises(ValueError, match="bias"):
        ep.make_product(w, bias=torch.zeros(4, 32))
    d, p = desc(), ep.make_product(w)
    x, out = torch.zeros(32, 64, dtype=BF), torch.zeros(32, 32, dtype=BF)
    plan = torch.zeros(ep.plan_bytes(d), dtype=torch.uint8)
    with pytest.raises(ValueError, match="experts"):
        ep.expert_product(desc(n_experts=6), p, [x], plan, out)
    with pytest.raises(ValueError, match="x holds"):
        ep.expert_product(d, p, [x[:31]], plan, out)
    with pytest.raises(ValueError, match="out holds"):
        ep.expert_product(d, p, [x], plan, out[:31])
    with pytest.raises(ValueError, match="residual"):
        ep.expert_product(d, p, [x], plan, out, residual=out.float())
    with pytest.raises(ValueError, match="pre"):
        ep.expert_product(d, p, [x], plan, out, pre=out[:8])
    with pytest.raises(ValueError, match="ws holds"):
        ep.expert_product_grad(d, p, out, x, None, plan, torch.empty(8, dtype=torch.uint8), dx=x)
    ws = torch.empty(ep.expert_product_grad_bytes(d, p), dtype=torch.uint8)
    with pytest.raises(ValueError, match="dbias"):
        ep.expert_product_grad(d, p, out, x, None, plan, ws, dbias=torch.zeros(4, 32, dtype=BF))
    with pytest.raises(ValueError, match="dw holds"):
        ep.expert_product_grad(d, p, out, x, None, plan, ws, dw=w[:3])


def test_binding_checks_route_gradients():
    d = desc()
    y, dout = torch.zeros(32, 64, dtype=BF), torch.zeros(2, 8, 64, dtype=BF)
    w, plan = torch.zeros(2, 8, 2), torch.zeros(ep.plan_bytes(d), dtype=torch.uint8)
    with pytest.raises(ValueError, match="dout holds"):
        ep.combine_grad(d, dout[:1], y, w, plan, y)
    with pytest.raises(ValueError, match="dy holds"):
        ep.combine_grad(d, dout, y, w, plan, y[:8])
    with pytest.raises(ValueError, match="weights"):
        ep.combine_grad(d, dout, y, w.double(), plan, y)
    with pytest.raises(ValueError, match="dx holds"):
        ep.dispatch_grad(d, y, plan, dout[:1])
    with pytest.raises(ValueError, match="add has dtype"):
        ep.dispatch_grad(d, y, plan, dout, add=dout.float())
