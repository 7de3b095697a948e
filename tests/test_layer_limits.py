"""Sizes that the experts' products take and refuse (no GPU). Rows that a plan can deliver count, not the capacity
that the buffers have for them."""
import ctypes

import pytest

import combine_ep_plan_amd as ep

FAKE = 0x10000
TOO_LARGE = ep.EP_ERR_UNSUPPORTED


def forward(d, p, plan=FAKE):
    return ep.lib().ep_expert_product(ctypes.byref(d), ctypes.byref(p), (ctypes.c_void_p * 2)(FAKE, p.w_scale), plan,
                                      None, None, FAKE, None)


def backward(d, p, plan=FAKE, dx=FAKE, dw=FAKE, dbias=FAKE):
    pre = FAKE if p.act != ep.EP_ACT_NONE else None
    return ep.lib().ep_expert_product_grad(ctypes.byref(d), ctypes.byref(p), FAKE, FAKE, pre, plan, FAKE, dx, dw, dbias,
                                           None)


def product(inn, out, act=ep.EP_ACT_NONE, dtype=ep.EP_DTYPE_BF16):
    return ep.Product(FAKE, FAKE if dtype == ep.EP_DTYPE_E4M3 else None, None, inn, out, act, dtype)


# Ranks, tokens, experts, top-k, each with the default capacity (any routing fits).
@pytest.mark.parametrize("shape", [(8, 4096, 256, 8), (32, 128, 256, 8), (8, 2048, 256, 8), (1, 32768, 256, 8),
                                   (8, 4096, 64, 8), (8, 16384, 64, 8)])
def test_default_capacity_is_not_refused(shape):
    """The worst-case capacity of the prefill and decode workloads and of others: fewer rows are ever delivered."""
    n, t, e, r = shape
    d = ep.make_desc(n, t, 7168, e, r)
    for p in (product(7168, 2048, ep.EP_ACT_SWIGLU), product(2048, 7168), product(7168, 2048, ep.EP_ACT_GELU)):
        assert forward(d, p) != TOO_LARGE
        assert backward(d, p) != TOO_LARGE
    assert forward(d, product(7168, 2048, ep.EP_ACT_SWIGLU, ep.EP_DTYPE_E4M3)) != TOO_LARGE


def test_each_call_has_its_own_limit():
    """2^24 slots of 8 experts: 2^19 + 8 blocks of 32 rows."""
    d = ep.make_desc(1, 1 << 21, 8, 8, 8)
    # Forward: the outputs' columns count, not the inputs'.
    assert forward(d, product(8, 8128)) != TOO_LARGE
    assert forward(d, product(8, 8192)) == TOO_LARGE
    assert forward(d, product(8192, 8)) != TOO_LARGE
    # dx: the inputs' columns; the weights' gradient alone has no such limit.
    assert backward(d, product(8128, 8), dbias=None) != TOO_LARGE
    assert backward(d, product(8192, 8), dbias=None) == TOO_LARGE
    assert backward(d, product(8192, 8), dx=None, dbias=None) != TOO_LARGE
    # The elementwise part, which a bias or an activation needs.
    assert backward(d, product(8, 8192), dx=None) == TOO_LARGE
    assert backward(d, product(8, 8192), dx=None, dbias=None) != TOO_LARGE
    assert backward(d, product(8, 8192, ep.EP_ACT_SILU), dx=None, dbias=None) == TOO_LARGE
    assert backward(d, product(8, 7936, ep.EP_ACT_SILU)) != TOO_LARGE


def test_dense_products_count_their_capacity():
    """Without a plan every row of the capacity is the expert's."""
    d = ep.make_desc(1, 8, 8, 1, 1, cap_rows=1 << 24)
    assert forward(d, product(8, 8192)) != TOO_LARGE                 # eight slots
    assert forward(d, product(8, 8192), plan=None) == ep.EP_ERR_UNSUPPORTED
    assert forward(d, product(8, 8128), plan=None) != TOO_LARGE
