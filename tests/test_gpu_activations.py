"""The activations of the experts' products and their slopes at every finite bf16 value, against 64 bits.

A row that is 1 in its first column and 0 elsewhere makes z the first column of the weights, exactly; dbias of a single
row whose gradient is 1 is the 32-bit slope. Tolerances, from the arithmetic: an exponential of a is off by
a (2^-24 + 2^-24 + 2^-26) relative (a's own rounding, that of its product with log2 e, and the constant's) and 2^-23;
a is under 89 where the result is not below 2^-126: under 2^-16.3. Mills' ratio is within 2^-20 and its reciprocal
within 2^-22, the few products and sums that follow within 2^-22: 2^-16 of the terms' absolute values in all. Where an
exponential leaves the floats' range values and slopes come out as 0: under 2^-120 absolute. Outputs are rounded to
bf16: half a step."""
import math

import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, HALF, NAMES, TINY, Dense, check

pytestmark = pytest.mark.gpu
GONE = 2.0**-120


def every():
    """All finite bf16 values, in a number that is a multiple of 8."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    z = bits.to(torch.uint16).view(BF)
    return torch.cat([z[z.isfinite()], torch.zeros(8 - int(z.isfinite().sum()) % 8, dtype=BF)])


def terms_of(z, act):
    """The activation, its slope, and the absolute terms that the slope adds."""
    if act == ep.EP_ACT_GELU:
        below = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        density = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * below, below + z * density, below + (z * density).abs()
    s = torch.where(z < 0, torch.exp(z.clamp(max=0)), 1.0) / (1 + torch.exp(-z.abs()))
    t = torch.where(z > 0, torch.exp(-z.clamp(min=0)), 1.0) / (1 + torch.exp(-z.abs()))   # 1 - s
    return z * s, s + z * s * t, s + (z * s * t).abs()


@pytest.mark.parametrize("act", [ep.EP_ACT_SILU, ep.EP_ACT_GELU, ep.EP_ACT_SWIGLU], ids=NAMES.get)
def test_activation_and_slope_of_every_value(act):
    note(f"activations {NAMES[act]}")
    z = every()
    n = len(z)
    where = Dense(1, 1)
    glu = act == ep.EP_ACT_SWIGLU
    w = torch.zeros(1, 2 * n if glu else n, 8, dtype=BF)
    w[0, :n, 0] = z
    if glu:
        w[0, n:, 0] = 1.0
    p = ep.make_product(w.cuda(), act)
    x = torch.zeros(1, 8, dtype=BF)
    x[0, 0] = 1.0
    out, pre = torch.empty(1, n, dtype=BF, device="cuda"), torch.empty(1, w.shape[1], dtype=BF, device="cuda")
    ep.expert_product(where.desc, p, [x.cuda()], None, out, pre=pre)
    ws = torch.empty(ep.expert_product_grad_bytes(where.desc, p), dtype=torch.uint8, device="cuda")
    db = torch.empty(1, w.shape[1], device="cuda")
    pre[0, :n] = z.cuda()    # denormal values too, whatever the matrix unit makes of them
    ep.expert_product_grad(where.desc, p, torch.ones(1, n, dtype=BF, device="cuda"), x.cuda(), pre, None, ws, dbias=db)
    torch.cuda.synchronize()
    value, slope, terms = terms_of(z.double(), act)
    check(out[0], value, value.abs() * (HALF[BF] + 2.0**-16) + GONE + TINY[BF], "value")
    check(db[0, :n], slope, terms * 2.0**-16 + GONE, "slope")
    if glu:    # the up rows' gradient is the gate's activation
        check(db[0, n:], value, value.abs() * 2.0**-16 + GONE, "up")
