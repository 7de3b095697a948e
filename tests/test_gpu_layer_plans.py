"""Plans that do not fit the call they are given to: the products read and write nothing outside their buffers, and
results that do not depend on the plan are right."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF

pytestmark = pytest.mark.gpu


def group_offsets(d, plan):
    """The plan's group offsets, int32 [n_ranks, local experts + 1], as a view of its workspace: behind the counts, the
    send offsets, the slots' places and the receive offsets, each array on a 256-byte boundary."""
    n, e, slots = d.n_ranks, d.n_experts, d.n_ranks * d.tokens * d.topk
    at = sum((4 * m + 255) // 256 * 256 for m in (n * e, n * (e + 1), slots, n * (n + 1)))
    m = n * (e // n + 1)
    return plan[at:at + 4 * m].view(torch.int32).view(n, e // n + 1)


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
def test_no_tokens_and_a_plan_that_was_never_made(act):
    """A step without tokens, buffers with capacity: dw and dbias are zeros whatever the plan's workspace holds."""
    note(f"no tokens, no plan {act}")
    dev, cap, k, m = "cuda", 70, 72, 40
    d = ep.make_desc(2, 0, 8, 4, 2, cap_rows=cap)
    plan = torch.zeros(ep.plan_bytes(d), dtype=torch.uint8, device=dev)
    wrows = 2 * m if act == ep.EP_ACT_SWIGLU else m
    p = ep.make_product(torch.ones(4, wrows, k, dtype=BF, device=dev), act)
    x, dout = (torch.ones(2 * cap, s, dtype=BF, device=dev) for s in (k, m))
    pre = torch.ones(2 * cap, wrows, dtype=BF, device=dev) if act != ep.EP_ACT_NONE else None
    ws = torch.full((ep.expert_product_grad_bytes(d, p),), 63, dtype=torch.uint8, device=dev)
    for offsets in ([0, 30, cap], [5, cap, 2**31 - 1], [-3, 64, 65]):
        group_offsets(d, plan).copy_(torch.tensor([offsets, offsets[::-1]], dtype=torch.int32))
        out = torch.full((2 * cap, m), 7.0, dtype=BF, device=dev)
        ep.expert_product(d, p, [x], plan, out)
        dx = torch.full((2 * cap, k), 7.0, dtype=BF, device=dev)
        dw, db = torch.full((4, wrows, k), 7.0, dtype=BF, device=dev), torch.full((4, wrows), 7.0, device=dev)
        ep.expert_product_grad(d, p, dout, x, pre, plan, ws, dx, dw, db)
        torch.cuda.synchronize()
        assert (out == 7).all() and (dx == 7).all() and (dw == 0).all() and (db == 0).all()
