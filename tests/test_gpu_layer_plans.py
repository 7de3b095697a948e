"""Plans that do not fit the call they are given to: the products read and write nothing outside their buffers, and
results that do not depend on the plan are right."""
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import BF, guarded

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


def broken(kind, n, local, cap, g):
    """Group offsets that no plan has, int32 [n, local + 1]; their groups together are far more rows than slots."""
    j = torch.arange(local + 1)
    big, small = 2**31 - 1, -2**31
    one = {
        "all or nothing": (j % 2) * cap,
        "descending": cap - cap * j // local,
        "out of range": torch.where(j % 2 == 1, torch.tensor(big), torch.tensor(small)),
        "one past another": (j * 37) % (cap + 1),
        "random": torch.randint(small, big, (local + 1,), generator=g),
        "random rows": torch.randint(0, cap + 1, (local + 1,), generator=g),
    }[kind]
    return one.to(torch.int32).expand(n, -1).contiguous()


KINDS = ["all or nothing", "descending", "out of range", "one past another", "random", "random rows"]
# ranks, tokens, experts, top-k, capacity, columns in, columns out: so that the forward pass takes tiles of 32 x 64, 32 x 128,
# 128 x 128, 256 x 256 and 32 x 128 in turn, dx of 32 x 128 (three times), 128 x 128 and 256 x 256, the capacity being far
# more rows than the slots.
PLANS = [(1, 20, 6, 2, 400, 128, 128), (2, 40, 16, 2, 300, 256, 1280), (1, 900, 4, 2, 2000, 128, 2048),
         (1, 4200, 3, 1, 5000, 256, 2048), (1, 4200, 3, 1, 5000, 4096, 128)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,t,e,r,cap,k,m", PLANS)
def test_product_of_broken_plans(n, t, e, r, cap, k, m, fp8, kind):
    note(f"product broken plan {kind} {fp8} {n} {t} {e} {r} {cap} {k} {m}")
    g = torch.Generator().manual_seed(1)
    d = ep.make_desc(n, t, 8, e, r, cap_rows=cap)
    plan, whole = guarded((ep.plan_bytes(d),), torch.uint8, 7)
    plan.zero_()
    group_offsets(d, plan).copy_(broken(kind, n, e // n, cap, g))
    rows = n * cap
    if fp8:
        x = [torch.zeros(rows, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.ones(rows, k // 128, device="cuda")]
        p = ep.make_product(torch.zeros(e, m, k, dtype=torch.float8_e4m3fn, device="cuda"), ep.EP_ACT_SILU,
                            w_scale=torch.ones(e, m // 128, k // 128, device="cuda"))
    else:
        x = [torch.zeros(rows, k, dtype=BF, device="cuda")]
        p = ep.make_product(torch.zeros(e, m, k, dtype=BF, device="cuda"), ep.EP_ACT_SILU)
    (out, a), (pre, b) = guarded((rows, m), BF), guarded((rows, m), BF)
    ep.expert_product(d, p, x, plan, out, pre=pre)
    torch.cuda.synchronize()
    for f in (a, b, whole):
        f()
    # Every row is some group's product, 0, or was left as it was.
    for o in (out, pre):
        assert ((o == 0) | (o == 7)).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
@pytest.mark.parametrize("n,t,e,r,cap,k,m", PLANS)
def test_product_grad_of_broken_plans(n, t, e, r, cap, k, m, act, kind):
    note(f"product grad broken plan {kind} {act} {n} {t} {e} {r} {cap} {k} {m}")
    g = torch.Generator().manual_seed(2)
    d = ep.make_desc(n, t, 8, e, r, cap_rows=cap)
    plan, whole = guarded((ep.plan_bytes(d),), torch.uint8, 7)
    plan.zero_()
    offsets = broken(kind, n, e // n, cap, g)
    group_offsets(d, plan).copy_(offsets)
    rows, wrows = n * cap, 2 * m if act == ep.EP_ACT_SWIGLU else m
    p = ep.make_product(torch.zeros(e, wrows, k, dtype=BF, device="cuda"), act)
    x, dout = torch.ones(rows, k, dtype=BF, device="cuda"), torch.ones(rows, m, dtype=BF, device="cuda")
    pre = torch.zeros(rows, wrows, dtype=BF, device="cuda") if act != ep.EP_ACT_NONE else None
    (ws, a), (dx, b) = guarded((ep.expert_product_grad_bytes(d, p),), torch.uint8, 9), guarded((rows, k), BF)
    (dw, c), (db, f) = guarded((e, wrows, k), BF), guarded((e, wrows), torch.float32)
    ep.expert_product_grad(d, p, dout, x, pre, plan, ws, dx, dw, db)
    torch.cuda.synchronize()
    for check in (a, b, c, f, whole):
        check()
    assert ((dx == 0) | (dx == 7)).all()
    if act == ep.EP_ACT_NONE:   # x and dout of ones: dw holds each group's rows, cut to its rank's
        off = offsets.long().clamp(0, cap)
        lo, hi = off[:, :-1].flatten(), off[:, 1:].flatten()
        want = (torch.maximum(hi, lo) - lo).to(BF).cuda()
        assert (dw == want[:, None, None]).all()


def test_default_capacity_far_beyond_the_slots():
    """2,048 slots, a capacity for any routing of them: 2^21 rows, of which the experts have one or so each."""
    note("product of a large default capacity")
    n, t, e, r, k, m = 32, 32, 2048, 2, 64, 8192
    d = ep.make_desc(n, t, 8, e, r)
    cap = ep.capacity(d)
    assert n * cap == 1 << 21
    g = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.rand((n * t, e), generator=g, device="cuda").argsort(1)[:, :r].to(torch.int32).view(n, t, r)
    plan = torch.zeros(ep.plan_bytes(d), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.plan(d, idx, plan, status)
    off = group_offsets(d, plan).long()
    assert int(off[:, -1].sum()) == n * t * r and int(status) == 0
    w = torch.empty((e, m, k), dtype=BF, device="cuda").normal_(generator=g)
    x = torch.zeros((n * cap, k), dtype=BF, device="cuda").normal_(generator=g)
    out, dx = torch.empty((n * cap, m), dtype=BF, device="cuda"), torch.empty((n * cap, k), dtype=BF, device="cuda")
    p = ep.make_product(w)
    ep.expert_product(d, p, [x], plan, out)
    # The outputs are the backward pass's dout: 34 GB of it are enough on the card.
    dw, db = torch.empty_like(w), torch.empty((e, m), device="cuda")
    ws = torch.empty(ep.expert_product_grad_bytes(d, p), dtype=torch.uint8, device="cuda")
    ep.expert_product_grad(d, p, out, x, None, plan, ws, dx, dw, db)
    torch.cuda.synchronize()
    had = 0
    for j in list(range(0, e, 97)) + [e - 1]:
        a, b = (int(off[j // (e // n), j % (e // n) + i]) + j // (e // n) * cap for i in (0, 1))
        had += b - a
        x64, w64 = x[a:b].double(), w[j].double()
        z, terms = x64 @ w64.T, x64.abs() @ w64.abs().T
        # Sums of k products in 32 bits, (k + 8) 2^-23 of their terms, then half a step of bf16.
        assert ((out[a:b].double() - z).abs() <= terms * (k + 8) * 2.0**-23 + z.abs() * 2.0**-7.99).all()
        do = out[a:b].double()
        for got, want, terms, count in ((dx[a:b], do @ w64, do.abs() @ w64.abs(), m),
                                        (dw[j], do.T @ x64, do.abs().T @ x64.abs(), b - a)):
            assert ((got.double() - want).abs() <= terms * (count + 8) * 2.0**-23 + want.abs() * 2.0**-7.99).all()
        assert ((db[j].double() - do.sum(0)).abs() <= do.abs().sum(0) * (b - a + 8) * 2.0**-24).all()
    assert had > 10
