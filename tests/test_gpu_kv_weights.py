"""Small weights beside a large one, as with a first token that takes most of a
row's weight and whose value is near nothing: what the other keys add up to is
the row's output.

The weights meet V in the rows' type. In fp16 they are held 2^7 times as large,
so that half a subnormal step of theirs is 2^-32 of a weight of 1, which is the
largest one's or, where the running maximum lags, less. So with n keys of
|v| <= 1: |out - o| <= (half + 2 e + n 2^-24) A + half |o| + n 2^-32 + 2^-25 (half a
subnormal step of out), with half, e and A as in the other tests of attention."""
import math

import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from kv_ref import attend
from test_gpu_kv_attend import BF, F8, HALF, HF, ints

pytestmark = pytest.mark.gpu
DIM, BT = 64, 16


@pytest.mark.parametrize("rows", [1, 40])               # the waves share the keys, the rows
@pytest.mark.parametrize("dtype,cache", [(HF, HF), (HF, F8), (BF, BF)])
@pytest.mark.parametrize("logit", [15.5, 17.46875, 19.0])
def test_many_small_weights_beside_one(dtype, cache, rows, logit):
    note(f"kv attend {dtype} {cache} rows {rows} logit {logit}")
    # So many sequences and KV heads that most items are held whole by one workgroup.
    seqs, kv, n = 96, 8, 8192
    pool = torch.zeros((n // BT, BT, 2, kv, DIM))
    pool[0, 0, 0, :, 0] = logit
    pool[:, :, 1] = 1.0
    pool[0, 0, 1] = 0.0
    pool = pool.cuda()
    scales = [None, None]
    if cache == F8:
        scales = [torch.full((kv,), logit / 8, device="cuda"), torch.ones(kv, device="cuda")]
        pool[:, :, 0] /= logit / 8                          # 8.0 exactly
    pool = pool.to(cache)
    c = ep.make_kv_cache(pool[:, :, 0], pool[:, :, 1], *scales)
    tables = torch.arange(n // BT, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    q = torch.zeros((seqs * rows, kv, DIM), dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    out, status = torch.empty_like(q), ints([0])
    lse = torch.empty((seqs * rows, kv), device="cuda")
    ws = torch.empty(ep.kv_attend_bytes(c, seqs, 0, seqs * rows, kv, rows), dtype=torch.uint8, device="cuda")
    ep.kv_attend(c, tables, ints([n] * seqs), ints([rows * b for b in range(seqs + 1)]), rows, None, None, q, out,
                 lse, 1.0, ws, status)
    k, v = torch.zeros((n, DIM), dtype=torch.float64), torch.ones((n, DIM), dtype=torch.float64)
    k[0, 0], v[0] = logit if cache == F8 else float(torch.tensor(logit).to(cache)), 0.0
    sees = torch.arange(n) <= torch.arange(n - rows, n)[:, None]
    one = torch.zeros((rows, DIM), dtype=torch.float64)
    one[:, 0] = 1.0
    o, m, a, top, _ = attend(one, k, v, sees, 1.0)
    e = (DIM + 8) * 2.0**-24 * top + 2.0**-20 * (1 + m.abs())
    got_m = lse.view(seqs, rows, kv).double().cpu()
    assert ((got_m - m[:, None]).abs() <= e[:, None]).all()
    half = HALF[dtype]
    tol = (half + 2 * e[:, None] + n * 2.0**-24) * a * 1.01 + half * 1.01 * o.abs() + \
        (n * 2.0**-32 + 2.0**-25 if dtype == HF else 0.0)
    off = (out.view(seqs, rows, kv, DIM).double().cpu() - o[:, None]).abs() - tol[:, None]
    assert off.max() <= 0, (float(off.max()), float(tol.max()), float(o[0, 0]), float(out[0, 0, 0]))
    assert int(status.item()) == 0 and math.isfinite(float(out.float().sum()))


def test_lse_and_shared_keys_under_a_large_weight():
    """The large weight lies in the shared keys, the small ones in a sequence's own, and the other way round."""
    for where in (0, 100):
        seqs, kv, shared, n = 70, 4, 64, 1024
        g = torch.Generator().manual_seed(where)
        pages = shared // BT + seqs * (n - shared) // BT
        pool = (torch.randn((pages, BT, 2, kv, DIM), generator=g) * 0.1).to(HF)
        tables = torch.zeros((seqs, n // BT), dtype=torch.int32)
        tables[:, :shared // BT] = torch.arange(shared // BT)
        tables[:, shared // BT:] = shared // BT + torch.arange(seqs * (n - shared) // BT).view(seqs, -1)
        for b in range(seqs):
            at = int(tables[b, where // BT]), where % BT
            pool[at][0] = 0.0
            pool[at][0, :, 0] = 18.0
            pool[at][1] = 0.0
        dev = pool.cuda()
        c = ep.make_kv_cache(dev[:, :, 0], dev[:, :, 1])
        q = torch.zeros((seqs, kv, DIM), dtype=HF)
        q[:, :, 0] = 1.0
        qd = q.cuda()
        out, lse, status = torch.empty_like(qd), torch.empty((seqs, kv), device="cuda"), ints([0])
        ws = torch.empty(ep.kv_attend_bytes(c, seqs, 1, seqs, kv), dtype=torch.uint8, device="cuda")
        ep.kv_attend(c, tables.cuda(), ints([n] * seqs), None, 1, ints([0, seqs]), ints([shared]), qd, out, lse, 1.0,
                     ws, status)
        out, lse = out.double().cpu(), lse.double().cpu()
        for b in range(0, seqs, 3):
            rows = pool[tables[b].long()].view(n, 2, kv, DIM).double()
            for h in range(kv):
                v = rows[:, 1, h]
                o, m, a, top, p = attend(q[b, h:h + 1].double(), rows[:, 0, h], v,
                                         torch.ones((1, n), dtype=torch.bool), 1.0)
                e = float((DIM + 8) * 2.0**-24 * top + 2.0**-20 * (1 + m.abs()))
                assert abs(float(lse[b, h] - m[0])) <= e
                tol = (2.0**-11 + 2 * e + n * 2.0**-24) * a * 1.01 + 2.0**-11 * 1.01 * o.abs() + \
                    2.0**-32 * float(p.max()) * v.abs().sum(0) + 2.0**-25
                assert ((out[b, h] - o[0]).abs() <= tol[0]).all(), (where, b, h)
        assert int(status.item()) == 0
