"""Rotary append on the GPU against the definition in 64 bits.

Tolerance: the rotated value x c - y s is formed in 32 bits. The angle is
exact to 2^-24 of a half turn (its last step rounds the reduced angle), sine
and cosine to 2 steps, mscale, each product and the sum to half a step: under
2^-20 (|x| + |y|) mscale. Then it is rounded once: half a step of the type
relative to the value, or half a subnormal step. An e4m3 value is divided by
its scale first (half a 32-bit step more, within the same 2^-20)."""
import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from kv_ref import BAD_PAGE, rotate, rows_of

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: (2.0**-8, 2.0**-134), torch.float16: (2.0**-11, 2.0**-25),
        torch.float8_e4m3fn: (2.0**-4, 2.0**-10)}


def near(got, want, size, dtype):
    rel, sub = HALF[dtype]
    slack = 2.0**-20 * size
    tol = slack + rel * (want.abs() + slack) + sub
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(got.double()).any()
    assert off.max() <= 0, (float(off.max()), int(off.argmax()))


def pair_size(x, rot, interleaved, mscale):
    """|x| + |y| of each element's pair, |x| of an element that does not turn."""
    a = x.abs()
    out = a.clone()
    if rot:
        r = a[..., :rot]
        other = r.unflatten(-1, (rot // 2, 2)).flip(-1).flatten(-2) if interleaved else \
            r.roll(rot // 2, -1)
        out[..., :rot] = (r + other) * mscale
    return out


def run(dtype, cache, heads, kv, dim, rot, layout, mscale, new, lens, bt, *, in_place=False,
        head_major=False, queries=True, extra_rows=0, no_off=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    seqs, t = len(new), sum(new) + extra_rows
    need = [max(1, -(-n // bt)) for n in lens]
    total = sum(need) + 2
    ids = torch.randperm(total, generator=g).to(torch.int32)
    tables = torch.full((seqs, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    qkv = torch.randn((t, heads + 2 * kv, dim), generator=g).to(dtype)
    dev = qkv.cuda()
    q, k, v = dev.split([heads, kv, kv], 1)
    shape = (total, 2, kv, bt, dim) if head_major else (total, bt, 2, kv, dim)
    pool = torch.randn(shape, generator=g).to(cache)
    before = pool.clone()
    pool = pool.cuda()
    kc, vc = (pool[:, i].transpose(1, 2) if head_major else pool[:, :, i] for i in (0, 1))
    scales = [None, None]
    if cache == torch.float8_e4m3fn:
        scales = [(torch.rand(kv, generator=g) * 0.02 + 0.002) for _ in range(2)]
    c = ep.make_kv_cache(kc, vc, *(None if s is None else s.cuda() for s in scales))
    inv, _ = ep.rope_freqs(rot, 10000.0) if rot else (np.zeros(0, np.float32), 1.0)
    inv = torch.from_numpy(inv)
    rope = ep.make_rope(inv.cuda(), rot, layout, mscale) if rot else None
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = q if in_place else torch.full_like(q, 7.0)
    q_off = None if no_off else torch.tensor(off, dtype=torch.int32, device="cuda")
    ep.kv_append(c, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), q_off,
                 q if queries else None, k, v, q_out if queries else None, rope, status)
    where = rows_of(lens, off)
    pos = torch.tensor([p for _, p in where])
    n = len(where)
    x = qkv[:n].double()
    turned = rotate(x, pos, inv, rot, layout == ep.EP_ROPE_INTERLEAVED, mscale) if rot else x
    turned[:, heads + kv:] = x[:, heads + kv:]
    size = pair_size(x, rot, layout == ep.EP_ROPE_INTERLEAVED, mscale)
    size[:, heads + kv:] = x[:, heads + kv:].abs()
    if queries:
        near(q_out.cpu()[:n], turned[:, :heads], size[:, :heads], dtype)
        rest = q_out.cpu()[n:]
        assert torch.equal(rest, qkv[n:, :heads] if in_place else torch.full_like(rest, 7.0))
    assert torch.equal(k.cpu(), qkv[:, heads:heads + kv]) and torch.equal(v.cpu(), qkv[:, heads + kv:])
    # Every slot that no token owns keeps its bytes; the others hold the rows.
    want = before.view(torch.uint8).clone()
    after = pool.cpu()
    for side, lo in ((0, heads), (1, heads + kv)):
        got = after[:, side].transpose(1, 2) if head_major else after[:, :, side]
        ref = want[:, side].transpose(1, 2) if head_major else want[:, :, side]
        for i, (b, p) in enumerate(where):
            if p < 0 or p // bt >= tables.shape[1] or not 0 <= tables[b, p // bt] < total:
                continue
            page, slot = int(tables[b, p // bt]), p % bt
            y, s = turned[i, lo:lo + kv], size[i, lo:lo + kv]
            if scales[side] is not None:
                w = scales[side].double()[:, None]
                y, s = (y / w), s / w
                s = torch.where(y.abs() > 448, torch.zeros_like(s), s)
                y = y.clamp(-448, 448)
            near(got[page, slot], y, s, cache)
            ref[page, slot] = got[page, slot].contiguous().view(torch.uint8)
    assert torch.equal(after.view(torch.uint8), want)
    return int(status.item())


BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
CASES = [
    # dtype, cache, heads, kv, dim, rot, layout, mscale, new, lens, page_tokens
    (BF, BF, 8, 2, 128, 128, 0, 1.0, [1, 1, 1], [1, 17, 500], 16),
    (BF, BF, 5, 1, 128, 128, 1, 1.2, [3, 1, 6], [3, 131072, 9], 16),
    (HF, HF, 4, 4, 64, 32, 0, 1.0, [7, 0, 2], [20, 5, 2], 1),
    (HF, HF, 3, 1, 80, 24, 1, 1.0, [5], [9], 7),
    (BF, F8, 4, 2, 128, 64, 1, 1.0, [9, 4], [40, 4], 16),
    (HF, F8, 2, 1, 256, 256, 0, 1.1, [2, 2], [2, 1000003], 64),
    (BF, BF, 2, 1, 8, 2, 0, 1.0, [4, 1], [4, 1], 3),         # pairs that fill no chunk
    (BF, F8, 3, 1, 16, 6, 1, 1.0, [5, 2], [5, 3], 2),
    (BF, BF, 6, 2, 96, 94, 0, 1.0, [3, 3], [100, 3], 5),
    (HF, HF, 2, 2, 96, 0, 0, 1.0, [3, 3], [8, 3], 5),        # no rotation
    (BF, BF, 2, 1, 128, 128, 0, 1.0, [1500, 900], [1500, 2000], 16),   # several tokens a block
]


# Many sequences to a block of tokens, more empty ones in a row than a wave has lanes, long ones.
MANY = [1] * 100 + [0] * 90 + [2900] + [0] * 70 + [5, 0, 2600, 2700, 0]
CASES.append((BF, BF, 1, 1, 16, 16, 1, 1.0, MANY, MANY, 16))


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append_matches_64_bits(case):
    note(f"kv append {case}")
    assert run(*case) == 0


def test_in_place_and_other_layouts():
    assert run(*CASES[0], in_place=True) == 0
    assert run(*CASES[3], in_place=True, extra_rows=3) == 0
    assert run(*CASES[4], head_major=True) == 0
    assert run(*CASES[1], queries=False, extra_rows=2) == 0
    assert run(BF, BF, 3, 1, 64, 64, 0, 1.0, [1] * 5, [4, 9, 1, 33, 70], 16, no_off=True) == 0


def test_positions_without_a_slot_are_skipped_and_flagged():
    """A length shorter than the new tokens: the first ones have no position of their own."""
    assert run(BF, BF, 2, 1, 64, 64, 0, 1.0, [4, 2], [2, 9], 4) == BAD_PAGE


def test_bad_pages_are_skipped_and_flagged():
    cache = torch.zeros((4, 4, 1, 64), dtype=BF, device="cuda")
    c = ep.make_kv_cache(cache, cache.clone())
    x = torch.ones((3, 1, 64), dtype=BF, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = ints([0])
    ep.kv_append(c, ints([[4], [-1], [2]]), ints([1, 1, 99]), None, None, x, x, None, None, status)
    assert status.item() == BAD_PAGE and not cache.any()


def test_nan_and_infinity_keep_their_place():
    inf = float("inf")
    for cache in (BF, F8):
        x = torch.zeros((1, 1, 32), dtype=BF, device="cuda")
        x[0, 0, :4] = torch.tensor([inf, -inf, float("nan"), 1e30], dtype=BF)
        pool = torch.zeros((2, 1, 1, 1, 32), dtype=cache, device="cuda")
        one = torch.ones(1, device="cuda") if cache == F8 else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        zero = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        c = ep.make_kv_cache(pool[0], pool[1], one, one)
        ep.kv_append(c, zero, zero[0] + 1, None, None, x, x, None, None, status)
        got = pool.float().cpu()[:, 0, 0, 0]
        top = 448.0 if cache == F8 else inf
        for row in got:
            assert row[0] == top and row[1] == -top and torch.isnan(row[2]) and not row[4:].any()
            assert row[3] == (448.0 if cache == F8 else torch.tensor(1e30, dtype=BF).float())


@pytest.mark.parametrize("scaling,rot", [(ep.EP_ROPE_LINEAR, 128), (ep.EP_ROPE_NTK, 64),
                                         (ep.EP_ROPE_YARN, 128)])
def test_far_positions_keep_their_angle(scaling, rot):
    """Position 10^6 under the scalings: a 32-bit angle would be off by up to 2^-5 radians."""
    inv, mscale = ep.rope_freqs(rot, 500000.0, scaling, 16.0, 8192)
    pos = 1000000
    pool = torch.zeros((1, 1, 1, 128), dtype=HF, device="cuda")
    c = ep.make_kv_cache(pool, pool.clone())
    x = torch.randn((1, 1, 128), generator=torch.Generator().manual_seed(1)).to(HF)
    zero = torch.zeros((1, pos + 1), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(x, device="cuda")
    ep.kv_append(c, zero, zero[0, :1] + pos + 1, None, x.cuda(), x.cuda(), x.cuda(), q_out,
                 ep.make_rope(torch.from_numpy(inv).cuda(), rot, ep.EP_ROPE_HALF, mscale), status)
    want = rotate(x.double(), torch.tensor([pos]), torch.from_numpy(inv), rot, False, mscale)
    near(q_out.cpu(), want, pair_size(x.double(), rot, False, mscale), HF)
    near(pool.cpu()[0], want, pair_size(x.double(), rot, False, mscale), HF)
    assert status.item() == 0


def test_rotation_keeps_relative_positions():
    """<R(i) q, R(j) k> depends on i - j alone (the property the formula is for)."""
    inv = torch.from_numpy(ep.rope_freqs(64)[0]).cuda()
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn((1, 1, 64), generator=g).to(HF).cuda() for _ in range(2))
    dots = []
    for shift in (0, 5, 777):
        out = []
        for x, pos in ((q, 40 + shift), (k, 17 + shift)):
            pool = torch.zeros((1, 1024, 1, 64), dtype=HF, device="cuda")
            zero = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            c = ep.make_kv_cache(pool, pool.clone())
            ep.kv_append(c, zero, zero[0] + pos + 1, None, None, x, x, None,
                         ep.make_rope(inv, 64), st)
            out.append(pool[0, pos, 0].double())
        dots.append(float(out[0] @ out[1]))
    # Each rotated value is off by half a step of fp16: 2^-11 of sum |q||k| for either side.
    tol = 2 * 2.0**-11 * 1.1 * float(q.double().norm() * k.double().norm())
    assert max(dots) - min(dots) <= 2 * tol
