"""Attention over pages on the GPU against the definition in 64 bits.

Tolerances, from the arithmetic. Scores are 32-bit sums of exact products of
16-bit values: off by at most (D + 8) 2^-24 S, S = max scale sum |q||k|, and
the exponential and the running rescales add under 2^-20 relative. So lse is
off by e = (D + 8) 2^-24 S + 2^-20 (1 + |lse|) and every weight by e relative
to itself, twice (numerator and sum). Weights may be rounded to the rows' type
before they meet V: half a step of it, relative (an fp16 weight under its
normal range: half a subnormal step of weights whose maximum is 1). The sums
over n keys are 32-bit: n 2^-24. With A = sum p |v|: |out - o| <= (half + 2 e +
n 2^-24) A + half (|o|) + the subnormal terms."""
import random

import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from kv_ref import BAD_PAGE, attend

pytestmark = pytest.mark.gpu
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
HALF = {BF: 2.0**-8, HF: 2.0**-11}
TINY = {BF: 0.0, HF: 2.0**-25}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Sequences over a pool whose unused slots hold NaN, in groups that share leading tokens."""

    def __init__(self, dtype, cache, heads, kv, dim, bt, lens, new, groups=(), shared=(), *, seed=0,
                 head_major=False, layers=1, spread=1.0, extra_rows=0, packed=False):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.cache, self.heads, self.kv, self.dim, self.bt = dtype, cache, heads, kv, dim, bt
        self.lens, self.new, self.scale = list(lens), list(new), dim ** -0.5
        self.groups, self.shared = list(groups), list(shared)
        seqs = len(lens)
        need = [-(-max(n, 0) // bt) for n in lens]
        total = sum(need) + 3
        ids = torch.randperm(total, generator=g).tolist()
        self.table = [[-1] * (max(need) + 1) for _ in range(seqs)]
        lead = {}  # sequence: (first of its group, whole pages it shares)
        for j, sh in enumerate(self.shared):
            for b in range(self.groups[j], self.groups[j + 1]):
                lead[b] = (self.groups[j], -(-sh // bt))
        for b in range(seqs):
            first, n = lead.get(b, (b, 0))
            for i in range(need[b]):
                self.table[b][i] = self.table[first][i] if b != first and i < min(n, need[first]) else ids.pop()
        shape = (total, layers, 2, kv, bt, dim) if head_major else (total, bt, layers, 2, kv, dim)
        pool = torch.full(shape, float("nan"))
        layer = layers - 1
        self.k32, self.v32 = (pool[:, layer, i].transpose(1, 2) if head_major else pool[:, :, layer, i]
                              for i in (0, 1))
        self.scales = [None, None]
        if cache == F8:
            self.scales = [torch.rand(kv, generator=g) * 0.02 + 0.01 for _ in range(2)]
        for b in range(seqs):
            for t in range(max(lens[b], 0)):
                at = self.table[b][t // bt], t % bt
                if torch.isnan(self.k32[at]).any():
                    for x, s in ((self.k32, self.scales[0]), (self.v32, self.scales[1])):
                        r = torch.randn((kv, dim), generator=g) * spread
                        x[at] = r if s is None else (r / s[:, None]).clamp(-448, 448)
        self.pool = pool.to(cache)
        self.t = sum(new) + extra_rows
        wide = torch.randn((self.t, heads + 2 * kv, dim), generator=g).to(dtype)
        self.q = (wide if packed else wide[:, :heads].contiguous())[:, :heads]
        self.head_major, self.layer = head_major, layer
        self.off = [0]
        for n in new:
            self.off.append(self.off[-1] + n)

    def views(self, pool):
        return [pool[:, self.layer, i].transpose(1, 2) if self.head_major else pool[:, :, self.layer, i]
                for i in (0, 1)]

    def device(self):
        """Everything a call takes, on the GPU."""
        d = type("D", (), {})()
        d.pool = self.pool.cuda()
        d.cache = ep.make_kv_cache(*self.views(d.pool), *(None if s is None else s.cuda() for s in self.scales))
        wide = torch.zeros((self.t, self.q.stride(0) // self.dim, self.dim), dtype=self.dtype)
        wide[:, :self.heads] = self.q
        d.q = wide.cuda()[:, :self.heads]
        d.out = torch.full((self.t, self.heads, self.dim), 3.0, dtype=self.dtype, device="cuda")
        d.lse = torch.full((self.t, self.heads), 3.0, device="cuda")
        d.tables, d.lens, d.q_off = ints(self.table), ints(self.lens), ints(self.off)
        d.group_off = ints(self.groups) if self.shared else None
        d.shared = ints(self.shared) if self.shared else None
        d.most = max(1, max(self.new))
        d.status = ints([0])
        d.ws = torch.full((ep.kv_attend_bytes(d.cache, len(self.lens), len(self.shared), self.t,
                                              self.heads, d.most),), 0xFF, dtype=torch.uint8,
                          device="cuda")
        return d

    def call(self, d, **kw):
        a = dict(q_off=d.q_off, most=d.most, lse=d.lse, ws=d.ws, out=d.out)
        a.update(kw)
        ep.kv_attend(d.cache, d.tables, d.lens, a["q_off"], a["most"], d.group_off, d.shared, d.q,
                     a["out"], a["lse"], self.scale, a["ws"], d.status)

    def check(self, out, lse, sees=None, rows=None):
        """out and lse (host) against 64 bits. sees(b, pos, t): whether a row sees key t."""
        kc, vc = self.views(self.pool)
        share, half = self.heads // self.kv, HALF[self.dtype]
        for b, (lo, hi) in enumerate(zip(self.off, self.off[1:])):
            n = max(self.lens[b], 0)
            if hi == lo:
                continue
            pages = [self.table[b][t // self.bt] for t in range(n)]
            good = torch.tensor([0 <= p < len(kc) for p in pages], dtype=torch.bool)
            page = torch.tensor([p if 0 <= p < len(kc) else 0 for p in pages], dtype=torch.long)
            slot = torch.arange(n) % self.bt
            k, v = (x.view(torch.uint8)[page, slot].view(x.dtype).double() for x in (kc, vc))
            if self.scales[0] is not None:
                k, v = k * self.scales[0].double()[:, None], v * self.scales[1].double()[:, None]
            pos = torch.arange(self.lens[b] - (hi - lo), self.lens[b])[:, None]
            see = (torch.arange(n) <= pos) & good
            for h in range(self.heads):
                kh, vh = k[:, h // share], v[:, h // share]
                # Keys that no row sees may hold anything.
                o, m, a, top, p = attend(self.q[lo:hi, h].double(), torch.where(see.any(0)[:, None], kh, 0),
                                         torch.where(see.any(0)[:, None], vh, 0), see, self.scale)
                fine = see.any(1)
                gl, go = lse[lo:hi, h].double(), out[lo:hi, h].double()
                assert torch.equal(gl[~fine], m[~fine]) and not go[~fine].any()
                e = ((self.dim + 8) * 2.0**-24 * top + 2.0**-20 * (1 + m.abs()))[fine]
                assert ((gl[fine] - m[fine]).abs() <= e).all(), (b, h, float((gl[fine] - m[fine]).abs().max()))
                if not fine.any():
                    continue
                biggest = p[fine].amax(1, keepdim=True)
                tiny = TINY[self.dtype] * (biggest * vh[see.any(0)].abs().sum(0) + 1)
                tol = (half + 2 * e[:, None] + n * 2.0**-24) * a[fine] * 1.01 + half * 1.01 * o[fine].abs() + tiny + 1e-37
                off = (go[fine] - o[fine]).abs() - tol
                assert off.max() <= 0, (b, h, float(off.max()), float(tol.min()))

    def test(self, status=0, **kw):
        d = self.device()
        self.call(d, **kw)
        out, lse = d.out.cpu(), d.lse.cpu()
        self.check(out, lse)
        assert (out[self.off[-1]:] == 3).all() and (lse[self.off[-1]:] == 3).all()
        assert int(d.status.item()) == status
        return d


CASES = {
    "one_token": dict(a=(BF, BF, 1, 1, 64, 16, [1], [1])),
    "one_key_many_heads": dict(a=(HF, HF, 40, 8, 128, 1, [1, 2], [1, 1])),
    "ragged": dict(a=(BF, BF, 8, 2, 128, 16, [1, 17, 300, 128, 129, 513], [1] * 6)),
    "more_new": dict(a=(BF, BF, 6, 2, 64, 7, [5, 40, 200, 9], [5, 3, 8, 0])),
    "prompt": dict(a=(HF, HF, 4, 2, 128, 16, [150, 333, 64], [150, 97, 1])),
    "prompt_wide_group": dict(a=(BF, BF, 16, 1, 64, 5, [70, 260], [70, 31])),
    "dim_80": dict(a=(BF, BF, 3, 1, 80, 3, [77, 140], [2, 1])),
    "dim_256": dict(a=(HF, HF, 4, 2, 256, 16, [100, 190, 31], [3, 1, 31])),
    "dim_8": dict(a=(BF, BF, 2, 2, 8, 16, [33, 200], [1, 4])),
    "e4m3": dict(a=(BF, F8, 10, 2, 128, 16, [90, 400, 3], [1, 2, 3])),
    "e4m3_fp16": dict(a=(HF, F8, 4, 4, 64, 1, [65, 129], [4, 1])),
    "e4m3_dim_48": dict(a=(HF, F8, 4, 1, 48, 64, [65, 1029], [40, 1])),
    "group": dict(a=(BF, BF, 8, 2, 128, 16, [530, 600, 513, 700], [1, 1, 1, 1], [0, 4], [512])),
    "groups": dict(a=(HF, HF, 5, 1, 64, 4, [100, 90, 70, 64, 33, 200, 210, 190], [2, 1, 3, 1, 1, 1, 0, 2],
                      [0, 3, 5, 8], [64, 32, 188])),
    "group_of_some": dict(a=(BF, BF, 4, 1, 128, 16, [40, 300, 290, 55], [1, 1, 2, 1], [1, 3], [256])),
    "group_past_lens": dict(a=(BF, BF, 4, 1, 64, 4, [40, 20, 38], [1, 2, 5], [0, 3], [37])),
    "group_prompt": dict(a=(BF, BF, 8, 2, 128, 16, [400, 350, 420], [70, 30, 100], [0, 3], [320])),
    "group_many_rows": dict(a=(BF, F8, 16, 2, 128, 16, [200 + i for i in range(20)], [1] * 20, [0, 20], [192])),
    "empty_groups": dict(a=(HF, HF, 4, 2, 64, 8, [30, 40], [1, 1], [0, 0, 2, 2], [16, 24, 8])),
    "one_long": dict(a=(BF, BF, 4, 1, 128, 16, [9000], [1])),
    "long_mix": dict(a=(HF, F8, 8, 4, 128, 16, [1, 4000, 2, 700, 1, 130], [1, 1, 2, 65, 1, 1])),
    "empty_sequences": dict(a=(BF, BF, 4, 2, 64, 4, [0, 5, 0, 3], [0, 1, 0, 1])),
    "peaked": dict(a=(BF, BF, 4, 2, 128, 16, [600, 90], [1, 20]), spread=20.0),
    "head_major": dict(a=(BF, BF, 8, 2, 64, 16, [100, 210], [1, 3], [0, 2], [96]), head_major=True),
    "layers": dict(a=(HF, HF, 4, 1, 128, 16, [100, 210], [1, 3]), layers=3, packed=True),
    "rows_behind": dict(a=(BF, BF, 4, 2, 128, 16, [100, 64], [2, 33]), extra_rows=5),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attend_matches_64_bits(name):
    note(f"kv attend {name}")
    kw = dict(CASES[name])
    Case(*kw.pop("a"), **kw).test()


def test_lengths_below_the_new_tokens_leave_empty_rows():
    c = Case(BF, BF, 4, 2, 64, 4, [2, 0, 9], [4, 3, 1])
    c.test()


def test_no_lse_and_no_offsets():
    c = Case(BF, BF, 4, 2, 64, 16, [20, 31, 200], [1, 1, 1])
    d = c.device()
    c.call(d, q_off=None, lse=None)
    want = c.device()
    c.call(want)
    c.check(d.out.cpu(), want.lse.cpu())
    assert (d.lse == 3).all()


def test_bad_pages_are_not_attended_to():
    c = Case(HF, HF, 4, 2, 64, 4, [40, 9, 300], [1, 2, 1])
    c.table[0][3], c.table[2][70], c.table[1][0] = -1, 1 << 30, len(c.pool)
    c.test(status=BAD_PAGE)


def test_tables_too_short_for_a_length():
    c = Case(HF, HF, 4, 2, 64, 4, [40, 9], [1, 1])
    d = c.device()
    d.lens = ints([40 + 4 * 2, 9])                     # the row ends 4 tokens before the length
    c.call(d)
    assert int(d.status.item()) == BAD_PAGE
    torch.cuda.synchronize()


def test_new_tokens_past_max_new_are_skipped():
    c = Case(BF, BF, 4, 2, 64, 4, [40, 9], [5, 2])
    d = c.device()
    c.call(d, most=3)
    assert int(d.status.item()) == BAD_PAGE
    out = d.out.cpu()
    assert (out[3:5] == 3).all() and not (out[:3] == 3).any() and not (out[5:] == 3).any()


def test_masked_keys_may_hold_anything():
    """A later new token of the same sequence is infinite or NaN: earlier rows do not see it."""
    for bad in (float("inf"), float("nan")):
        c = Case(BF, BF, 4, 2, 64, 16, [70, 200], [4, 40])
        for b, t in ((0, 69), (1, 190)):
            at = c.table[b][t // 16], t % 16
            for x in c.views(c.pool):
                x[at] = bad
        d = c.device()
        c.call(d)
        got, lse = d.out.cpu(), d.lse.cpu()
        clean = Case(BF, BF, 4, 2, 64, 16, [70, 200], [4, 40])
        keep = [0, 1, 2] + list(range(4, 4 + 30))     # rows before the bad key
        e = clean.device()
        clean.call(e)
        assert torch.equal(got[keep], e.out.cpu()[keep]) and torch.equal(lse[keep], e.lse.cpu()[keep])
        assert torch.isnan(got[[3] + list(range(34, 44))]).all()


def test_nan_queries_and_keys_reach_their_rows_and_no_others():
    """A row whose query is NaN, or that sees a NaN key, is NaN, however many pieces its keys are cut
    into; the others are as without it."""
    for lens, new in (([3000, 40], [1, 1]), ([300, 700], [2, 40])):
        c = Case(BF, BF, 4, 2, 64, 16, lens, new)
        d = c.device()
        c.call(d)
        out, lse = d.out.cpu(), d.lse.cpu()
        d.q[0, 1] = float("nan")
        c.call(d)
        bad = torch.zeros(out.shape[:2], dtype=torch.bool)
        bad[0, 1] = True
        assert torch.isnan(d.out.cpu()[bad]).all() and torch.isnan(d.lse.cpu()[bad]).all()
        assert torch.equal(d.out.cpu()[~bad], out[~bad]) and torch.equal(d.lse.cpu()[~bad], lse[~bad])
        e = c.device()
        c.views(e.pool)[0][c.table[1][1], 5, 0] = float("nan")   # key 21 of sequence 1, KV head 0
        c.call(e)
        bad = torch.zeros(out.shape[:2], dtype=torch.bool)
        bad[new[0]:, :2] = True
        assert torch.isnan(e.out.cpu()[bad]).all() and torch.isnan(e.lse.cpu()[bad]).all()
        assert torch.equal(e.out.cpu()[~bad], out[~bad]) and torch.equal(e.lse.cpu()[~bad], lse[~bad])


def test_results_do_not_depend_on_the_run():
    c = Case(BF, BF, 8, 2, 128, 16, [530, 600, 513, 700], [1, 9, 1, 1], [0, 4], [512])
    d = c.device()
    c.call(d)
    out, lse = d.out.clone(), d.lse.clone()
    for i in range(5):
        d.ws.random_(0, 256)
        d.out.fill_(9)
        c.call(d)
        assert torch.equal(d.out, out) and torch.equal(d.lse, lse), i


def test_two_streams_and_graph_replay():
    one = Case(BF, BF, 8, 2, 128, 16, [530, 600, 513], [1, 1, 1], [0, 3], [512], seed=1)
    two = Case(HF, HF, 4, 4, 64, 8, [230, 90], [30, 2], seed=2)
    a, b = one.device(), two.device()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, d, s in ((one, a, streams[0]), (two, b, streams[1])):
            with torch.cuda.stream(s):
                c.call(d)
    torch.cuda.synchronize()
    one.check(a.out.cpu(), a.lse.cpu())
    two.check(b.out.cpu(), b.lse.cpu())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.call(a)
    for i in range(4):
        a.out.fill_(3)
        a.lse.fill_(3)
        a.lens.copy_(ints([530 - i, 600, 513 + 2 * i]))   # lengths change between replays
        one.lens = [530 - i, 600, 513 + 2 * i]
        if one.lens[2] > 528:
            break
        for t in range(513, one.lens[2]):
            at = one.table[2][t // 16], t % 16
            for x, y in zip(one.views(one.pool), one.views(a.pool)):
                x[at] = 0.5
                y[at] = 0.5
        graph.replay()
        torch.cuda.synchronize()
        one.check(a.out.cpu(), a.lse.cpu())


def test_keys_past_32_bit_offsets():
    """Two pages 5 GiB apart in bytes."""
    stride = (5 << 30) // 2
    pool = torch.zeros(stride + 16 * 128, dtype=BF, device="cuda")
    view = pool.as_strided((2, 16, 1, 128), (stride, 128, 128, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    view.copy_(torch.randn((2, 16, 1, 128), device="cuda", generator=g))
    v = pool.as_strided((2, 16, 1, 128), (stride, 128, 128, 1))
    cache = ep.make_kv_cache(view, v)
    q = torch.randn((1, 1, 128), device="cuda", generator=g).to(BF)
    out, status = torch.empty_like(q), ints([0])
    ws = torch.empty(ep.kv_attend_bytes(cache, 1, 0, 1, 1), dtype=torch.uint8, device="cuda")
    ep.kv_attend(cache, ints([[1, 0]]), ints([30]), None, 1, None, None, q, out, None, 0.25, ws, status)
    x = torch.cat([view[1, :, 0], view[0, :14, 0]]).double().cpu()
    o, _, a, top, _ = attend(q[0].double().cpu(), x, x, torch.ones((1, 30), dtype=torch.bool), 0.25)
    tol = (2.0**-8 + 2 * (136 * 2.0**-24 * float(top.max()) + 2.0**-19)) * a + 2.0**-8 * o.abs()
    assert ((out[0].double().cpu() - o).abs() <= tol).all() and status.item() == 0
    del pool, view, v


def test_a_step_after_a_push_and_a_fork():
    """Push a prompt into a decoder's pool, fork it, then decode: extend, append, attend with the
    prompt as shared prefix, free, compact. Every step against one sequence at a time in 64 bits."""
    rng = random.Random(5)
    kv, heads, dim, bt, layers, prompt, pages = 2, 6, 64, 16, 2, 83, 64
    token_bytes = layers * 2 * kv * dim * 2
    g = torch.Generator().manual_seed(9)
    src = torch.randn((1, pages * bt, token_bytes // 2), generator=g).to(BF).cuda()
    pool = torch.full((1, pages, bt * token_bytes // 2), float("nan"), dtype=BF, device="cuda")
    status, notify = ints([0]), ints([0])
    tables = torch.full((4, 12), -1, dtype=torch.int32, device="cuda")
    lens, refs = ints([0] * 4), ints([0] * pages)
    state = ep.make_kv_pages(tables, lens, refs, pool, bt)
    ws = torch.empty(ep.kv_pages_bytes(state, 8), dtype=torch.uint8, device="cuda")
    busy = ints([3])
    ep.kv_extend(state, busy, ints([40]), ws, status)            # pages in front of the prompt's
    ep.kv_extend(state, ints([0]), ints([prompt]), ws, status)
    n = -(-prompt // bt)
    src_blocks = rng.sample(range(pages), n)
    reg = ep.kv_plan(prompt, token_bytes, bt, src_blocks, bt, tables[0, :n].tolist())
    total = int(reg[:, 2].sum())
    ep.kv_push(1, torch.from_numpy(reg).cuda(), len(reg), total, src, src.numel() * 2, pool,
               pool.numel() * 2, notify, status)
    ep.kv_fork(state, ints([0, 0]), ints([1, 2]), ws, status)
    ep.kv_free(state, busy, ws, status)
    ep.kv_compact(state, ws, status)
    kept = prompt // bt * bt
    view = pool.view(pages, bt, layers, 2, kv, dim)
    inv = torch.from_numpy(ep.rope_freqs(dim)[0]).cuda()
    rope = ep.make_rope(inv, dim)
    caches = [ep.make_kv_cache(view[:, :, i, 0], view[:, :, i, 1]) for i in range(layers)]
    attend_ws = torch.empty(ep.kv_attend_bytes(caches[0], 3, 1, 3, heads), dtype=torch.uint8, device="cuda")
    history = [[[], []] for _ in range(3)]                       # per sample: the k, v rows of layer 1
    packed = src.view(pages, bt, layers, 2, kv, dim).cpu()
    for t in range(prompt):
        row = packed[src_blocks[t // bt], t % bt, 1]
        for h in history:
            h[0].append(row[0].double())
            h[1].append(row[1].double())
    for step in range(20):
        ep.kv_extend(state, ints([0, 1, 2]), ints([1, 1, 1]), ws, status)
        for i, cache in enumerate(caches):
            q, k, v = (torch.randn((3, m, dim), generator=g).to(BF).cuda() for m in (heads, kv, kv))
            out, lse = torch.empty_like(q), torch.empty((3, heads), device="cuda")
            ep.kv_append(cache, tables[:3], lens[:3], None, q, k, v, q, rope, status)
            ep.kv_attend(cache, tables[:3], lens[:3], None, 1, ints([0, 3]), ints([kept]), q, out, lse, 0.125,
                         attend_ws, status)
            if i != 1:
                continue
            for b in range(3):
                page, slot = int(tables[b, (prompt + step) // bt]), (prompt + step) % bt
                history[b][0].append(view[page, slot, 1, 0].cpu().double())
                history[b][1].append(view[page, slot, 1, 1].cpu().double())
                for h in range(heads):
                    kk, vv = (torch.stack(x)[:, h // 3] for x in history[b])
                    see = torch.ones((1, len(kk)), dtype=torch.bool)
                    o, m, a, top, _ = attend(q[b, h:h + 1].cpu().double(), kk, vv, see, 0.125)
                    e = 72 * 2.0**-24 * float(top) + 2.0**-20 * (1 + float(m.abs()))
                    assert abs(float(lse[b, h]) - float(m)) <= e
                    tol = (2.0**-8 + 2 * e + 2.0**-16) * a + 2.0**-8 * 1.01 * o.abs()
                    assert ((out[b, h].cpu().double() - o[0]).abs() <= tol[0]).all(), (step, b, h)
    assert status.item() == 0 and notify.item() == 1
    # The samples share the prompt's whole pages and nothing else.
    rows = tables[:3].cpu()
    assert (rows[:, :kept // bt] == rows[0, :kept // bt]).all()
    own = rows[:, kept // bt:][rows[:, kept // bt:] >= 0]
    assert own.unique().numel() == own.numel()
    ep.kv_free(state, ints([0, 1, 2]), ws, status)
    assert not refs.any() and not lens.any() and (tables == -1).all() and status.item() == 0
