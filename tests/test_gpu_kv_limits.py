"""The paged-cache operators where their tables, tiles and rounds end: more
sequences, groups, requests and pages than one round or an LDS table takes,
padded heads of one-byte caches, signs of the scales, a captured decode step.
Against the same plain definitions and with the same tolerances as the other
tests of these operators."""
import random

import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from test_gpu_kv_append import run
from test_gpu_kv_attend import BF, F8, HF, Case, ints
from test_gpu_kv_pages import Both

pytestmark = pytest.mark.gpu


def lives(seed, seqs, top):
    rng = random.Random(seed)
    new = [rng.choice([0, 1, 1, 1, 2, 3]) for _ in range(seqs)]
    new[seqs // 2] = 40
    return [max(n, 16) + rng.randrange(1, top) for n in new], new


@pytest.mark.parametrize("seqs,groups", [(255, 0), (256, 0), (257, 0), (300, 70), (700, 64), (520, 65), (260, 1)])
def test_more_sequences_and_groups_than_one_round_takes(seqs, groups):
    note(f"kv attend {seqs} sequences, {groups} groups")
    lens, new = lives(seqs, seqs, 150)
    each = (seqs - 7) // groups if groups else 0
    Case(BF, BF, 4, 2, 64, 16, lens, new, [5 + j * each for j in range(groups + 1)] if groups else [],
         [16 * (j % 2) + 16 * (j % 3 == 0) for j in range(groups)]).test()


def test_many_sequences_of_one_token_without_offsets():
    lens = [1 + (i * 37) % 90 for i in range(600)]
    c = Case(HF, HF, 2, 1, 64, 16, lens, [1] * 600)
    c.test(q_off=None)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [16, 80, 144, 240, 256])
def test_one_byte_caches_of_any_head_size(dtype, dim):
    note(f"kv attend e4m3 {dtype} {dim}")
    Case(dtype, F8, 4, 2, dim, 16, [90, 3, 260, 700], [1, 3, 70, 1]).test()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [24, 72, 136, 248, 256])
def test_two_byte_caches_of_any_head_size(dtype, dim):
    note(f"kv attend {dtype} {dim}")
    Case(dtype, dtype, 4, 2, dim, 16, [90, 3, 260, 700, 720], [1, 3, 70, 1, 2], [3, 5], [640]).test()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-3])
@pytest.mark.parametrize("cache", [BF, F8])
def test_signs_of_the_scales(cache, scale):
    c = Case(BF, cache, 4, 2, 64, 16, [90, 5, 260, 1500], [1, 3, 70, 1])
    c.scale = scale
    if cache == F8:
        # Head 0 of K and head 1 of V are stored with their signs turned.
        kc, vc = c.views(c.pool)
        for x, h in ((kc, 0), (vc, 1)):
            x[:, :, h] = (-x[:, :, h].float()).to(cache)
        c.scales[0][0] *= -1
        c.scales[1][1] *= -1
    c.test()


def test_more_new_tokens_allowed_than_there_are():
    for most in (8, 9, 33, 1000):
        c = Case(BF, BF, 8, 2, 128, 16, [90, 5, 260], [1, 3, 2])
        d = c.device()
        ws = torch.empty(ep.kv_attend_bytes(d.cache, 3, 0, c.t, 8, most), dtype=torch.uint8, device="cuda")
        c.call(d, most=most, ws=ws)
        c.check(d.out.cpu(), d.lse.cpu())
        assert int(d.status.item()) == 0


@pytest.mark.parametrize("bt", [129, 300, 2048])
def test_pages_longer_than_a_tile(bt):
    Case(BF, BF, 4, 2, 128, bt, [90, 301, 2300, 2200], [1, 3, 40, 2], [2, 4], [bt if bt < 2000 else 2048]).test()


def test_rows_of_q_are_not_written_over():
    c = Case(BF, BF, 4, 2, 64, 16, [90, 5], [1, 3])
    d = c.device()
    with pytest.raises(ep.EPError):
        ep.kv_attend(d.cache, d.tables, d.lens, d.q_off, d.most, None, None, d.q, d.q, d.lse, 0.1, d.ws,
                     d.status)


def test_two_graphs_replayed_at_once():
    cases = [Case(BF, BF, 8, 2, 128, 16, [530, 600, 513], [1, 1, 1], [0, 3], [512], seed=1),
             Case(HF, HF, 4, 4, 64, 8, [230, 90], [30, 2], seed=2)]
    runs, graphs, streams = [], [], []
    for c in cases:
        d = c.device()
        c.call(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(d)
        runs.append((d, d.out.clone(), d.lse.clone()))
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    for i in range(5):
        for d, _, _ in runs:
            d.out.fill_(3)
            d.lse.fill_(3)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, (d, out, lse) in zip(cases, runs):
            assert torch.equal(d.out, out) and torch.equal(d.lse, lse), i


def test_a_captured_decode_step_equals_eager_ones():
    """extend, append and attend of three samples of a prompt, captured once: the lengths, the pages and
    the shared prefix are read on the device, so every replay is the next step."""
    kv, heads, dim, bt, pages = 2, 6, 64, 4, 40
    g = torch.Generator().manual_seed(3)
    fill = torch.randn((1, pages, bt * 2 * kv * dim), generator=g).to(BF)
    rows = [torch.randn((3, heads + 2 * kv, dim), generator=g).to(BF).cuda() for _ in range(9)]
    inv = torch.from_numpy(ep.rope_freqs(dim)[0]).cuda()

    class State:
        def __init__(self):
            self.pool, self.status = fill.cuda(), ints([0])
            self.tables, self.lens = torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), ints([0] * 3)
            self.refs = ints([0] * pages)
            self.g = ep.make_kv_pages(self.tables, self.lens, self.refs, self.pool, bt)
            self.ws = torch.empty(ep.kv_pages_bytes(self.g, 3), dtype=torch.uint8, device="cuda")
            view = self.pool.view(pages, bt, 2, kv, dim)
            self.cache = ep.make_kv_cache(view[:, :, 0], view[:, :, 1])
            self.attend_ws = torch.empty(ep.kv_attend_bytes(self.cache, 3, 1, 3, heads), dtype=torch.uint8,
                                         device="cuda")
            self.all, self.one = ints([0, 1, 2]), ints([1, 1, 1])
            self.group, self.shared = ints([0, 3]), ints([8])
            self.rope = ep.make_rope(inv, dim)
            self.new = torch.zeros_like(rows[0])
            self.out, self.lse = torch.zeros((3, heads, dim), dtype=BF, device="cuda"), torch.zeros((3, heads), device="cuda")
            ep.kv_extend(self.g, ints([0]), ints([10]), self.ws, self.status)
            ep.kv_fork(self.g, ints([0, 0]), ints([1, 2]), self.ws, self.status)
            self.turned = torch.zeros((3, heads, dim), dtype=BF, device="cuda")

        def step(self):
            q, k, v = self.new.split([heads, kv, kv], 1)
            ep.kv_extend(self.g, self.all, self.one, self.ws, self.status)
            ep.kv_append(self.cache, self.tables, self.lens, None, q, k, v, self.turned, self.rope, self.status)
            ep.kv_attend(self.cache, self.tables, self.lens, None, 1, self.group, self.shared, self.turned, self.out,
                         self.lse, 0.125, self.attend_ws, self.status)

        def everything(self):
            return [self.pool, self.tables, self.lens, self.refs, self.out, self.lse, self.status]

    eager, other = State(), State()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step()
    for i, r in enumerate(rows):
        eager.new.copy_(r)
        other.new.copy_(r)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager.everything(), other.everything()):
            assert torch.equal(x, y), i
    assert eager.lens.tolist() == [19, 19, 19] and eager.status.item() == 0


def test_more_sequences_requests_and_pages_than_the_planner_keeps_at_hand():
    note("kv pages: 9000 sequences")
    b = Both(7, 9000, 4, 30000, 3, 1, 16)
    b.ws = torch.full((ep.kv_pages_bytes(b.g, 9000),), 0x5A, dtype=torch.uint8, device="cuda")
    rng = random.Random(8)
    ids = list(range(9000))
    rng.shuffle(ids)
    old, young = ids[:4000], ids[4000:]
    b.do("extend", old, [1 + i % 12 for i in range(4000)])          # about 10000 pages
    b.do("extend", old[:500] + old[:3] + [9000, -1], [1] * 505)     # few pages, requests that do not count
    b.do("fork", [old[i % 4000] for i in range(5000)] + [old[0]], young + [young[0]])
    b.do("free", old[::2] + old[:4])
    b.do("compact")
    b.do("extend", young, [12] * 5000)                              # some rows end before it
    b.do("free", ids)


def test_append_of_many_sequences_and_of_blocks_that_end_early():
    note("kv append: 8200 sequences")
    lens = [1 + (i * 7) % 23 for i in range(8200)]
    assert run(BF, BF, 1, 1, 16, 8, 1, 1.0, [1] * 8200, lens, 16, no_off=True) == 0
    assert run(HF, HF, 1, 1, 16, 16, 0, 1.0, [2043, 60], [2043, 70], 16, extra_rows=5) == 0
    assert run(BF, F8, 1, 1, 16, 16, 0, 1.0, [8200], [8250], 64, extra_rows=30) == 0
