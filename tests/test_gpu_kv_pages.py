"""Page bookkeeping on the GPU against sequential Python: tables, lengths,
counts, every byte of the pool and the status word, all exact."""
import random

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep
from gpu_util import note
from kv_ref import Pages

pytestmark = pytest.mark.gpu


class Both:
    """The library's state on the GPU beside the plain one."""

    def __init__(self, seed, seqs, max_pages, pages, page_tokens, ranks, page_bytes):
        g = torch.Generator().manual_seed(seed)
        pool = torch.randint(0, 256, (ranks, pages, page_bytes), dtype=torch.uint8, generator=g)
        tables = [[-1] * max_pages for _ in range(seqs)]
        self.ref = Pages(tables, [0] * seqs, [0] * pages, pool, page_tokens)
        self.tables = torch.tensor(tables, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.pool = pool.cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.g = ep.make_kv_pages(self.tables, self.lens, self.refs, self.pool, page_tokens)
        self.ws = torch.full((ep.kv_pages_bytes(self.g, 4096),), 0x5A, dtype=torch.uint8,
                             device="cuda")

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def upload(self):
        """The plain state (changed by the test) onto the GPU."""
        self.tables.copy_(torch.tensor(self.ref.tables, dtype=torch.int32))
        self.lens.copy_(torch.tensor(self.ref.lens, dtype=torch.int32))
        self.refs.copy_(torch.tensor(self.ref.refs, dtype=torch.int32))

    def do(self, op, *args):
        dev = [self.ints(a) for a in args]
        if op == "compact":
            live = torch.full((1,), -1, dtype=torch.int32, device="cuda")
            ep.kv_compact(self.g, self.ws, self.status, live)
            want, moved = self.ref.compact()
            assert int(live.item()) == want
            ids = self.ws[:4 * len(self.ref.refs)].cpu().numpy().view(np.int32)
            assert {int(p): int(t) for p, t in enumerate(ids) if t >= 0} == moved
        else:
            fn = ep.kv_copy_pages if op == "copy" else getattr(ep, "kv_" + op)
            fn(self.g, *dev, self.ws, self.status)
            getattr(self.ref, op)(*args)
        self.check(op)

    def check(self, op):
        assert self.tables.cpu().tolist() == self.ref.tables, op
        assert self.lens.cpu().tolist() == self.ref.lens, op
        assert self.refs.cpu().tolist() == self.ref.refs, op
        assert torch.equal(self.pool.cpu(), self.ref.pool), op
        assert int(self.status.item()) == self.ref.status, op


SHAPES = [  # seqs, max_pages, pages, page_tokens, ranks, page_bytes
    (1, 1, 1, 1, 1, 16),
    (5, 3, 9, 4, 2, 48),
    (40, 20, 150, 16, 1, 1024),
    (17, 64, 700, 1, 3, 32),
    (9, 12, 60, 7, 2, 16400),        # a page ends inside a piece of the copy
    (300, 40, 9000, 5, 1, 16),       # more pages than one pass over the counts takes
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_random_lives_match_the_plain_state(shape):
    seqs, max_pages, pages, bt, ranks, page_bytes = shape
    rng = random.Random(pages)
    b = Both(pages, *shape)
    for step in range(24):
        op = rng.choice(["extend", "extend", "fork", "fork", "free", "compact", "copy"])
        note(f"kv pages {shape} step {step} {op}")
        m = rng.randint(1, min(2 * seqs, 60))
        some = lambda: rng.randrange(-1, seqs + 1)  # noqa: E731  (ids out of range, repeated ids)
        if op == "extend":
            top = max(1, 2 * max_pages * bt // 3)
            b.do(op, [some() for _ in range(m)], [rng.randint(-1, top) for _ in range(m)])
        elif op == "fork":
            b.do(op, [some() for _ in range(m)], [some() for _ in range(m)])
        elif op == "free":
            b.do(op, [some() for _ in range(rng.randint(1, max(1, seqs // 3)))])
        elif op == "copy":
            page = lambda: rng.randrange(-1, pages + 1)  # noqa: E731
            b.do(op, [page() for _ in range(m)], [page() for _ in range(m)])
        else:
            b.do(op)


def test_requests_past_one_round_of_the_planner():
    b = Both(1, 2600, 4, 6000, 2, 1, 16)
    ids = list(range(2600))
    random.Random(2).shuffle(ids)
    b.do("extend", ids, [1 + i % 8 for i in range(2600)])
    b.do("free", ids[:1500])
    b.do("fork", [ids[1500 + i % 1100] for i in range(1500)], ids[:1500])
    b.do("compact")


def test_capacity_is_granted_in_request_order():
    b = Both(3, 6, 8, 10, 4, 1, 64)
    b.do("extend", [0, 1, 2, 3], [16, 17, 8, 0])     # 4 + 5 pages fit, 2 more do not, 0 need none
    assert b.ref.status == ep.EP_STATUS_CAPACITY and b.ref.lens == [16, 17, 0, 0, 0, 0]
    b.do("fork", [1, 1, 0], [2, 3, 4])               # one page left: the second child is refused
    assert b.ref.lens == [16, 17, 17, 0, 16, 0]


def test_fork_in_one_call_sees_the_state_before_it():
    b = Both(4, 6, 4, 12, 4, 2, 32)
    b.do("extend", [0], [6])
    b.do("fork", [0, 1, 2], [1, 2, 3])               # 1 and 2 are empty before the call
    assert b.ref.lens == [6, 6, 0, 0, 0, 0]
    assert b.ref.status == 0


def test_broken_tables_are_flagged_and_touch_nothing_else():
    b = Both(5, 6, 6, 20, 4, 1, 64)
    b.do("extend", [0, 1, 2], [20, 9, 3])
    b.ref.tables[0][1], b.ref.tables[0][4] = 20, -5
    b.ref.tables[2][0] = 1 << 30
    b.upload()
    b.do("fork", [0, 2], [3, 4])
    assert b.ref.status == ep.EP_STATUS_BAD_PAGE
    b.do("compact")
    b.do("free", [0, 3, 1, 2])
    b.ref.lens[5], b.ref.lens[4] = 1 << 30, -7       # lengths outside the table
    b.upload()
    for op, args in (("extend", ([5, 4], [1, 1])), ("fork", ([5], [0])), ("compact", ()),
                     ("free", ([5, 4],))):
        b.do(op, *args)


def test_copy_by_list_refuses_pairs_that_depend_on_order():
    b = Both(6, 1, 1, 12, 1, 2, 16 * 1025)
    b.do("copy", [0, 2, 4, 6, 6, 8], [1, 1, 5, 4, 7, 8])   # 1 twice; 4 is read and written
    assert b.ref.status == ep.EP_STATUS_BAD_PAGE
    assert torch.equal(b.ref.pool[:, 1], b.ref.pool[:, 0])


def test_empty_calls_and_graph_replay():
    b = Both(7, 8, 6, 40, 4, 2, 256)
    none = b.ints([])
    ep.kv_extend(b.g, none, none, b.ws, b.status)
    ep.kv_fork(b.g, none, none, b.ws, b.status)
    ep.kv_free(b.g, none, b.ws, b.status)
    ep.kv_copy_pages(b.g, none, none, b.ws, b.status)
    b.check("nothing")
    b.do("extend", [0, 1], [9, 18])
    slots, add = b.ints([2, 3, 4, 5]), b.ints([5, 7])
    parents, children = b.ints([0, 2]), b.ints([4, 5])

    def step():
        ep.kv_free(b.g, slots, b.ws, b.status)
        ep.kv_extend(b.g, slots[:2], add, b.ws, b.status)
        ep.kv_fork(b.g, parents, children, b.ws, b.status)
        ep.kv_compact(b.g, b.ws, b.status)

    def plain():
        b.ref.free([2, 3, 4, 5])
        b.ref.extend([2, 3], [5, 7])
        b.ref.fork([0, 2], [4, 5])
        b.ref.compact()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    plain()
    b.check("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        add.copy_(b.ints([5, 7]))
        graph.replay()
        plain()
        b.check(f"replay {i}")
        b.do("extend", [1], [1])


def test_pool_offsets_past_32_bits():
    """Pages 5 GiB apart: rank 1 of a pool of almost 3 GiB per rank, and a page near its end."""
    page, n = 1 << 20, 3000
    pool = torch.zeros((2, n, page // 8), dtype=torch.int64, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    refs = ints([1] * (n - 2) + [0, 1])
    tables, lens = ints([[n - 1], [-1]]), ints([3, 0])
    status = ints([0])
    g = ep.make_kv_pages(tables, lens, refs, pool, 4)
    ws = torch.empty(ep.kv_pages_bytes(g, 4), dtype=torch.uint8, device="cuda")
    pool[0, n - 1], pool[1, n - 1] = 11, 22
    ep.kv_fork(g, ints([0]), ints([1]), ws, status)
    assert (pool[:, n - 2, 0].tolist(), pool[:, n - 2, -1].tolist()) == ([11, 22], [11, 22])
    pool[1, 0] = 33
    ep.kv_copy_pages(g, ints([0]), ints([n - 1]), ws, status)
    assert pool[1, n - 1].unique().tolist() == [33] and pool[0, n - 1].unique().tolist() == [0]
    assert tables.tolist() == [[n - 1], [n - 2]] and status.item() == 0
