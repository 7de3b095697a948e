"""Groups whose offsets name no such sequences or rows: their sequences read the
leading keys through their own rows of the table, as without a group, and the
status word says so. Tolerances as in the other tests of attention."""
import pytest
import torch

from gpu_util import note
from kv_ref import BAD_PAGE
from test_gpu_kv_attend import BF, F8, HF, Case, ints

pytestmark = pytest.mark.gpu


def checked(c, off, **kw):
    d = c.device()
    d.group_off = ints(off)
    for name, v in kw.items():
        setattr(d, name, v)
    c.call(d)
    c.check(d.out.cpu(), d.lse.cpu())
    assert int(d.status.item()) == BAD_PAGE


@pytest.mark.parametrize("off", [[0, 4], [-1, 3], [-5, 40], [0, 1 << 30]])
@pytest.mark.parametrize("dtype,cache,new", [(BF, BF, [1, 3, 2]), (HF, F8, [70, 1, 9])])
def test_a_group_outside_the_sequences_shares_nothing(dtype, cache, new, off):
    note(f"kv attend {cache} group {off}")
    checked(Case(dtype, cache, 8, 2, 64, 16, [130, 140, 90], new, [0, 3], [64]), off)


@pytest.mark.parametrize("seqs,groups", [(9, 3), (128, 64), (140, 70), (300, 60)])
def test_the_other_groups_keep_what_they_share(seqs, groups):
    """The last group reaches past the sequences; with more groups than LDS holds, and with more
    sequences than one round places."""
    note(f"kv attend {seqs} sequences, {groups} groups, the last too long")
    each = seqs // groups
    off = [each * j for j in range(groups)] + [seqs]
    c = Case(BF, BF, 4, 2, 64, 16, [70 + b % 5 for b in range(seqs)], [1] * seqs, off, [64] * groups)
    checked(c, off[:-1] + [seqs + 1])
    checked(c, off[:-1] + [seqs + 1], q_off=None)
    checked(c, [-1] + off[1:])


def test_groups_in_descending_order_are_flagged():
    c = Case(BF, BF, 4, 2, 64, 16, [70, 75, 90, 66], [1, 1, 1, 1], [1, 1, 4], [64, 64])
    c.test(status=0)
    checked(c, [2, 1, 4])


def test_offsets_past_the_rows_take_their_groups_shared_keys_from_no_one():
    """The last sequence's offset names rows that are not there. It has no row itself (first case) or
    its rows are skipped (second); the rows of the others see all their keys."""
    for new, extra in (([1, 3, 0], 0), ([1, 3, 0], 2)):
        c = Case(BF, BF, 8, 2, 64, 16, [130, 140, 90], new, [0, 3], [64], extra_rows=extra)
        d = c.device()
        d.q_off = ints([0, 1, 4, 9])
        c.call(d)
        out, lse = d.out.cpu(), d.lse.cpu()
        c.check(out, lse)
        assert (out[4:] == 3).all() and (lse[4:] == 3).all()
        assert int(d.status.item()) == BAD_PAGE


def test_offsets_that_are_not_a_batchs_are_flagged_without_groups():
    c = Case(BF, BF, 8, 2, 64, 16, [130, 140, 90], [1, 3, 0])
    for last in (9, 2, -1):
        d = c.device()
        d.q_off = ints([0, 1, 4, last])
        c.call(d)
        c.check(d.out.cpu(), d.lse.cpu())
        assert int(d.status.item()) == BAD_PAGE


def test_empty_groups_and_sequences_without_rows_are_no_fault():
    c = Case(BF, BF, 8, 2, 64, 16, [130, 140, 90, 77], [0, 0, 2, 1], [0, 2, 2, 4], [64, 16, 48])
    c.test(status=0)


def test_refused_groups_in_a_replayed_graph():
    c = Case(BF, BF, 8, 2, 64, 16, [130, 140, 90], [1, 1, 1], [0, 3], [64])
    d = c.device()
    c.call(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(d)
    for i, last in enumerate((4, 3, -2, 3, 9)):
        d.group_off.copy_(ints([0, last]))
        d.status.zero_()
        d.out.fill_(3)
        d.lse.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert int(d.status.item()) == (0 if last == 3 else BAD_PAGE), i
        c.check(d.out.cpu(), d.lse.cpu())
