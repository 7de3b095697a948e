"""Infinities and NaN of V at keys that some rows see and others do not, on every
way through the kernel: tiles copied or widened, rows or keys shared out among
the waves, items cut or written whole, shared keys that rows of a group see
part of. Rows that do not see such a key, and elements that hold none, are
bit-equal to a run without it. Also lengths that pass the table's end."""
import pytest
import torch

from gpu_util import note
from kv_ref import BAD_PAGE
from test_gpu_kv_attend import BF, F8, HF, Case, ints

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def planted(make, keys):
    """make() twice, once with +inf, -inf and NaN (NaN alone in one byte) in elements 3, 5 and 6 of V at
    keys (sequence, position). Rows that see any of them by sequence and position, both results."""
    clean, c = make(), make()
    one_byte = c.cache == F8
    v = c.views(c.pool)[1]
    for b, t in keys:
        row = torch.zeros((c.kv, c.dim), dtype=torch.float32)
        row.copy_(v[c.table[b][t // c.bt], t % c.bt].float())
        row[:, 3], row[:, 5], row[:, 6] = (NAN, NAN, NAN) if one_byte else (INF, -INF, NAN)
        v[c.table[b][t // c.bt], t % c.bt] = row.to(c.cache)
    d, e = c.device(), clean.device()
    c.call(d)
    clean.call(e)
    assert int(d.status.item()) == 0 and int(e.status.item()) == 0
    clean.check(e.out.cpu(), e.lse.cpu())
    return c, d.out.cpu().float(), e.out.cpu().float(), d.lse.cpu(), e.lse.cpu(), one_byte


def compare(got, want, sees, one_byte):
    """got and want [rows, heads, dim]; sees [rows]."""
    assert torch.equal(got[~sees], want[~sees])
    rest = [i for i in range(got.shape[2]) if i not in (3, 5, 6)]
    assert torch.equal(got[sees][..., rest], want[sees][..., rest])
    at = got[sees]
    assert torch.isnan(at[..., 6]).all()
    if one_byte:
        assert torch.isnan(at[..., 3]).all() and torch.isnan(at[..., 5]).all()
    else:
        assert (at[..., 3] == INF).all() and (at[..., 5] == -INF).all()


FORMS = [(BF, BF, 64), (HF, HF, 128), (BF, F8, 64), (HF, F8, 128), (BF, BF, 256), (HF, F8, 256), (HF, HF, 80)]


def sees_of(c, keys, shared_by_all=False):
    rows = torch.zeros(c.t, dtype=torch.bool)
    for b, (lo, hi) in enumerate(zip(c.off, c.off[1:])):
        for j in range(hi - lo):
            pos = c.lens[b] - (hi - lo) + j
            rows[lo + j] = any((shared_by_all or s == b) and t <= pos for s, t in keys)
    return rows


@pytest.mark.parametrize("dtype,cache,dim", FORMS)
def test_hidden_values_in_pieces(dtype, cache, dim):
    """Few items, each cut for many workgroups; a key in the middle of the new tokens of either sequence."""
    note(f"kv attend special pieces {dtype} {cache} {dim}")
    keys = [(0, 297), (1, 190), (1, 181)]
    c, got, want, gl, wl, one = planted(
        lambda: Case(dtype, cache, 4, 2, dim, 16, [300, 200], [5, 40], seed=3), keys)
    compare(got, want, sees_of(c, keys), one)
    assert torch.equal(gl, wl)


@pytest.mark.parametrize("dtype,cache,dim", FORMS)
@pytest.mark.parametrize("new", [3, 40])
def test_hidden_values_in_items_written_whole(dtype, cache, dim, new):
    """More items of one or two tiles than workgroups: most are written by one workgroup."""
    note(f"kv attend special whole {dtype} {cache} {dim} {new}")
    seqs = 320
    keys = [(b, 60 + b % 70 - 1 - b % new) for b in range(0, seqs, 2)]
    c, got, want, gl, wl, one = planted(
        lambda: Case(dtype, cache, 4, 2, dim, 16, [60 + b % 70 for b in range(seqs)], [new] * seqs, seed=4), keys)
    compare(got, want, sees_of(c, keys), one)
    assert torch.equal(gl, wl)


@pytest.mark.parametrize("dtype,cache,dim", FORMS)
@pytest.mark.parametrize("new,keys", [([1, 2, 5], [(0, 36)]), ([1, 30, 5], [(0, 36), (0, 17)])])
def test_hidden_values_in_shared_keys(dtype, cache, dim, new, keys):
    """The shared keys reach past the positions of some rows of the group."""
    note(f"kv attend special shared {dtype} {cache} {dim} {new}")
    c, got, want, gl, wl, one = planted(
        lambda: Case(dtype, cache, 8, 2, dim, 4, [40, 34, 38], new, [0, 3], [37], seed=5), keys)
    sees = sees_of(c, keys, shared_by_all=True)
    assert sees.any() and not sees.all()
    compare(got, want, sees, one)
    assert torch.equal(gl, wl)


@pytest.mark.parametrize("length", [45, 48, 1 << 20])
@pytest.mark.parametrize("new", [1, 40])
def test_a_length_past_the_end_of_a_full_table(length, new):
    """Every entry of the row is a page: the length alone is past the table's end. The row's keys are the
    44 that there are; rows behind the end see all of them."""
    c = Case(HF, HF, 4, 2, 64, 4, [40, 9], [new, 1])
    spare = next(p for p in range(len(c.pool)) if all(p not in r for r in c.table))
    c.table[0][10] = spare
    g = torch.Generator().manual_seed(8)
    for x in c.views(c.pool):
        x[spare] = torch.randn((4, 2, 64), generator=g).to(HF)
    d = c.device()
    d.lens = ints([length, 9])
    c.call(d)
    out, lse = d.out.cpu(), d.lse.cpu()
    assert int(d.status.item()) == BAD_PAGE
    # For the definition: as many keys as there are, for rows that stand at or behind the end of them.
    first = length - new
    behind = [j for j in range(new) if first + j >= 43]
    assert behind
    for j in (behind[0], behind[-1]):
        one = Case(HF, HF, 4, 2, 64, 4, [40, 9], [new, 1])
        one.pool, one.table, one.q = c.pool, c.table, torch.cat([c.q[j:j + 1], c.q[new:]])
        one.lens, one.off = [44, 9], [0, 1, 2]
        one.check(torch.cat([out[j:j + 1], out[new:]]), torch.cat([lse[j:j + 1], lse[new:]]))
