"""Workspaces, status words and other small outputs of the paged-cache operators
that are too small or of another type: the binding refuses them before anything
is launched (no GPU). The library itself sees the allocation behind an address,
which under a caching allocator is more than the tensor."""
import pytest
import torch

import combine_ep_plan_amd as ep


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def buf(n):
    return torch.zeros(n, dtype=torch.uint8)


def state():
    return ep.make_kv_pages(i32(4, 8), i32(4), i32(32), torch.zeros((1, 32, 256), dtype=torch.uint8), 16)


def page_calls(m):
    """name: a call of m requests with the given workspace and status."""
    a, b = i32(m), i32(m)
    return {
        "extend": lambda g, ws, st: ep.kv_extend(g, a, b, ws, st, 0),
        "fork": lambda g, ws, st: ep.kv_fork(g, a, b, ws, st, 0),
        "free": lambda g, ws, st: ep.kv_free(g, a, ws, st, 0),
        "copy": lambda g, ws, st: ep.kv_copy_pages(g, a, b, ws, st, 0),
    }


def attend(ws, status, max_new=1, tokens=3, heads=4, groups=0, cache=None, **kw):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    c = cache or ep.make_kv_cache(k, k)
    q = torch.zeros((tokens, heads, 64), dtype=torch.bfloat16)
    g = (i32(groups + 1), i32(groups)) if groups else (None, None)
    ep.kv_attend(c, i32(3, 4), i32(3), i32(4), max_new, *g, q, torch.zeros_like(q), None, 0.1, ws, status, 0)


def need_of(max_new=1, tokens=3, heads=4, groups=0):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    return ep.kv_attend_bytes(ep.make_kv_cache(k, k), 3, groups, tokens, heads, max_new)


@pytest.mark.parametrize("m", [1, 5, 1000])
@pytest.mark.parametrize("name", ["extend", "fork", "free", "copy"])
def test_page_workspaces_are_measured(name, m):
    g = state()
    need = ep.kv_pages_bytes(g, m)
    call = page_calls(m)[name]
    for short in (buf(need - 1), buf(need)[1:], buf(0), torch.zeros((need - 1) // 4, dtype=torch.int32)):
        with pytest.raises(ValueError, match="ws"):
            call(g, short, i32(1))
    with pytest.raises(ep.EPError):          # on to the library, which finds no device memory
        call(g, buf(need), i32(1))
    with pytest.raises(ep.EPError):
        call(g, torch.zeros(need, dtype=torch.int64), i32(1))


def test_a_workspace_of_fewer_requests_is_refused():
    g = state()
    ws = buf(ep.kv_pages_bytes(g, 8))
    with pytest.raises(ValueError, match="ws"):
        page_calls(500)["extend"](g, ws, i32(1))


def test_compact_measures_its_workspace_and_its_count():
    g = state()
    need = ep.kv_pages_bytes(g, 0)
    with pytest.raises(ValueError, match="ws"):
        ep.kv_compact(g, buf(need - 1), i32(1), None, 0)
    for live in (i32(0), torch.zeros(1), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError, match="n_live"):
            ep.kv_compact(g, buf(need), i32(1), live, 0)
    with pytest.raises(ep.EPError):
        ep.kv_compact(g, buf(need), i32(1), i32(1), 0)


@pytest.mark.parametrize("kw", [dict(), dict(max_new=9), dict(max_new=40, tokens=60), dict(groups=2),
                                dict(heads=40, tokens=90)])
def test_attention_workspaces_are_measured(kw):
    need = need_of(**kw)
    for short in (buf(need - 1), buf(0)):
        with pytest.raises(ValueError, match="ws"):
            attend(short, i32(1), **kw)
    with pytest.raises(ep.EPError):
        attend(buf(need), i32(1), **kw)


def test_a_decode_steps_workspace_is_refused_for_a_prompt():
    with pytest.raises(ValueError, match="ws"):
        attend(buf(need_of(tokens=60)), i32(1), max_new=40, tokens=60)


STATUS = [torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int16), torch.zeros(1, dtype=torch.uint8),
          torch.zeros(2, dtype=torch.float32), torch.zeros(1, dtype=torch.int64)]


@pytest.mark.parametrize("status", STATUS, ids=[f"{t.dtype}-{t.numel()}" for t in STATUS])
def test_status_words_are_checked(status):
    g = state()
    for name, call in page_calls(2).items():
        with pytest.raises(ValueError, match="status"):
            call(g, buf(ep.kv_pages_bytes(g, 2)), status)
    with pytest.raises(ValueError, match="status"):
        ep.kv_compact(g, buf(ep.kv_pages_bytes(g, 0)), status, None, 0)
    with pytest.raises(ValueError, match="status"):
        attend(buf(need_of()), status)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="status"):
        ep.kv_append(ep.make_kv_cache(k, k), i32(3, 4), i32(3), None, None, rows, rows, None, None, status, 0)


def test_an_empty_batch_needs_no_workspace():
    """On to the library, which is where a call without a device ends."""
    with pytest.raises(ep.EPError):
        attend(buf(0), i32(1), tokens=0)


def test_invalid_sizes_keep_the_librarys_own_error():
    """A size that the library cannot lay out has no workspace: its error is the one that counts."""
    g = state()
    ws = buf(ep.kv_pages_bytes(g, 2))
    g.page_tokens = 0
    with pytest.raises(ep.EPError, match="sizes must be positive"):
        page_calls(2)["extend"](g, ws, i32(1))
    g = state()
    g.n_pages = -1
    with pytest.raises(ep.EPError, match="sizes must be positive"):
        page_calls(2)["extend"](g, buf(0), i32(1))
    with pytest.raises(ep.EPError, match="n_heads"):
        attend(buf(64), i32(1), heads=3)


def test_addresses_pass_unmeasured():
    """A raw address has no size: the library's own check is all there is."""
    g = state()
    ws = buf(ep.kv_pages_bytes(g, 2))
    with pytest.raises(ep.EPError):
        page_calls(2)["extend"](g, ws.data_ptr(), i32(1).data_ptr())


def test_page_workspaces_are_measured_as_the_library_lays_them_out():
    """For every size: the binding's own measure is the library's."""
    for seqs, n_pages, m in ((1, 1, 1), (4, 32, 63), (9000, 30000, 9000), (7, 1 << 20, 16384)):
        g = ep.KvPages(None, None, None, None, seqs, 3, n_pages, 16, 2, 0, 256, 256 * n_pages)
        need = ep.kv_pages_bytes(g, m)
        assert need > 0
        assert ep._page_room(g, m, buf(need)) is not None
        with pytest.raises(ValueError):
            ep._page_room(g, m, buf(need - 1))
