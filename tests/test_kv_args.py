"""Refusals and host-side arithmetic of the paged-cache operators (no GPU):
the checks that come before the device is looked up, the binding's own
checks, and the rotary frequencies against their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import combine_ep_plan_amd as ep

FAKE = 0x10000


def pages(**kw):
    a = dict(tables=FAKE, lens=FAKE, refs=FAKE, pool=FAKE, n_seqs=4, max_pages=8, n_pages=32,
             page_tokens=16, ranks=1, reserved=0, page_bytes=256, rank_bytes=32 * 256)
    a.update(kw)
    return ep.KvPages(**a)


@pytest.mark.parametrize("kw,m,code", [
    (dict(n_seqs=0), 1, ep.EP_ERR_INVALID_ARG),
    (dict(max_pages=0), 1, ep.EP_ERR_INVALID_ARG),
    (dict(n_pages=-1), 1, ep.EP_ERR_INVALID_ARG),
    (dict(page_tokens=0), 1, ep.EP_ERR_INVALID_ARG),
    (dict(ranks=0), 1, ep.EP_ERR_INVALID_ARG),
    (dict(reserved=1), 1, ep.EP_ERR_INVALID_ARG),
    (dict(page_bytes=8), 1, ep.EP_ERR_INVALID_ARG),
    (dict(page_bytes=264), 1, ep.EP_ERR_INVALID_ARG),
    (dict(rank_bytes=32 * 256 - 16), 1, ep.EP_ERR_INVALID_ARG),
    (dict(rank_bytes=32 * 256 + 8), 1, ep.EP_ERR_INVALID_ARG),
    (dict(rank_bytes=-16), 1, ep.EP_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 30, page_bytes=1 << 40, rank_bytes=1 << 44), 1, ep.EP_ERR_UNSUPPORTED),
    (dict(ranks=1 << 30, rank_bytes=1 << 44), 1, ep.EP_ERR_UNSUPPORTED),
    (dict(ranks=65535), 1, ep.EP_ERR_UNSUPPORTED),
    (dict(n_seqs=1 << 30, max_pages=1 << 30), 1, ep.EP_ERR_UNSUPPORTED),
    (dict(), -1, ep.EP_ERR_INVALID_ARG),
    (dict(), ep.EP_KV_MAX_REQUESTS + 1, ep.EP_ERR_UNSUPPORTED),
])
def test_page_state_is_checked_before_the_device(kw, m, code):
    g, lib = ctypes.byref(pages(**kw)), ep.lib()
    assert ep.kv_pages_bytes(pages(**kw), m) == 0 and ep.last_error() != ""
    assert lib.ep_kv_extend(g, FAKE, FAKE, m, FAKE, FAKE, None) == code
    assert lib.ep_kv_fork(g, FAKE, FAKE, m, FAKE, FAKE, None) == code
    assert lib.ep_kv_free(g, FAKE, m, FAKE, FAKE, None) == code
    assert lib.ep_kv_copy_pages(g, FAKE, FAKE, m, FAKE, FAKE, None) == code
    if kw:
        assert lib.ep_kv_compact(g, None, FAKE, FAKE, None) == code


def test_page_workspace_holds_its_arrays():
    for n_pages, m in ((1, 0), (32, 5), (100000, ep.EP_KV_MAX_REQUESTS)):
        g = pages(n_pages=n_pages, rank_bytes=n_pages * 256)
        assert ep.kv_pages_bytes(g, m) >= 4 * (2 * n_pages + 4 + 2 * m + n_pages // 2048 + 2)


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, page_stride=16 * 512, token_stride=512, head_stride=256, n_pages=8,
             page_tokens=16, n_heads=2, head_dim=128, dtype=ep.EP_DTYPE_BF16)
    a.update(kw)
    return ep.KvCache(**a)


def batch(**kw):
    a = dict(tables=FAKE, lens=FAKE, q_off=FAKE, n_seqs=2, max_pages=4, n_tokens=3, dtype=ep.EP_DTYPE_BF16)
    a.update(kw)
    return ep.KvBatch(**a)


ROWS = ep.Rows(FAKE, 2048, 256)


def append(c=None, b=None, q=ROWS, heads=4, q_out=ROWS, rope=None):
    return ep.lib().ep_kv_append(c or cache(), b or batch(), q, heads, ROWS, ROWS, q_out, rope, FAKE, None)


def attend(c=None, b=None, groups=None, max_new=1, heads=4, scale=0.1):
    return ep.lib().ep_kv_attend(c or cache(), b or batch(), groups, max_new, ROWS, heads, ROWS, None,
                                 scale, FAKE, FAKE, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), ep.EP_ERR_INVALID_ARG),
    (dict(reserved=2), ep.EP_ERR_INVALID_ARG),
    (dict(n_pages=0), ep.EP_ERR_INVALID_ARG),
    (dict(page_tokens=0), ep.EP_ERR_INVALID_ARG),
    (dict(n_heads=0), ep.EP_ERR_INVALID_ARG),
    (dict(head_dim=100), ep.EP_ERR_INVALID_ARG),
    (dict(head_dim=72, dtype=ep.EP_DTYPE_E4M3), ep.EP_ERR_INVALID_ARG),
    (dict(head_dim=264, head_stride=1024), ep.EP_ERR_UNSUPPORTED),
    (dict(token_stride=520), ep.EP_ERR_INVALID_ARG),
    (dict(page_stride=-16), ep.EP_ERR_INVALID_ARG),
    (dict(head_stride=240), ep.EP_ERR_INVALID_ARG),
    (dict(token_stride=128), ep.EP_ERR_INVALID_ARG),
    (dict(n_pages=1 << 30, page_stride=1 << 40), ep.EP_ERR_UNSUPPORTED),
    (dict(dtype=ep.EP_DTYPE_F16), ep.EP_ERR_UNSUPPORTED),        # rows are bf16
])
def test_caches_are_checked_before_the_device(kw, code):
    assert append(cache(**kw)) == code and ep.last_error() != ""
    assert attend(cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=ep.EP_DTYPE_E4M3), ep.EP_ERR_INVALID_ARG),
    (dict(n_seqs=-1), ep.EP_ERR_INVALID_ARG),
    (dict(n_tokens=-1), ep.EP_ERR_INVALID_ARG),
    (dict(max_pages=0), ep.EP_ERR_INVALID_ARG),
    (dict(n_tokens=(1 << 24) + 1), ep.EP_ERR_UNSUPPORTED),
    (dict(n_seqs=1 << 30, max_pages=1 << 30), ep.EP_ERR_UNSUPPORTED),
])
def test_batches_are_checked_before_the_device(kw, code):
    assert append(b=batch(**kw)) == code and ep.last_error() != ""
    assert attend(b=batch(**kw)) == code


def test_other_arguments_are_checked_before_the_device():
    bad = ep.EP_ERR_INVALID_ARG
    assert append(heads=3) == bad and attend(heads=3) == bad and attend(heads=0) == bad
    assert append(q=None) == bad and append(q_out=None) == bad
    assert append(rope=ep.Rope(FAKE, 130, 0, 1.0, 0)) == bad
    assert append(rope=ep.Rope(FAKE, 63, 0, 1.0, 0)) == bad
    assert append(rope=ep.Rope(FAKE, 64, 2, 1.0, 0)) == bad
    assert append(rope=ep.Rope(FAKE, 64, 0, 1.0, 5)) == bad
    assert attend(max_new=0) == bad and attend(scale=math.inf) == bad and attend(scale=math.nan) == bad
    assert attend(groups=ep.KvGroups(FAKE, FAKE, -1, 0)) == bad
    assert attend(groups=ep.KvGroups(FAKE, FAKE, 1, 9)) == bad
    assert ep.lib().ep_kv_append(None, batch(), ROWS, 4, ROWS, ROWS, ROWS, None, FAKE, None) == bad
    assert ep.lib().ep_kv_append(cache(), None, ROWS, 4, ROWS, ROWS, ROWS, None, FAKE, None) == bad
    assert ep.kv_attend_bytes(cache(), 2, 0, 3, 3) == 0 and ep.kv_attend_bytes(cache(), 2, 0, 3, 4, 0) == 0
    assert ep.kv_attend_bytes(cache(), 2, 1, 3, 4) > 0


def test_the_binding_refuses_what_it_cannot_pass():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for bad in ((k, k[:, :, :1]), (k, k.half()), (k.transpose(2, 3), k.transpose(2, 3)),
                (k.float(), k.float()), (k, k.transpose(1, 2).contiguous().transpose(1, 2)), (k[0], k[0])):
        with pytest.raises(ValueError):
            ep.make_kv_cache(*bad)
    with pytest.raises(ValueError):
        ep.make_kv_cache(k, k, torch.zeros(3))
    pool = torch.zeros((1, 32, 256), dtype=torch.uint8)
    for tables, lens, refs, p in ((i32(4, 8).long(), i32(4), i32(32), pool), (i32(4, 8), i32(5), i32(32), pool),
                                  (i32(4, 8), i32(4), i32(31), pool), (i32(4, 8).t(), i32(8), i32(32), pool),
                                  (i32(4, 8), i32(4), i32(32), pool[:, :, ::2])):
        with pytest.raises(ValueError):
            ep.make_kv_pages(tables, lens, refs, p, 16)
    g = ep.make_kv_pages(i32(4, 8), i32(4), i32(32), pool, 16)
    with pytest.raises(ValueError):
        ep.kv_extend(g, i32(3), i32(2), pool, i32(1))
    with pytest.raises(ValueError):
        ep.kv_fork(g, i32(3), i32(3, 1), pool, i32(1))
    c = ep.make_kv_cache(k, k)
    q, kk = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for a in ((q, kk[:2], kk, q), (q, kk, kk, None), (q.half(), kk, kk, q), (q, kk, kk.transpose(0, 1), q),
              (torch.zeros((3, 4, 128), dtype=torch.bfloat16)[..., ::2], kk, kk, q)):
        with pytest.raises(ValueError):
            ep.kv_append(c, i32(3, 4), i32(3), None, *a, None, i32(1))
    with pytest.raises(ValueError):
        ep.kv_attend(c, i32(3, 4), i32(3), None, 1, i32(2), None, q, q, None, 0.1, pool, i32(1))
    with pytest.raises(ValueError):
        ep.kv_attend(c, i32(3, 4), i32(3), i32(3), 1, None, None, q, q, None, 0.1, pool, i32(1))
    with pytest.raises(ValueError):
        ep.kv_attend(c, i32(3, 4), i32(3), None, 1, None, None, q, q, torch.zeros((3, 3)), 0.1, pool, i32(1))
    with pytest.raises(ValueError):
        ep.make_rope(torch.zeros(31), 64)


def test_frequencies_follow_their_formulas():
    """Each frequency is the 64-bit value rounded once (2^-24), plus the 64-bit library's own error."""
    rot, base, f, orig = 128, 10000.0, 8.0, 16384
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    close = lambda a, b: np.abs(a.astype(np.float64) - b).max() <= 2.0**-23 * np.abs(b).max() and \
        (np.abs(a - b) <= 2.0**-23 * b).all()  # noqa: E731
    got, m = ep.rope_freqs(rot, base)
    assert close(got, plain) and m == 1.0
    got, m = ep.rope_freqs(rot, base, ep.EP_ROPE_LINEAR, f)
    assert close(got, plain / f) and m == 1.0
    got, m = ep.rope_freqs(rot, base, ep.EP_ROPE_NTK, f)
    assert close(got, (base * f ** (rot / (rot - 2))) ** (-2.0 * i / rot)) and m == 1.0
    # The lowest frequency of the NTK form is the linear one's; the highest is kept.
    assert abs(got[-1] / (plain[-1] / f) - 1) < 1e-6 and got[0] == 1.0
    got, m = ep.rope_freqs(rot, base, ep.EP_ROPE_YARN, f, orig, 32.0, 1.0)
    turns = orig * plain / (2 * math.pi)
    assert m == np.float32(0.1 * math.log(f) + 1)
    assert close(got[turns > 33], plain[turns > 33])                   # fast pairs stay
    assert close(got[turns < 0.8], plain[turns < 0.8] / f)             # slow ones are divided
    assert (np.diff(got) < 0).all()
    assert (got <= plain * (1 + 1e-6)).all() and (got >= plain / f * (1 - 1e-6)).all()
    assert len(ep.rope_freqs(2, base, ep.EP_ROPE_NTK, f)[0]) == 1      # one pair: the base has no effect


@pytest.mark.parametrize("args", [(0,), (3,), (258,), (64, 1.0), (64, math.inf), (64, 1e4, 4), (64, 1e4, 1, 0.5),
                                  (64, 1e4, 1, math.nan), (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096, 1.0, 2.0),
                                  (64, 1e4, 3, 2.0, 4096, 32.0, 0.0)])
def test_frequencies_refuse_what_has_no_meaning(args):
    with pytest.raises(ep.EPError):
        ep.rope_freqs(*args)
