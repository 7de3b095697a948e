"""Python binding of the gfx950 MoE expert-parallel dispatch/combine library.

Thin ctypes layer over the C ABI in ``include/ep.h``: the functions below
have the same names as the C entry points and only marshal arguments
(tensor data pointers, the current HIP stream). Every step of the path runs
in the library's HIP kernels; there is no fallback. If the compiled library
is missing, importing this package raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libep_mi355x.so")

EP_OK = 0
EP_ERR_INVALID_ARG = -1
EP_ERR_UNSUPPORTED = -2
EP_ERR_DEVICE_MISMATCH = -3
EP_ERR_HIP = -4
EP_STATUS_BAD_EXPERT = 1
EP_STATUS_CAPACITY = 2
EP_STATUS_BAD_REGION = 4
EP_STATUS_BAD_PAGE = 8
EP_PAYLOAD_BF16 = 0
EP_PAYLOAD_FP8_B128 = 1
EP_KV_STATIC_SLOTS = 64
EP_PROBE_COPY, EP_PROBE_FILL, EP_PROBE_READ, EP_PROBE_SCATTER, EP_PROBE_SCATTER_WIDE = range(5)
EP_KV_MAX_REQUESTS = 16384
EP_DTYPE_BF16, EP_DTYPE_F16, EP_DTYPE_E4M3 = range(3)
EP_ROPE_HALF, EP_ROPE_INTERLEAVED = range(2)
EP_ROPE_NONE, EP_ROPE_LINEAR, EP_ROPE_NTK, EP_ROPE_YARN = range(4)
EP_PROBE_NT_LOADS, EP_PROBE_XCD, EP_PROBE_ONE_WAVE = 1, 2, 4

# Every entry point the C header declares (checked by the tests).
EXPORTS = (
    "ep_recv_bound", "ep_capacity", "ep_num_planes", "ep_row_bytes",
    "ep_plan_bytes", "ep_plan_views", "ep_plan", "ep_dispatch", "ep_dispatch_quant",
    "ep_dispatch_pack",
    "ep_dispatch_pack_quant",
    "ep_dispatch_transfer", "ep_dispatch_unpack", "ep_dispatch_recv",
    "ep_dispatch_send", "ep_dispatch_recv_split", "ep_dispatch_send_plan",
    "ep_dispatch_send_pack", "ep_dispatch_recv_plan", "ep_dispatch_recv_pull",
    "ep_expert_stub", "ep_combine",
    "ep_combine_presum", "ep_kv_plan", "ep_kv_push", "ep_kv_push_staged",
    "ep_kv_push_staged_static",
    "ep_kv_pages_bytes", "ep_kv_extend", "ep_kv_fork", "ep_kv_free", "ep_kv_compact",
    "ep_kv_copy_pages", "ep_rope_freqs", "ep_kv_append", "ep_kv_attend_bytes", "ep_kv_attend",
    "ep_probe_copy", "ep_probe_pattern", "ep_status_string",
    "ep_last_error",
)


class EPError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where} failed ({code}): {msg}")
        self.code = code


class Desc(ctypes.Structure):
    """ep_desc: N, T, H, E, R, payload, cap_rows (0 = worst-case bound)."""
    _fields_ = [
        ("n_ranks", ctypes.c_int32), ("tokens", ctypes.c_int32),
        ("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
        ("topk", ctypes.c_int32), ("payload", ctypes.c_int32),
        ("cap_rows", ctypes.c_int64),
    ]


class PlanView(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "cnt", "send_off", "send_pos", "recv_off", "grp_off", "grp_pos",
        "src_off", "comb_row", "grp_slot", "send_slot", "recv_rows", "send_seg", "win_list")]


class KvPages(ctypes.Structure):
    """ep_kv_pages: tables, lens, refs and pool of a paged cache (see make_kv_pages)."""
    _fields_ = [
        ("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
        ("pool", ctypes.c_void_p),
        ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32), ("ranks", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("page_bytes", ctypes.c_int64), ("rank_bytes", ctypes.c_int64),
    ]


class KvCache(ctypes.Structure):
    """ep_kv_cache: K and V of one layer in the pages of a pool (see make_kv_cache)."""
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("n_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class KvBatch(ctypes.Structure):
    """ep_kv_batch: tables, lengths and row offsets of the sequences of one step."""
    _fields_ = [
        ("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("q_off", ctypes.c_void_p),
        ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class Rows(ctypes.Structure):
    """ep_rows: [tokens][heads][head_dim] rows by their byte strides."""
    _fields_ = [("p", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Rope(ctypes.Structure):
    """ep_rope: pair frequencies and layout of rotary positions (see make_rope)."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class KvGroups(ctypes.Structure):
    """ep_kv_groups: ranges of sequences that share their leading tokens."""
    _fields_ = [("group_off", ctypes.c_void_p), ("shared", ctypes.c_void_p),
                ("n_groups", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    # torch first: it loads its own HIP runtime, and the library's dependency
    # on libamdhip64.so.7 must resolve to that same, already-loaded copy
    # (two HIP runtimes in one process would not share devices or memory).
    global _torch
    import torch as _torch

    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, D, I64 = ctypes.c_void_p, ctypes.POINTER(Desc), ctypes.c_int64
    sig = {
        "ep_recv_bound": (ctypes.c_int64, [D]),
        "ep_capacity": (ctypes.c_int64, [D]),
        "ep_num_planes": (ctypes.c_int, [D]),
        "ep_row_bytes": (ctypes.c_int64, [D, ctypes.c_int]),
        "ep_plan_bytes": (ctypes.c_size_t, [D]),
        "ep_plan_views": (ctypes.c_int, [D, P, ctypes.POINTER(PlanView)]),
        "ep_plan": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch": (ctypes.c_int, [D, P, P, P, P, P, P, P]),
        "ep_dispatch_quant": (ctypes.c_int, [D, P, P, P, P, P, P, P]),
        "ep_dispatch_pack": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch_pack_quant": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch_transfer": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch_unpack": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch_recv": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch_send": (ctypes.c_int, [D, P, P, P, P, P, ctypes.c_int32, P, P]),
        "ep_dispatch_recv_split": (ctypes.c_int, [D, P, P, ctypes.c_int32, P, P, P, P]),
        "ep_dispatch_send_plan": (ctypes.c_int, [D, P, P, P, P]),
        "ep_dispatch_send_pack": (ctypes.c_int, [D, P, P, P, P, P, ctypes.c_int32, P]),
        "ep_dispatch_recv_plan": (ctypes.c_int, [D, P, P, P]),
        "ep_dispatch_recv_pull": (ctypes.c_int, [D, P, P, ctypes.c_int32, P, P, P]),
        "ep_expert_stub": (ctypes.c_int, [D, P, P, P, P, P]),
        "ep_combine": (ctypes.c_int, [D, P, P, P, P, P]),
        "ep_combine_presum": (ctypes.c_int, [D, P, P, P, P, P, P]),
        "ep_kv_plan": (ctypes.c_int64, [I64, I64, I64, P, I64, P, ctypes.c_int32, P, I64]),
        "ep_kv_push": (ctypes.c_int, [ctypes.c_int32, P, I64, I64, P, I64, P, I64, P, P, P]),
        "ep_kv_push_staged": (ctypes.c_int, [ctypes.c_int32, P, I64, I64, P, I64, P, I64, P,
                                             ctypes.c_int32, P, P, P]),
        "ep_kv_push_staged_static": (ctypes.c_int, [ctypes.c_int32, P, I64, I64, P, I64, P, I64,
                                                    ctypes.c_int32, P, P, P]),
        "ep_kv_pages_bytes": (ctypes.c_size_t, [ctypes.POINTER(KvPages), I64]),
        "ep_kv_extend": (ctypes.c_int, [ctypes.POINTER(KvPages), P, P, I64, P, P, P]),
        "ep_kv_fork": (ctypes.c_int, [ctypes.POINTER(KvPages), P, P, I64, P, P, P]),
        "ep_kv_free": (ctypes.c_int, [ctypes.POINTER(KvPages), P, I64, P, P, P]),
        "ep_kv_compact": (ctypes.c_int, [ctypes.POINTER(KvPages), P, P, P, P]),
        "ep_kv_copy_pages": (ctypes.c_int, [ctypes.POINTER(KvPages), P, P, I64, P, P, P]),
        "ep_rope_freqs": (ctypes.c_int, [ctypes.c_int32, ctypes.c_double, ctypes.c_int32,
                                         ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                         ctypes.c_double, P, ctypes.POINTER(ctypes.c_float)]),
        "ep_kv_append": (ctypes.c_int, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch),
                                        ctypes.POINTER(Rows), ctypes.c_int32,
                                        ctypes.POINTER(Rows), ctypes.POINTER(Rows),
                                        ctypes.POINTER(Rows), ctypes.POINTER(Rope), P, P]),
        "ep_kv_attend_bytes": (ctypes.c_size_t, [ctypes.POINTER(KvCache)] + [ctypes.c_int32] * 5),
        "ep_kv_attend": (ctypes.c_int, [ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch),
                                        ctypes.POINTER(KvGroups), ctypes.c_int32,
                                        ctypes.POINTER(Rows), ctypes.c_int32,
                                        ctypes.POINTER(Rows), P, ctypes.c_float, P, P, P]),
        "ep_probe_copy": (ctypes.c_int, [P, P, ctypes.c_size_t, P]),
        "ep_probe_pattern": (ctypes.c_int, [P, P, P, I64, I64, I64, I64, ctypes.c_int,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_int, I64, P]),
        "ep_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "ep_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
_INT32 = _torch.int32


def lib() -> ctypes.CDLL:
    return _lib


# ---------------------------------------------------------------------------
# Marshalling helpers
# ---------------------------------------------------------------------------

def make_desc(n_ranks, tokens, hidden, n_experts, topk,
              payload=EP_PAYLOAD_BF16, cap_rows=0) -> Desc:
    return Desc(n_ranks, tokens, hidden, n_experts, topk, payload, cap_rows)


def _addr(t) -> Optional[int]:
    """Address of a buffer: None, a raw device address, or a tensor, which
    must be contiguous (the library reads every buffer as dense row-major
    bytes; a strided view would be read as if it were dense)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError(f"buffer of shape {tuple(t.shape)} and strides {t.stride()} is not "
                         "contiguous: the library takes dense row-major buffers")
    return t.data_ptr()


def _planes(ts: Sequence) -> ctypes.Array:
    ts = list(ts) + [None] * (2 - len(ts))
    return (ctypes.c_void_p * 2)(*[_addr(t) for t in ts[:2]])


def _stream_finder(c):
    """A function that gives the handle of torch's current stream. `c`: torch's C module. Its short
    way to the handle is taken where it has one: building a torch.cuda.Stream takes 3 us of a call's
    10 to 17 on the host."""
    raw, device = (getattr(c, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is None or device is None:
        return lambda: _torch.cuda.current_stream().cuda_stream

    def find():
        if not _torch.cuda.is_initialized():
            _torch.cuda.init()
        return raw(device())
    return find


_current_stream = _stream_finder(_torch._C)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> int:
    if rc != EP_OK:
        raise EPError(rc, where, _lib.ep_last_error().decode())
    return rc


def status_string(code: int) -> str:
    return _lib.ep_status_string(code).decode()


def last_error() -> str:
    return _lib.ep_last_error().decode()


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def recv_bound(d: Desc) -> int:
    return int(_lib.ep_recv_bound(ctypes.byref(d)))


def capacity(d: Desc) -> int:
    return int(_lib.ep_capacity(ctypes.byref(d)))


def num_planes(d: Desc) -> int:
    return int(_lib.ep_num_planes(ctypes.byref(d)))


def row_bytes(d: Desc, plane: int) -> int:
    return int(_lib.ep_row_bytes(ctypes.byref(d), plane))


def plan_bytes(d: Desc) -> int:
    return int(_lib.ep_plan_bytes(ctypes.byref(d)))


def plan_views(d: Desc, plan_ws) -> PlanView:
    v = PlanView()
    _check(_lib.ep_plan_views(ctypes.byref(d), _addr(plan_ws), ctypes.byref(v)), "ep_plan_views")
    return v


def plan(d: Desc, topk_idx, plan_ws, status, stream=None) -> None:
    _check(_lib.ep_plan(ctypes.byref(d), _addr(topk_idx), _addr(plan_ws), _addr(status),
                        _stream(stream)), "ep_plan")


def dispatch(d: Desc, topk_idx, x: Sequence, plan_ws, send: Sequence, grouped: Sequence, status,
             stream=None) -> None:
    _check(_lib.ep_dispatch(ctypes.byref(d), _addr(topk_idx), _planes(x), _addr(plan_ws),
                            _planes(send), _planes(grouped), _addr(status), _stream(stream)),
           "ep_dispatch")


def dispatch_quant(d: Desc, topk_idx, x_bf16, plan_ws, send: Sequence, grouped: Sequence, status,
                   stream=None) -> None:
    _check(_lib.ep_dispatch_quant(ctypes.byref(d), _addr(topk_idx), _addr(x_bf16), _addr(plan_ws),
                                  _planes(send), _planes(grouped), _addr(status), _stream(stream)),
           "ep_dispatch_quant")


def dispatch_pack(d: Desc, x: Sequence, plan_ws, send: Sequence, stream=None) -> None:
    _check(_lib.ep_dispatch_pack(ctypes.byref(d), _planes(x), _addr(plan_ws), _planes(send),
                                 _stream(stream)), "ep_dispatch_pack")


def dispatch_pack_quant(d: Desc, x_bf16, plan_ws, send: Sequence, stream=None) -> None:
    _check(_lib.ep_dispatch_pack_quant(ctypes.byref(d), _addr(x_bf16), _addr(plan_ws), _planes(send),
                                       _stream(stream)), "ep_dispatch_pack_quant")


def dispatch_transfer(d: Desc, send: Sequence, plan_ws, recv: Sequence, stream=None) -> None:
    _check(_lib.ep_dispatch_transfer(ctypes.byref(d), _planes(send), _addr(plan_ws),
                                     _planes(recv), _stream(stream)), "ep_dispatch_transfer")


def dispatch_unpack(d: Desc, recv: Sequence, plan_ws, grouped: Sequence, stream=None) -> None:
    _check(_lib.ep_dispatch_unpack(ctypes.byref(d), _planes(recv), _addr(plan_ws),
                                   _planes(grouped), _stream(stream)), "ep_dispatch_unpack")


def dispatch_recv(d: Desc, send: Sequence, plan_ws, grouped: Sequence, stream=None) -> None:
    _check(_lib.ep_dispatch_recv(ctypes.byref(d), _planes(send), _addr(plan_ws),
                                 _planes(grouped), _stream(stream)), "ep_dispatch_recv")


def dispatch_send(d: Desc, topk_idx, x: Sequence, plan_ws, send: Sequence, priv: Sequence,
                  priv_rows: int, status, stream=None) -> None:
    _check(_lib.ep_dispatch_send(ctypes.byref(d), _addr(topk_idx), _planes(x), _addr(plan_ws),
                                 _planes(send), _planes(priv), int(priv_rows), _addr(status),
                                 _stream(stream)), "ep_dispatch_send")


def dispatch_recv_split(d: Desc, send: Sequence, priv: Sequence, priv_rows: int, plan_ws,
                        grouped: Sequence, status, stream=None) -> None:
    _check(_lib.ep_dispatch_recv_split(ctypes.byref(d), _planes(send), _planes(priv),
                                       int(priv_rows), _addr(plan_ws), _planes(grouped),
                                       _addr(status), _stream(stream)), "ep_dispatch_recv_split")


def dispatch_send_plan(d: Desc, topk_idx, plan_ws, status, stream=None) -> None:
    _check(_lib.ep_dispatch_send_plan(ctypes.byref(d), _addr(topk_idx), _addr(plan_ws),
                                      _addr(status), _stream(stream)), "ep_dispatch_send_plan")


def dispatch_send_pack(d: Desc, topk_idx, x: Sequence, plan_ws, send: Sequence, priv: Sequence,
                       priv_rows: int, stream=None) -> None:
    _check(_lib.ep_dispatch_send_pack(ctypes.byref(d), _addr(topk_idx), _planes(x),
                                      _addr(plan_ws), _planes(send), _planes(priv),
                                      int(priv_rows), _stream(stream)), "ep_dispatch_send_pack")


def dispatch_recv_plan(d: Desc, plan_ws, status, stream=None) -> None:
    _check(_lib.ep_dispatch_recv_plan(ctypes.byref(d), _addr(plan_ws), _addr(status),
                                      _stream(stream)), "ep_dispatch_recv_plan")


def dispatch_recv_pull(d: Desc, send: Sequence, priv: Sequence, priv_rows: int, plan_ws,
                       grouped: Sequence, stream=None) -> None:
    _check(_lib.ep_dispatch_recv_pull(ctypes.byref(d), _planes(send), _planes(priv),
                                      int(priv_rows), _addr(plan_ws), _planes(grouped),
                                      _stream(stream)), "ep_dispatch_recv_pull")


def priv_buffers(d: Desc, priv_rows: int, device="cuda") -> list:
    """Private regions of a split dispatch: per plane [N][N][P][row_p] bytes."""
    import torch
    N = d.n_ranks
    return [torch.empty((N, N, priv_rows, row_bytes(d, p)), dtype=torch.uint8, device=device)
            for p in range(num_planes(d))]


def expert_stub(d: Desc, grouped: Sequence, alpha, plan_ws, expert_out, stream=None) -> None:
    _check(_lib.ep_expert_stub(ctypes.byref(d), _planes(grouped), _addr(alpha), _addr(plan_ws),
                               _addr(expert_out), _stream(stream)), "ep_expert_stub")


def combine(d: Desc, expert_out, weights, plan_ws, out, stream=None) -> None:
    _check(_lib.ep_combine(ctypes.byref(d), _addr(expert_out), _addr(weights), _addr(plan_ws),
                           _addr(out), _stream(stream)), "ep_combine")


def combine_presum(d: Desc, expert_out, weights, plan_ws, partial, out, stream=None) -> None:
    _check(_lib.ep_combine_presum(ctypes.byref(d), _addr(expert_out), _addr(weights),
                                  _addr(plan_ws), _addr(partial), _addr(out), _stream(stream)),
           "ep_combine_presum")


class KvRegion(ctypes.Structure):
    """ep_kv_region: src_off, dst_off, bytes, first (int64 each)."""
    _fields_ = [("src_off", ctypes.c_int64), ("dst_off", ctypes.c_int64),
                ("bytes", ctypes.c_int64), ("first", ctypes.c_int64)]


def kv_plan(n_tokens: int, token_bytes: int, src_block_tokens: int, src_blocks,
            dst_block_tokens: int, dst_blocks, merge: bool = True):
    """Host-only region planner; returns an int64 numpy array [m, 4] of
    (src_off, dst_off, bytes, first)."""
    import numpy as np
    sb = np.ascontiguousarray(src_blocks, dtype=np.int32)
    db = np.ascontiguousarray(dst_blocks, dtype=np.int32)
    cap = max(int(n_tokens), 1)
    out = np.zeros((cap, 4), np.int64)
    m = _lib.ep_kv_plan(int(n_tokens), int(token_bytes), int(src_block_tokens),
                        sb.ctypes.data, int(dst_block_tokens), db.ctypes.data, int(bool(merge)),
                        out.ctypes.data, cap)
    if m < 0:
        raise EPError(int(m), "ep_kv_plan", _lib.ep_last_error().decode())
    return out[:m].copy()


def kv_push(ranks: int, regions, n_regions: int, total_bytes: int, src_pool, src_rank_bytes: int,
            dst_pool, dst_rank_bytes: int, notify, status, stream=None) -> None:
    _check(_lib.ep_kv_push(int(ranks), _addr(regions), int(n_regions), int(total_bytes),
                           _addr(src_pool), int(src_rank_bytes), _addr(dst_pool),
                           int(dst_rank_bytes), _addr(notify), _addr(status),
                           _stream(stream)), "ep_kv_push")


def kv_push_staged(ranks: int, regions, n_regions: int, total_bytes: int, src_pool,
                   src_rank_bytes: int, dst_pool, dst_rank_bytes: int, bounce, bounce_slots: int,
                   notify, status, stream=None) -> None:
    _check(_lib.ep_kv_push_staged(int(ranks), _addr(regions), int(n_regions), int(total_bytes),
                                  _addr(src_pool), int(src_rank_bytes), _addr(dst_pool),
                                  int(dst_rank_bytes), _addr(bounce), int(bounce_slots),
                                  _addr(notify), _addr(status), _stream(stream)),
           "ep_kv_push_staged")


def kv_push_staged_static(ranks: int, regions, n_regions: int, total_bytes: int, src_pool,
                          src_rank_bytes: int, dst_pool, dst_rank_bytes: int, bounce_slots: int,
                          notify, status, stream=None) -> None:
    _check(_lib.ep_kv_push_staged_static(int(ranks), _addr(regions), int(n_regions),
                                         int(total_bytes), _addr(src_pool), int(src_rank_bytes),
                                         _addr(dst_pool), int(dst_rank_bytes), int(bounce_slots),
                                         _addr(notify), _addr(status), _stream(stream)),
           "ep_kv_push_staged_static")


# ---------------------------------------------------------------------------
# Paged KV cache: page state, rotary append, attention
# ---------------------------------------------------------------------------

def _ints(t, shape, name: str):
    """Address of a contiguous int32 tensor of the given shape (None: any size)."""
    have = t.shape
    if have != shape and (len(have) != len(shape) or
                          any(n is not None and n != m for n, m in zip(shape, have))):
        raise ValueError(f"{name} has shape {tuple(have)}, not {shape}")
    if t.dtype is not _INT32:
        raise ValueError(f"{name} must be int32, not {t.dtype}")
    return t.data_ptr() if t.is_contiguous() else _addr(t)


def _word(t, name: str):
    """Address of a tensor of at least one int32, or None."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is not _INT32 or t.numel() < 1:
        raise ValueError(f"{name} must be int32 with at least one element, not {t.dtype} "
                         f"{tuple(t.shape)}")
    return t.data_ptr() if t.is_contiguous() else _addr(t)


def _room(ws, need: int):
    """Address of a workspace of at least `need` bytes (0: sizes that the library refuses). The
    library sees no more than the allocation around it, which may hold other tensors."""
    if ws is None or isinstance(ws, int):
        return ws
    if ws.nbytes < need:
        raise ValueError(f"ws holds {ws.nbytes} bytes, the call needs {need}")
    return ws.data_ptr() if ws.is_contiguous() else _addr(ws)


@functools.lru_cache(maxsize=4096)
def _pages_bytes(n_seqs: int, n_pages: int, m: int) -> int:
    """ep_kv_pages_bytes by what it depends on: a call to the library takes 1 us of the 5 that a
    page operation takes on the host."""
    g = KvPages(None, None, None, None, n_seqs, 1, n_pages, 1, 1, 0, 16, 16 * n_pages)
    return _lib.ep_kv_pages_bytes(ctypes.byref(g), m)


def _page_room(g: KvPages, m: int, ws):
    return _room(ws, _pages_bytes(g.n_seqs, g.n_pages, m))


def make_kv_pages(tables, lens, refs, pool, page_tokens: int) -> KvPages:
    """Page state from tables [n_seqs, max_pages], lens [n_seqs], refs [n_pages] (int32) and a
    contiguous pool [ranks, n_pages, ...]; all of them are read and changed in place."""
    seqs, n_pages = tables.shape[0], refs.shape[0]
    if pool.dim() < 3 or pool.shape[1] != n_pages:
        raise ValueError(f"pool has shape {tuple(pool.shape)}, not [ranks, {n_pages}, ...]")
    page_bytes = pool[0, 0].numel() * pool.element_size()
    g = KvPages(_ints(tables, (None, None), "tables"), _ints(lens, (seqs,), "lens"),
                _ints(refs, (None,), "refs"), _addr(pool), seqs, tables.shape[1], n_pages,
                int(page_tokens), pool.shape[0], 0, page_bytes, n_pages * page_bytes)
    g.tensors = (tables, lens, refs, pool)   # they live as long as the addresses are used
    return g


def kv_pages_bytes(g: KvPages, m: int) -> int:
    return int(_lib.ep_kv_pages_bytes(ctypes.byref(g), int(m)))


def kv_extend(g: KvPages, seqs, add, ws, status, stream=None) -> None:
    m = seqs.numel()
    _check(_lib.ep_kv_extend(ctypes.byref(g), _ints(seqs, (m,), "seqs"), _ints(add, (m,), "add"),
                             m, _page_room(g, m, ws), _word(status, "status"), _stream(stream)),
           "ep_kv_extend")


def kv_fork(g: KvPages, parents, children, ws, status, stream=None) -> None:
    m = parents.numel()
    _check(_lib.ep_kv_fork(ctypes.byref(g), _ints(parents, (m,), "parents"),
                           _ints(children, (m,), "children"), m, _page_room(g, m, ws),
                           _word(status, "status"), _stream(stream)), "ep_kv_fork")


def kv_free(g: KvPages, seqs, ws, status, stream=None) -> None:
    m = seqs.numel()
    _check(_lib.ep_kv_free(ctypes.byref(g), _ints(seqs, (m,), "seqs"), m, _page_room(g, m, ws),
                           _word(status, "status"), _stream(stream)), "ep_kv_free")


def kv_compact(g: KvPages, ws, status, n_live=None, stream=None) -> None:
    _check(_lib.ep_kv_compact(ctypes.byref(g), _word(n_live, "n_live"), _page_room(g, 0, ws),
                              _word(status, "status"), _stream(stream)), "ep_kv_compact")


def kv_copy_pages(g: KvPages, src, dst, ws, status, stream=None) -> None:
    m = src.numel()
    _check(_lib.ep_kv_copy_pages(ctypes.byref(g), _ints(src, (m,), "src"), _ints(dst, (m,), "dst"),
                                 m, _page_room(g, m, ws), _word(status, "status"),
                                 _stream(stream)), "ep_kv_copy_pages")


def _dtype(t, name: str) -> int:
    codes = {_torch.bfloat16: EP_DTYPE_BF16, _torch.float16: EP_DTYPE_F16,
             _torch.float8_e4m3fn: EP_DTYPE_E4M3}
    if t.dtype not in codes:
        raise ValueError(f"{name} has dtype {t.dtype}: bfloat16, float16 or float8_e4m3fn are taken")
    return codes[t.dtype]


def _row_strides(t, dims: int, name: str):
    """Element strides of rows whose last axis is dense."""
    st = t.stride()
    if len(st) != dims or (st[-1] != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} of shape {tuple(t.shape)} and strides {st}: {dims} axes, the last "
                         "one dense, are taken")
    return st


def make_kv_cache(k, v, k_scale=None, v_scale=None) -> KvCache:
    """One layer's cache from k and v [n_pages, page_tokens, n_heads, head_dim]: strided views of
    a pool, with equal strides. float8_e4m3fn ones take a float32 scale per head each."""
    st = _row_strides(k, 4, "k")
    _row_strides(v, 4, "v")
    if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
        raise ValueError("k and v must have equal shapes, strides and dtypes")
    es = k.element_size()
    for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if s is not None and (tuple(s.shape) != (k.shape[2],) or s.dtype != _torch.float32):
            raise ValueError(f"{name} must be float32 [{k.shape[2]}]")
    c = KvCache(k.data_ptr(), v.data_ptr(), _addr(k_scale), _addr(v_scale), st[0] * es,
                st[1] * es, st[2] * es, k.shape[0], k.shape[1], k.shape[2],
                k.shape[3], _dtype(k, "k"), 0)
    c.tensors = (k, v, k_scale, v_scale)
    return c


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: int = EP_ROPE_NONE,
               factor: float = 1.0, orig_tokens: float = 0.0, beta_fast: float = 32.0,
               beta_slow: float = 1.0):
    """Host-only pair frequencies: (float32 numpy array [rot_dim / 2], mscale)."""
    import numpy as np
    out = np.zeros(max(int(rot_dim) // 2, 1), np.float32)
    mscale = ctypes.c_float()
    _check(_lib.ep_rope_freqs(int(rot_dim), float(base), int(scaling), float(factor),
                              float(orig_tokens), float(beta_fast), float(beta_slow),
                              out.ctypes.data, ctypes.byref(mscale)), "ep_rope_freqs")
    return out, mscale.value


def make_rope(inv_freq, rot_dim: int, layout: int = EP_ROPE_HALF, mscale: float = 1.0) -> Rope:
    """Rotary positions from a float32 tensor of rot_dim / 2 frequencies."""
    if inv_freq.dtype != _torch.float32 or inv_freq.numel() != int(rot_dim) // 2:
        raise ValueError(f"inv_freq must be float32 [{int(rot_dim) // 2}]")
    r = Rope(_addr(inv_freq), int(rot_dim), int(layout), float(mscale), 0)
    r.tensors = (inv_freq,)
    return r


def _rows(t, name: str, dtype, shape) -> Rows:
    """Rows of 16-bit elements of the given dtype and shape."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, not {dtype} {tuple(shape)}")
    st = _row_strides(t, 3, name)
    return Rows(t.data_ptr(), 2 * st[0], 2 * st[1])


def _batch(tables, lens, q_off, n_tokens: int, dtype: int) -> KvBatch:
    seqs, max_pages = tables.shape
    return KvBatch(_ints(tables, (seqs, max_pages), "tables"), _ints(lens, (seqs,), "lens"),
                   None if q_off is None else _ints(q_off, (seqs + 1,), "q_off"), seqs, max_pages,
                   n_tokens, dtype)


def kv_append(cache: KvCache, tables, lens, q_off, q, k, v, q_out, rope, status,
              stream=None) -> None:
    """Rotate the new tokens' q into q_out (which may be q) and write their rotated k, and v, to
    the pages. q and q_out None: only k and v. rope None: no rotation. q_off None: one new token
    per sequence."""
    shape, dtype = k.shape, k.dtype
    if tuple(shape[1:]) != (cache.n_heads, cache.head_dim):
        raise ValueError(f"k has shape {tuple(shape)}, not [tokens, {cache.n_heads}, "
                         f"{cache.head_dim}]")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out must be given together")
    b = _batch(tables, lens, q_off, shape[0], _dtype(k, "k"))
    rq = ro = None
    heads = 0
    if q is not None:
        heads = q.shape[1]
        wide = (shape[0], heads, shape[2])
        rq, ro = _rows(q, "q", dtype, wide), _rows(q_out, "q_out", dtype, wide)
    _check(_lib.ep_kv_append(
        ctypes.byref(cache), ctypes.byref(b), rq, heads, _rows(k, "k", dtype, shape),
        _rows(v, "v", dtype, shape), ro, None if rope is None else ctypes.byref(rope),
        _word(status, "status"), _stream(stream)), "ep_kv_append")


def kv_attend_bytes(cache: KvCache, n_seqs: int, n_groups: int, n_tokens: int, n_heads: int,
                    max_new: int = 1) -> int:
    return int(_lib.ep_kv_attend_bytes(ctypes.byref(cache), int(n_seqs), int(n_groups),
                                       int(n_tokens), int(n_heads), int(max_new)))


def kv_attend(cache: KvCache, tables, lens, q_off, max_new: int, group_off, shared, q, out, lse,
              sm_scale: float, ws, status, stream=None) -> None:
    """Attention of the new tokens' q over their pages into out, and lse (or None). group_off and
    shared (or both None): ranges of sequences that share their leading tokens."""
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError(f"q has shape {tuple(shape)}, not [tokens, heads, {cache.head_dim}]")
    b = _batch(tables, lens, q_off, shape[0], _dtype(q, "q"))
    if (group_off is None) != (shared is None):
        raise ValueError("group_off and shared must be given together")
    groups, n = None, 0
    if shared is not None:
        n = shared.numel()
        groups = KvGroups(_ints(group_off, (n + 1,), "group_off"), _ints(shared, (n,), "shared"),
                          n, 0)
    if lse is not None and (lse.shape != shape[:2] or lse.dtype != _torch.float32):
        raise ValueError(f"lse must be float32 {tuple(shape[:2])}")
    need = 0   # an empty batch needs no workspace
    if shape[0] > 0 and b.n_seqs > 0:
        need = _lib.ep_kv_attend_bytes(ctypes.byref(cache), b.n_seqs, n, shape[0], shape[1],
                                       int(max_new))
    _check(_lib.ep_kv_attend(
        ctypes.byref(cache), ctypes.byref(b), None if groups is None else ctypes.byref(groups),
        int(max_new), _rows(q, "q", dtype, shape), shape[1], _rows(out, "out", dtype, shape),
        _addr(lse), float(sm_scale),
        _room(ws, need), _word(status, "status"), _stream(stream)), "ep_kv_attend")


def probe_copy(dst, src, nbytes: int, stream=None) -> None:
    _check(_lib.ep_probe_copy(_addr(dst), _addr(src), nbytes, _stream(stream)), "ep_probe_copy")


def probe_pattern(dst, src, table, rows: int, indexed_rows: int, row_bytes: int,
                  piece_bytes: int, fan_in: int = 1, in_flight: int = 0,
                  mode: int = EP_PROBE_COPY, flags: int = 0, waves: int = 0,
                  stream=None) -> None:
    """in_flight 0 means all fan_in rows at once (1 for a scatter)."""
    if not in_flight:
        in_flight = 1 if mode in (EP_PROBE_SCATTER, EP_PROBE_SCATTER_WIDE) else fan_in
    _check(_lib.ep_probe_pattern(_addr(dst), _addr(src), _addr(table), int(rows),
                                 int(indexed_rows), int(row_bytes), int(piece_bytes),
                                 int(fan_in), int(in_flight), int(mode), int(flags), int(waves),
                                 _stream(stream)), "ep_probe_pattern")


# ---------------------------------------------------------------------------
# Device buffers for one descriptor (torch allocations; plumbing only)
# ---------------------------------------------------------------------------

class Buffers:
    """Caller-owned device buffers of one dispatch/combine step."""

    def __init__(self, d: Desc, device="cuda", staged: bool = False):
        import torch
        self.desc = d
        N, T, H, R = d.n_ranks, d.tokens, d.hidden, d.topk
        cap = capacity(d)
        if cap < 0:
            raise EPError(EP_ERR_INVALID_ARG, "Buffers", last_error())
        self.cap = cap
        self.planes = num_planes(d)
        rows = [row_bytes(d, p) for p in range(self.planes)]
        u8 = torch.uint8
        self.idx = torch.empty((N, T, R), dtype=torch.int32, device=device)
        self.weights = torch.empty((N, T, R), dtype=torch.float32, device=device)
        self.x = [torch.empty((N, T, r), dtype=u8, device=device) for r in rows]
        self.send = [torch.empty((N, T * R, r), dtype=u8, device=device) for r in rows]
        self.grouped = [torch.empty((N, cap, r), dtype=u8, device=device) for r in rows]
        self.recv = ([torch.empty((N, cap, r), dtype=u8, device=device) for r in rows]
                     if staged else None)
        self.expert_out = torch.empty((N, cap, H), dtype=torch.int16, device=device)
        self.out = torch.empty((N, T, H), dtype=torch.int16, device=device)
        self.plan_ws = torch.empty(plan_bytes(d), dtype=u8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
