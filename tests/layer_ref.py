"""The operators around dispatch and combine in 64 bits, and the routing that their tests use."""
import math

import torch

import combine_ep_plan_amd as ep

BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
HALF = {BF: 2.0**-8, HF: 2.0**-11}        # half a step, relative
TINY = {BF: 2.0**-134, HF: 2.0**-25}      # half a step of the subnormals
NAMES = {ep.EP_ACT_NONE: "none", ep.EP_ACT_SILU: "silu", ep.EP_ACT_GELU: "gelu", ep.EP_ACT_SWIGLU: "swiglu"}


def norm(h, weight, eps):
    return h * weight / (h.square().mean(-1, keepdim=True) + eps).sqrt()


def norm_grad(dy, h, weight, dsum, eps):
    """dx and dweight by the formula."""
    var = h.square().mean(-1, keepdim=True) + eps
    g = dy * weight
    dx = g / var.sqrt() - h * (g * h).mean(-1, keepdim=True) / var**1.5
    return dx + dsum, (dy * h / var.sqrt()).reshape(-1, h.shape[-1]).sum(0)


def activate(z, act):
    if act == ep.EP_ACT_SWIGLU:
        gate, up = z.chunk(2, -1)
        return gate / (1 + torch.exp(-gate)) * up
    if act == ep.EP_ACT_SILU:
        return z / (1 + torch.exp(-z))
    if act == ep.EP_ACT_GELU:
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z


def activate_grad(z, d, act):
    if act in (ep.EP_ACT_SILU, ep.EP_ACT_SWIGLU):
        gate, up = z.chunk(2, -1) if act == ep.EP_ACT_SWIGLU else (z, None)
        s = torch.sigmoid(gate)
        slope = s + gate * s * torch.sigmoid(-gate)
        return d * slope if up is None else torch.cat([d * up * slope, d * gate * s], -1)
    if act == ep.EP_ACT_GELU:
        return d * (0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    return d


def ids(n, t, e, r, seed, only=None):
    """Distinct expert ids per token, int32 [n, t, r]; `only`: from these experts."""
    g = torch.Generator().manual_seed(seed)
    pool = torch.tensor(list(range(e)) if only is None else only)
    order = torch.rand((n * t, len(pool)), generator=g).argsort(1)[:, :r]
    return pool[order].to(torch.int32).view(n, t, r)


class Routed:
    """A plan on the GPU and, by sequential Python, the rows it stands for."""

    def __init__(self, n, t, e, r, idx, hidden=8, cap=0, payload=ep.EP_PAYLOAD_BF16):
        self.desc = ep.make_desc(n, t, hidden, e, r, payload, cap)
        self.cap = ep.capacity(self.desc)
        self.rows = n * self.cap
        self.plan = torch.zeros(ep.plan_bytes(self.desc), dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ep.plan(self.desc, idx.cuda(), self.plan, self.status)
        local = e // n
        members = [[] for _ in range(e)]
        for slot, x in enumerate(idx.flatten().tolist()):
            if 0 <= x < e:
                members[x].append(slot)
        self.row = torch.full((n * t * r,), -1, dtype=torch.long)   # of each slot
        self.groups = []                                            # (first, rows) of each expert
        for d in range(n):
            at = 0
            for j in range(local):
                slots = members[d * local + j]
                lo, hi = min(at, self.cap), min(at + len(slots), self.cap)
                self.groups.append((d * self.cap + lo, hi - lo))
                for i, s in enumerate(slots):
                    if at + i < self.cap:
                        self.row[s] = d * self.cap + at + i
                at += len(slots)
        self.owned = torch.zeros(self.rows, dtype=torch.bool)
        for a, m in self.groups:
            self.owned[a:a + m] = True


class Dense:
    """One expert per rank that owns all its rows."""

    def __init__(self, n, rows):
        self.desc = ep.make_desc(n, rows, 8, n, 1, cap_rows=rows)
        self.cap, self.rows, self.plan = rows, n * rows, None
        self.groups = [(d * rows, rows) for d in range(n)]
        self.owned = torch.ones(self.rows, dtype=torch.bool)


def check(got, want, tol, what):
    """Every element within its own tolerance; NaN where the definition has one."""
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           [(float(got[tuple(i)]), float(want[tuple(i)]), float(tol[tuple(i)]))
                            for i in bad.nonzero()[:4].tolist()])


def guarded(shape, dtype, fill=7.0):
    """A tensor between two guards of at least 64 KB, and a function that asserts that the guards are whole."""
    count = 1
    for s in shape:
        count *= s
    size = torch.empty(0, dtype=dtype).element_size()
    edge = 65536 // size
    whole = torch.full((count + 2 * edge,), fill, dtype=dtype, device="cuda")

    def check():
        assert (whole[:edge] == fill).all() and (whole[-edge:] == fill).all()
    return whole[edge:-edge].view(shape), check
