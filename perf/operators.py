"""Cases of the paged KV-cache operators: page management, rotary append, shared-prefix attention.

Each case describes one pass of one operator as a serving loop calls it:

* ``pages``: a sampler finishes its requests, admits new prompts and forks each into several samples
  (free, extend, fork); ``compact`` squeezes a fragmented pool; ``copy`` duplicates given pages.
* ``append``: the new tokens' q and k are rotated, k and v are written to the sequences' pages.
* ``attend``: the new tokens attend to their pages; the sequences of a group share their leading pages.

With ``own`` false, ``run`` computes the pass from elementary torch operations; with ``own`` true it calls
the library. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _pages(name, ranks, pages, page_tokens, token_bytes, live, max_pages, prompts, children, prompt):
    return dict(name=name, op="pages", ranks=ranks, pages=pages, page_tokens=page_tokens, token_bytes=token_bytes,
                live=live, max_pages=max_pages, prompts=prompts, children=children, prompt=prompt)


def _append(name, seqs, new, context, heads, kv_heads, dim, rot, layout, scaling, dtype, cache, page_tokens, layers):
    return dict(name=name, op="append", seqs=seqs, new=new, context=context, heads=heads, kv_heads=kv_heads, dim=dim,
                rot=rot, layout=layout, scaling=scaling, dtype=dtype, cache=cache, page_tokens=page_tokens,
                layers=layers)


def _attend(name, groups, per, prefix, suffix, new, heads, kv_heads, dim, dtype, cache, page_tokens, layers):
    return dict(name=name, op="attend", groups=groups, per=per, prefix=prefix, suffix=suffix, new=new, heads=heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, cache=cache, page_tokens=page_tokens, layers=layers)


def listed():
    return [
        # One prompt of the smallest KV workload, sampled four times: launch latency.
        _pages("pages_tiny", 2, 120, 4, 64, 3, 16, 1, 4, 37),
        # A sampling service: 16 prompts of up to 4096 tokens, eight samples each, beside 32 running requests.
        _pages("pages_sampling", 2, 8192, 16, 4096, 32, 288, 16, 8, 4096),
        # A fragmented pool of 512 KiB pages (16 tokens of 64 layers) squeezed before it is shrunk.
        dict(name="compact_large", op="compact", ranks=2, pages=2048, page_tokens=16, token_bytes=32768, live=64,
             max_pages=64, fill=0.5),
        # Pages of one token, 32 KiB each, duplicated by a given list.
        dict(name="copy_page1", op="copy", ranks=1, pages=16384, page_tokens=1, token_bytes=32768, pairs=4096),
        # One decoding sequence on one of eight ranks: launch latency.
        _append("append_one", 1, 1, 500, 5, 1, 128, 128, "half", "none", "bf16", "bf16", 16, 4),
        # A decode batch at far positions under YaRN scaling, the pool token-major over all layers.
        _append("append_decode", 128, 1, 131072, 40, 8, 128, 128, "half", "yarn", "bf16", "bf16", 16, 1),
        # Ragged prompts, a partly rotated head in interleaved pairs, an fp8 cache.
        _append("append_prompts", 37, 801, 0, 32, 8, 128, 64, "interleaved", "linear", "bf16", "fp8", 16, 1),
        # One decoding sequence with a short context: launch latency.
        _attend("attend_one", 1, 1, 0, 300, 1, 40, 8, 128, "bf16", "bf16", 16, 1),
        # Samples of a 16k prompt: the prefix is read once for 128 sequences.
        _attend("attend_samples", 1, 128, 16384, 1024, 1, 40, 8, 128, "bf16", "bf16", 16, 1),
        # One rank of eight (one KV head), pages holding all 64 layers of a token, four prompts of eight samples.
        _attend("attend_rank", 4, 8, 4096, 256, 1, 5, 1, 128, "bf16", "bf16", 16, 64),
        # Speculative tokens, one head per KV head, head size 64, pages of one token, fp16 queries over an fp8 cache.
        _attend("attend_drafts", 6, 5, 1500, 333, 4, 16, 16, 64, "fp16", "fp8", 1, 1),
        # Questions asked on a shared document: ragged prompts of up to 256 tokens behind an 8k prefix.
        _attend("attend_questions", 2, 6, 8192, 256, 256, 40, 8, 128, "bf16", "bf16", 16, 1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["pages", "compact", "copy", "append", "append", "attend", "attend", "attend"])
    if op in ("pages", "compact", "copy"):
        page_tokens = rng.choice([1, 4, 5, 16, 32, 64])
        ranks, pages = rng.randint(1, 4), _log(rng, 120, 16384)
        page_bytes = _log(rng, 256, min(1 << 19, (1 << 30) // (ranks * pages)))
        token_bytes = max(16, page_bytes // page_tokens // 16 * 16)
        if op == "copy":
            return dict(op="copy", ranks=ranks, pages=pages, page_tokens=page_tokens, token_bytes=token_bytes,
                        pairs=_log(rng, 1, pages // 3))
        if op == "compact":
            live = _log(rng, 1, 64)
            return dict(op="compact", ranks=ranks, pages=pages, page_tokens=page_tokens, token_bytes=token_bytes,
                        live=live, max_pages=max(1, pages // live), fill=round(rng.uniform(0.1, 0.9), 3))
        prompts, children, live = _log(rng, 1, 16), _log(rng, 1, 8), _log(rng, 1, 32)
        most = max(1, (pages // 2 - prompts * (children + 1)) // prompts)  # pages of one prompt
        most = min(most, 512)
        prompt = _log(rng, 1, most * page_tokens)
        while prompts * (children + 1 + -(-prompt // page_tokens)) > pages // 2 - 2:
            children, prompts = max(1, children // 2), max(1, prompts - 1)
            prompt = max(1, prompt // 2)
        return {k: v for k, v in _pages("", ranks, pages, page_tokens, token_bytes, live,
                                        max(-(-prompt // page_tokens) + 3, pages // 2 // live), prompts, children,
                                        prompt).items() if k != "name"}
    kv_heads, share = rng.choice([1, 2, 8, 16]), rng.choice([1, 2, 3, 5, 8])
    heads = kv_heads * share
    dim, dtype = rng.choice([64, 80, 96, 128, 128, 256]), rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "fp8"])
    page_tokens, layers = rng.choice([1, 7, 16, 16, 64]), rng.choice([1, 1, 3])
    if op == "append":
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        seqs, new = (_log(rng, 1, 256), 1) if rng.random() < 0.5 else (_log(rng, 1, 40), _log(rng, 2, 800))
        while seqs * new * (heads + kv_heads) * dim > 16384 * 48 * 128 or seqs * new * layers > 40000:
            seqs, new = max(1, seqs // 2), max(1, new // 2)
        context = _log(rng, 1, 131072)
        if seqs * (context // page_tokens) > 1 << 21:
            context = max(1, (1 << 21) // seqs * page_tokens)
        case = _append("", seqs, new, context, heads, kv_heads, dim, rot, rng.choice(["half", "interleaved"]),
                       rng.choice(["none", "linear", "ntk", "yarn"]), dtype, cache, page_tokens, layers)
    else:
        groups, per = _log(rng, 1, 8), _log(rng, 1, 64)
        prefix = 0 if rng.random() < 0.2 else _log(rng, 1, 16384)
        new = 1 if rng.random() < 0.6 else _log(rng, 2, 8) if rng.random() < 0.6 else _log(rng, 9, 200)
        suffix = max(new, _log(rng, 1, 1024))
        case = _attend("", groups, per, prefix, suffix, new, heads, kv_heads, dim, dtype, cache, page_tokens, layers)
        # The plain form holds a score for each row and key in 32 bits, and K and V of every suffix.
        while (groups * per * new * heads * (prefix + suffix) > 3e8 or work(case)["flops"] > 1.5e11 or
               groups * (prefix + per * suffix) * kv_heads * dim * layers > 3e8):
            case["per"] = per = max(1, per * 2 // 3)
            case["prefix"] = prefix = prefix * 2 // 3
            case["new"] = new = max(1, new * 2 // 3)
            case["suffix"] = suffix = max(new, suffix * 2 // 3)
    return {k: v for k, v in case.items() if k != "name"}


def _spread(lo, hi, n):
    """n whole numbers from lo to hi in even steps (hi first): the same sum for every seed."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _append_new(c):
    return _spread(1, c["new"], c["seqs"])


def _attend_lens(c):
    """Shared tokens of each group, tokens behind them and new tokens of each sequence (in even steps, unshuffled)."""
    b = c["groups"] * c["per"]
    new = _spread(1, c["new"], b)
    return _spread((c["prefix"] + 1) // 2, c["prefix"], c["groups"]), \
        [max(s, n) for s, n in zip(_spread(1, c["suffix"], b), new)], new


def _page_bytes(c):
    return c["page_tokens"] * c["token_bytes"]


def _row_elems(c):
    return c["heads"] * c["dim"], c["kv_heads"] * c["dim"]


def work(case):
    c, op = case, case["op"]
    if op == "copy":
        return {"bytes": 2 * c["pairs"] * c["ranks"] * _page_bytes(c) + 8 * c["pairs"], "flops": 0}
    if op == "compact":
        moved = c["pages"] * c["fill"] * (1 - c["fill"])
        return {"bytes": 2 * moved * c["ranks"] * _page_bytes(c) + 8 * c["pages"] * (1 + c["fill"]), "flops": 0}
    if op == "pages":
        n = [-(-p // c["page_tokens"]) for p in _spread(1, c["prompt"], c["prompts"])]
        part = sum(p % c["page_tokens"] > 0 for p in _spread(1, c["prompt"], c["prompts"])) * c["children"]
        rows = sum(n) * (1 + c["children"])  # table entries: read and cleared, written again
        return {"bytes": 2 * part * c["ranks"] * _page_bytes(c) + 12 * rows + 8 * c["pages"], "flops": 0}
    es = 1 if c["cache"] == "fp8" else 2
    q, kv = _row_elems(c)
    if op == "append":
        t = sum(_append_new(c))
        pairs = t * (c["heads"] + c["kv_heads"]) * c["rot"] // 2
        return {"bytes": t * (2 * 2 * q + 2 * kv * (2 + es)) + 12 * c["seqs"] + 2 * c["rot"], "flops": 6 * pairs}
    pre, suf, new = _attend_lens(c)
    t = sum(new)
    seen = sum(n * (pre[b // c["per"]] + s) - n * (n - 1) // 2 for b, (s, n) in enumerate(zip(suf, new)))
    return {"bytes": (sum(pre) + sum(suf)) * 2 * kv * es + t * (2 * 2 * q + 4 * c["heads"]),
            "flops": 4 * c["dim"] * c["heads"] * seen}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pool(c, g):
    words = _page_bytes(c) // 8
    return torch.randint(-2**62, 2**62, (c["ranks"], c["pages"], words), dtype=torch.int64, device=DEV, generator=g)


def _live_tables(c, g, rng, seqs, counts):
    """Tables of the live sequences: pages anywhere in the pool; every second one shares the leading half of the
    sequence before it, as a fork leaves them."""
    tables = torch.full((seqs, c["max_pages"]), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(seqs, dtype=torch.int32, device=DEV)
    perm = torch.randperm(c["pages"], device=DEV, generator=g).to(torch.int32)
    at = 0
    for b, n in enumerate(counts):
        keep = min(n - 1, counts[b - 1] // 2) if b % 2 else 0
        tables[b, :keep] = tables[b - 1, :keep]
        tables[b, keep:n] = perm[at:at + n - keep]
        at += n - keep
        lens[b] = n * c["page_tokens"] - rng.randrange(c["page_tokens"])
    refs = torch.zeros(c["pages"] + 1, dtype=torch.int32, device=DEV)
    refs.index_add_(0, tables.flatten().long() % (c["pages"] + 1), torch.ones_like(tables.flatten()))
    return tables, lens, refs[:-1].clone()


def _prepare_pages(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    s = {"case": c, "pool": _pool(c, g), "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if c["op"] == "copy":
        perm = torch.randperm(c["pages"], device=DEV, generator=g).to(torch.int32)
        s["src"], s["dst"] = perm[:c["pairs"]].clone(), perm[c["pairs"]:2 * c["pairs"]].clone()
        s["tables"], s["lens"], s["refs"] = _ints([[-1]]), _ints([0]), _ints([1] * c["pages"])
        m = c["pairs"]
    elif c["op"] == "compact":
        most = min(c["max_pages"], max(1, int(2 * c["pages"] * c["fill"] / c["live"])))
        counts = [max(1, n) for n in _spread(max(1, most // 4), most, c["live"])]
        rng.shuffle(counts)
        while sum(counts) > c["pages"]:
            counts.pop()
        s["start"], s["lens"], s["start_refs"] = _live_tables(c, g, rng, c["live"], counts)
        # Pages that a prefix store holds, so that the pool is filled as stated.
        spare = int(c["pages"] * c["fill"]) - int((s["start_refs"] > 0).sum())
        if spare > 0:
            idle = (s["start_refs"] == 0).nonzero()[:, 0]
            s["start_refs"][idle[torch.randperm(len(idle), device=DEV, generator=g)[:spare]]] = 1
        s["tables"], s["refs"] = s["start"].clone(), s["start_refs"].clone()
        m = 0
    else:
        n, k = c["prompts"], c["children"]
        most = max(1, min(c["max_pages"], c["pages"] // 2 // c["live"]))
        counts = _spread(1, most, c["live"])
        rng.shuffle(counts)
        seqs = c["live"] + n * (k + 1)
        s["tables"], s["lens"], s["refs"] = _live_tables(c, g, rng, seqs, counts)
        slots = list(range(c["live"], seqs))
        rng.shuffle(slots)
        add = _spread(1, c["prompt"], n)
        rng.shuffle(add)
        s["slots"], s["add"], s["prompts"] = _ints(slots), _ints(add), _ints(slots[:n])
        s["parents"], s["children"] = _ints([p for p in slots[:n] for _ in range(k)]), _ints(slots[n:])
        m = len(slots)
    if own:
        import combine_ep_plan_amd as ep
        s["ep"] = ep
        s["pages"] = ep.make_kv_pages(s["tables"], s["lens"], s["refs"], s["pool"], c["page_tokens"])
        s["ws"] = torch.empty(ep.kv_pages_bytes(s["pages"], m), dtype=torch.uint8, device=DEV)
    return s


def _rope_freqs(rot, scaling):
    """Pair frequencies and the factor of the rotated values, as 64-bit numbers rounded once to 32 bits."""
    base, factor, orig = 10000.0, 8.0, 16384
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base *= factor ** (rot / (rot - 2)) if rot > 2 else 1.0
    inv = base ** (-2 * i / rot)
    if scaling == "linear":
        inv = inv / factor
    if scaling != "yarn":
        return inv.float(), 1.0
    at = [rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return (inv / factor * ramp + inv * (1 - ramp)).float(), 0.1 * math.log(factor) + 1


def _cache(c, g, total_pages):
    """K and V of one layer in a pool whose pages hold all layers of a token."""
    shape = (total_pages, c["page_tokens"], c["layers"], 2, c["kv_heads"], c["dim"])
    if c["cache"] == "fp8":
        pool = torch.empty(shape, dtype=DTYPES["fp8"], device=DEV)
        scales = [torch.rand(c["kv_heads"], device=DEV, generator=g) * 0.01 + 0.005 for _ in range(2)]
    else:
        pool = torch.empty(shape, dtype=DTYPES[c["cache"]], device=DEV)
        scales = [None, None]
    layer = c["layers"] // 2
    for part in (0, 1):
        x = torch.randn(shape[:2] + shape[4:], device=DEV, generator=g)
        if scales[part] is not None:
            x = (x / scales[part][:, None]).clamp_(-448, 448)
        pool[:, :, layer, part] = x.to(pool.dtype)
    return pool[:, :, layer, 0], pool[:, :, layer, 1], scales


def _offsets(new):
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    return _ints(off)


def _prepare_append(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    new = _append_new(c)
    rng.shuffle(new)
    bt = c["page_tokens"]
    lens = [rng.randint(c["context"] // 2, c["context"]) + n for n in new]
    # Only the pages that the new tokens reach are in the pool: the contexts before them share page 0.
    tables = torch.zeros((c["seqs"], -(-max(lens) // bt)), dtype=torch.int32, device=DEV)
    first = [(n - k) // bt for n, k in zip(lens, new)]
    count = [-(-n // bt) - f for n, f in zip(lens, first)]
    total = 1 + sum(count)
    ids = (1 + torch.randperm(total - 1, device=DEV, generator=g)).to(torch.int32)
    at = 0
    for b, (f, n) in enumerate(zip(first, count)):
        tables[b, f:f + n] = ids[at:at + n]
        at += n
    k_cache, v_cache, scales = _cache(c, g, total)
    t = sum(new)
    # q, k and v as one projection leaves them, side by side in a row.
    qkv = torch.randn((t, c["heads"] + 2 * c["kv_heads"], c["dim"]), device=DEV, generator=g).to(DTYPES[c["dtype"]])
    q, k, v = qkv.split([c["heads"], c["kv_heads"], c["kv_heads"]], 1)
    inv, mscale = _rope_freqs(c["rot"], c["scaling"])
    s = {"case": c, "tables": tables, "lens": _ints(lens), "q_off": _offsets(new), "q": q, "k": k, "v": v,
         "k_cache": k_cache, "v_cache": v_cache, "scales": scales, "inv": inv.to(DEV), "mscale": mscale,
         "q_out": torch.empty(q.shape, dtype=q.dtype, device=DEV),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if own:
        import combine_ep_plan_amd as ep
        s["ep"] = ep
        s["cache"] = ep.make_kv_cache(k_cache, v_cache, *scales)
        s["rope"] = ep.make_rope(s["inv"], c["rot"],
                                 ep.EP_ROPE_HALF if c["layout"] == "half" else ep.EP_ROPE_INTERLEAVED, mscale)
    return s


def _prepare_attend(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    bt, per, groups = c["page_tokens"], c["per"], c["groups"]
    pre, suf, new = _attend_lens(c)
    order = list(range(groups * per))
    rng.shuffle(order)
    # A sequence keeps its own suffix and new tokens; which group it is in follows from its place.
    both = [(suf[b], new[b]) for b in order] if groups == 1 else list(zip(suf, new))
    suf, new = [x for x, _ in both], [y for _, y in both]
    lens = [pre[b // per] + suf[b] for b in range(groups * per)]
    tables = torch.full((groups * per, -(-max(lens) // bt)), -1, dtype=torch.int32, device=DEV)
    total = sum(-(-p // bt) for p in pre) + sum(-(-n // bt) - pre[b // per] // bt for b, n in enumerate(lens))
    ids = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    at = 0
    for j in range(groups):
        full = pre[j] // bt  # whole pages are shared; a sequence has its own copy of the page that is partly shared
        tables[j * per:(j + 1) * per, :full] = ids[at:at + full]
        at += full
        for b in range(j * per, (j + 1) * per):
            n = -(-lens[b] // bt) - full
            tables[b, full:full + n] = ids[at:at + n]
            at += n
    k_cache, v_cache, scales = _cache(c, g, total)
    shared = [p // bt * bt for p in pre]
    t = sum(new)
    q = (torch.randn((t, c["heads"], c["dim"]), device=DEV, generator=g) * 1.5).to(DTYPES[c["dtype"]])
    s = {"case": c, "tables": tables, "lens": _ints(lens), "q_off": _offsets(new), "q": q, "new": max(new),
         "k_cache": k_cache, "v_cache": v_cache, "scales": scales, "shared": _ints(shared),
         "group_off": _ints([per * j for j in range(groups + 1)]), "most": (max(shared), max(
             n - shared[b // per] for b, n in enumerate(lens))), "scale": c["dim"] ** -0.5,
         "out": torch.empty_like(q), "lse": torch.empty((t, c["heads"]), dtype=torch.float32, device=DEV),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if own:
        import combine_ep_plan_amd as ep
        s["ep"] = ep
        s["cache"] = ep.make_kv_cache(k_cache, v_cache, *scales)
        s["ws"] = torch.empty(ep.kv_attend_bytes(s["cache"], groups * per, groups, t, c["heads"], s["new"]),
                              dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    if case["op"] == "append":
        return _prepare_append(case, seed)
    if case["op"] == "attend":
        return _prepare_attend(case, seed)
    return _prepare_pages(case, seed)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_free(s, seqs):
    bt, rows = s["case"]["page_tokens"], s["tables"][seqs]
    used = torch.arange(rows.shape[1], device=DEV) < ((s["lens"][seqs] + bt - 1) // bt)[:, None]
    s["refs"].index_add_(0, torch.where(used, rows, 0).flatten(), -used.flatten().to(torch.int32))
    s["tables"][seqs] = -1
    s["lens"][seqs] = 0


def _free_pages(s):
    """Page ids, the free ones first, ascending."""
    return torch.sort((s["refs"] > 0).to(torch.int8), stable=True)[1].to(torch.int32)


def _plain_extend(s, seqs, add):
    bt, rows, n = s["case"]["page_tokens"], s["tables"][seqs], s["lens"][seqs]
    have, want = (n + bt - 1) // bt, (n + add + bt - 1) // bt
    col = torch.arange(rows.shape[1], device=DEV)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    rank = (fresh.flatten().cumsum(0) - 1).view_as(rows).clamp(min=0)
    page = _free_pages(s)[rank]
    s["tables"][seqs] = torch.where(fresh, page, rows)
    s["refs"].index_add_(0, torch.where(fresh, page, 0).flatten(), fresh.flatten().to(torch.int32))
    s["lens"][seqs] = n + add


def _plain_fork(s, parents, children):
    bt, rows, n = s["case"]["page_tokens"], s["tables"][parents], s["lens"][parents]
    full, part = n // bt, n % bt > 0
    page = _free_pages(s)[(part.cumsum(0) - 1).clamp(min=0)]
    col = torch.arange(rows.shape[1], device=DEV)
    shares, last = col < full[:, None], (col == full[:, None]) & part[:, None]
    s["tables"][children] = torch.where(shares, rows, torch.where(last, page[:, None], -1))
    s["lens"][children] = n
    s["refs"].index_add_(0, torch.where(shares, rows, 0).flatten(), shares.flatten().to(torch.int32))
    s["refs"].index_add_(0, torch.where(part, page, 0), part.to(torch.int32))
    src = rows.gather(1, torch.where(part, full, 0).long()[:, None])[:, 0]
    s["pool"][:, torch.where(part, page, src).long()] = s["pool"][:, src.long()]


def _plain_compact(s):
    live, at = s["refs"] > 0, torch.arange(s["refs"].numel(), device=DEV)
    count = live.sum()
    src, dst = (live & (at >= count)).nonzero()[:, 0], (~live & (at < count)).nonzero()[:, 0]
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["tables"].copy_(torch.where(s["tables"] >= 0, to[s["tables"].clamp(min=0)], s["tables"]))
    s["pool"][:, dst] = s["pool"][:, src]
    s["refs"][dst] = s["refs"][src]
    s["refs"][src] = 0


def _rows_of(s, q_off, lens):
    """Sequence and position of every new token."""
    i = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(q_off, i, right=True) - 1
    return b, lens[b].long() - q_off[b + 1].long() + i


def _rotate(x, cos, sin, rot, layout):
    x = x.float()
    y, keep = x[..., :rot], x[..., rot:]
    a, b = (y[..., :rot // 2], y[..., rot // 2:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y, keep], -1)


def _store(cache, page, slot, x, scale):
    if scale is not None:
        x = (x.float() / scale[:, None]).clamp(-448, 448)
    cache.view(torch.uint8).index_put_((page, slot), x.to(cache.dtype).view(torch.uint8))


def _plain_append(s):
    c = s["case"]
    b, pos = _rows_of(s, s["q_off"], s["lens"])
    angle = pos.double()[:, None] * s["inv"].double()
    cos, sin = ((f(angle) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))
    q = _rotate(s["q"], cos, sin, c["rot"], c["layout"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, c["rot"], c["layout"])
    page, slot = s["tables"][b, pos // c["page_tokens"]].long(), pos % c["page_tokens"]
    _store(s["k_cache"], page, slot, k, s["scales"][0])
    _store(s["v_cache"], page, slot, s["v"], s["scales"][1])
    return q


def _gather(cache, scale, tables, first, count, bt):
    """Rows [n, count, heads, dim] in 32 bits: `count` tokens from `first` of each table."""
    t = first[:, None] + torch.arange(count, device=DEV)
    page = tables.gather(1, (t // bt).clamp(max=tables.shape[1] - 1)).clamp(min=0).long()
    x = cache.view(torch.uint8)[page, t % bt].view(cache.dtype).float()
    return x if scale is None else x * scale[:, None]


def _plain_attend(s):
    """Scores of every row against its group's prefix and its own suffix, one softmax over both."""
    c, per, groups = s["case"], s["case"]["per"], s["case"]["groups"]
    heads, kv, d, bt = c["heads"], c["kv_heads"], c["dim"], c["page_tokens"]
    share, most_p, most_s, new = heads // kv, s["most"][0], s["most"][1], s["new"]
    lens, shared = s["lens"].long(), s["shared"].long().repeat_interleave(per)
    b, pos = _rows_of(s, s["q_off"], s["lens"])
    row = torch.arange(b.numel(), device=DEV) - s["q_off"][b]
    # Rows padded to [sequences, new, ...].
    q = torch.zeros((groups * per, new, kv, share, d), device=DEV)
    q[b, row] = s["q"].float().view(-1, kv, share, d)
    q = q.permute(0, 2, 3, 1, 4).contiguous() * s["scale"]  # [sequence, kv head, share, new, dim]
    last = torch.zeros((groups * per, new), dtype=torch.long, device=DEV)
    last[b, row] = pos
    zero = torch.zeros(groups, dtype=torch.long, device=DEV)
    kp, vp = (_gather(x, y, s["tables"][::per], zero, most_p, bt).permute(0, 2, 1, 3).contiguous()
              for x, y in zip((s["k_cache"], s["v_cache"]), s["scales"]))
    ks, vs = (_gather(x, y, s["tables"], shared, most_s, bt).permute(0, 2, 1, 3).contiguous()
              for x, y in zip((s["k_cache"], s["v_cache"]), s["scales"]))
    by_group = q.view(groups, per, kv, share * new, d).transpose(1, 2).reshape(groups, kv, per * share * new, d)
    sp = (by_group @ kp.transpose(2, 3).contiguous()).view(groups, kv, per, share, new, most_p).transpose(1, 2)
    ss = q.reshape(groups * per, kv, share * new, d) @ ks.transpose(2, 3).contiguous()
    score = torch.cat([sp.reshape(groups * per, kv, share, new, most_p), ss.view(-1, kv, share, new, most_s)], -1)
    at_p, at_s = torch.arange(most_p, device=DEV), torch.arange(most_s, device=DEV)
    key = torch.cat([at_p.expand(groups * per, -1), shared[:, None] + at_s], 1)
    valid = torch.cat([at_p < shared[:, None], at_s < (lens - shared)[:, None]], 1)
    see = valid[:, None] & (key[:, None] <= last[..., None])
    score = score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    pp = p[..., :most_p].reshape(groups, per, kv, share * new, most_p).transpose(1, 2)
    pp = pp.reshape(groups, kv, per * share * new, most_p)
    o = (pp @ vp).view(groups, kv, per, share * new, d).transpose(1, 2).reshape(groups * per, kv, share * new, d)
    o = o + p[..., most_p:].reshape(groups * per, kv, share * new, most_s) @ vs
    o = (o.view(groups * per, kv, share, new, d) / total).permute(0, 3, 1, 2, 4)[b, row]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[b, row]
    return o.reshape(-1, heads, d).to(s["q"].dtype), lse.reshape(-1, heads)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_pages(s):
    if own:
        s["ep"].kv_free(s["pages"], s["slots"], s["ws"], s["status"])
        s["ep"].kv_extend(s["pages"], s["prompts"], s["add"], s["ws"], s["status"])
        s["ep"].kv_fork(s["pages"], s["parents"], s["children"], s["ws"], s["status"])
    else:
        _plain_free(s, s["slots"])
        _plain_extend(s, s["prompts"], s["add"])
        _plain_fork(s, s["parents"], s["children"])
    return {"tables": s["tables"], "lens": s["lens"], "refs": s["refs"], "pool": s["pool"]}


def _run_compact(s):
    # The fragmented tables again, so that every pass moves the same pages.
    s["tables"].copy_(s["start"])
    s["refs"].copy_(s["start_refs"])
    if own:
        s["ep"].kv_compact(s["pages"], s["ws"], s["status"])
    else:
        _plain_compact(s)
    return {"tables": s["tables"], "refs": s["refs"], "pool": s["pool"]}


def _run_copy(s):
    if own:
        s["ep"].kv_copy_pages(s["pages"], s["src"], s["dst"], s["ws"], s["status"])
    else:
        s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return {"pool": s["pool"]}


def _run_append(s):
    if own:
        q = s["q_out"]
        s["ep"].kv_append(s["cache"], s["tables"], s["lens"], s["q_off"], s["q"], s["k"], s["v"], q, s["rope"],
                          s["status"])
    else:
        q = _plain_append(s)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_attend(s):
    if own:
        out, lse = s["out"], s["lse"]
        s["ep"].kv_attend(s["cache"], s["tables"], s["lens"], s["q_off"], s["new"], s["group_off"], s["shared"],
                          s["q"], out, lse, s["scale"], s["ws"], s["status"])
    else:
        out, lse = _plain_attend(s)
    return {"out": out, "lse": lse}


def run(state):
    op = state["case"]["op"]
    return {"pages": _run_pages, "compact": _run_compact, "copy": _run_copy, "append": _run_append,
            "attend": _run_attend}[op](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_append(s):
    c, bt = s["case"], s["case"]["page_tokens"]
    off, lens, half = s["q_off"].tolist(), s["lens"].tolist(), s["case"]["rot"] // 2
    first, second = (range(half), range(half, 2 * half)) if c["layout"] == "half" else \
        (range(0, 2 * half, 2), range(1, 2 * half, 2))
    first, second = list(first), list(second)
    out = {"q": torch.empty(s["q"].shape, dtype=torch.float64, device=DEV),
           "k_cache": s["k_cache"].to(torch.float64), "v_cache": s["v_cache"].to(torch.float64)}
    for b, (lo, hi) in enumerate(zip(off, off[1:])):
        pos = torch.arange(lens[b] - (hi - lo), lens[b], device=DEV)
        phi = torch.outer(pos.double(), s["inv"].double())[:, None]
        turned = []
        for x in (s["q"][lo:hi].double(), s["k"][lo:hi].double()):
            y = x.clone()
            y[..., first] = s["mscale"] * (x[..., first] * phi.cos() - x[..., second] * phi.sin())
            y[..., second] = s["mscale"] * (x[..., second] * phi.cos() + x[..., first] * phi.sin())
            turned.append(y)
        out["q"][lo:hi] = turned[0]
        page, slot = s["tables"][b].long()[pos // bt], pos % bt
        for name, x, scale in zip(("k_cache", "v_cache"), (turned[1], s["v"][lo:hi].double()), s["scales"]):
            out[name][page, slot] = x if scale is None else (x / scale.double()[:, None]).clamp(-448, 448)
    return out


def _exact_attend(s):
    c, bt, share = s["case"], s["case"]["page_tokens"], s["case"]["heads"] // s["case"]["kv_heads"]
    off, lens = s["q_off"].tolist(), s["lens"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, (lo, hi) in enumerate(zip(off, off[1:])):
        n, t = lens[b], torch.arange(lens[b], device=DEV)
        page, slot = s["tables"][b].long()[t // bt], t % bt
        k, v = (x.view(torch.uint8)[page, slot].view(x.dtype).double() for x in (s["k_cache"], s["v_cache"]))
        if s["scales"][0] is not None:
            k, v = k * s["scales"][0].double()[:, None], v * s["scales"][1].double()[:, None]
        hidden = t > torch.arange(n - (hi - lo), n, device=DEV)[:, None]
        for h in range(c["heads"]):
            score = s["scale"] * torch.mm(s["q"][lo:hi, h].double(), k[:, h // share].t())
            score[hidden] = -math.inf
            lse[lo:hi, h] = torch.logsumexp(score, 1)
            out[lo:hi, h] = torch.mm((score - lse[lo:hi, h, None]).exp(), v[:, h // share])
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    if case["op"] == "attend":
        return _exact_attend(prepare(case, seed))
    return None
