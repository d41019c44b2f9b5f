"""Cases of rotary positions and of cache eviction by accumulated attention weight.

``rotary`` normalises and rotates the heads' rows of queries, keys and probes (``rotary_backward`` is its gradient):

    y = m Rot(pos f) (gain x / sqrt(mean(x^2) + eps)),     f the table's frequencies, m its magnitude.

Keys are cached rotated, so a cached key keeps its position when eviction moves it.  After a step's attention
``paged_weigh`` adds to every cached position's score the attention that the step's rows gave it,

    score_j <- decay score_j + sum_rows exp(tau q.k_j - lse_row)          (0 before, for the step's own tokens);

now and then ``paged_evict`` keeps the ``keep`` positions of largest score of every sequence and key head (the first
``sinks`` and the last ``recent`` positions before all others), kept rows behind slot ``keep`` filling the holes before
it, and ``paged_trim`` cuts the lengths and gives the pages behind them back to the free stack.
Caches are [pages, key heads, page, d], scores and positions [pages, key heads, page].
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def _rotary(name, op, B, n, heads, d, rot, dtype, layout, norm=True, interleaved=False, scaling="none", factor=1.0,
            far=0, seqs=0, dy="same"):
    """heads: "16,2" are tensors of 16 and 2 heads.  layout "rows": slices of one projection [n, ...] (B = 1); "heads":
    tensors [B, heads, n, d].  far: positions begin there; seqs: sequences whose evicted tokens shift them."""
    return {"name": name, "op": op, "B": B, "n": n, "heads": heads, "d": d, "rot": rot, "dtype": dtype, "layout": layout,
            "norm": norm, "interleaved": interleaved, "scaling": scaling, "factor": factor, "far": far, "seqs": seqs, "dy": dy}


def _weigh(name, S, new, ctx, Hq, Hkv, d, page, dtype="bf16", last=0, decay=1.0, causal=True, lens=1):
    return {"name": name, "op": "weigh", "S": S, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype, "last": last, "decay": decay, "causal": causal,
            "lens": lens}


def _evict(name, S, held, keep, Hkv, d, page, dtype="bf16", sinks=4, recent=64, again=False, lens=1):
    """held: lengths before.  again: the first `keep` slots went through an eviction before."""
    return {"name": name, "op": "evict", "S": S, "lo": held[0], "hi": held[1], "keep": keep, "Hkv": Hkv, "d": d,
            "page": page, "dtype": dtype, "sinks": sinks, "recent": recent, "again": again, "lens": lens}


def _trim(name, S, held, keep, page, ended=0.0, lens=1):
    """ended: share of the sequences that end and keep nothing."""
    return {"name": name, "op": "trim", "S": S, "lo": held[0], "hi": held[1], "keep": keep, "page": page, "ended": ended,
            "lens": lens}


def listed():
    return [
        # queries, keys and probes of a decode step of 64 requests whose caches were evicted from before
        _rotary("rotary_decode", "rotary", 1, 64, "32,4,32", 128, 128, "bf16", "rows", far=4000, seqs=64),
        # queries and keys of the language-model training shape
        _rotary("rotary_train", "rotary", 8, 4096, "16,16", 128, 128, "bf16", "heads"),
        # their gradients, from the fp32 dq and dk of the attention's backward pass
        _rotary("rotary_grad_train", "rotary_backward", 8, 4096, "16,16", 128, 128, "bf16", "heads", dy="fp32"),
        # fp32 regression streams: part of the head rotated, neighbours paired, no normalisation
        _rotary("rotary_grad_stream", "rotary_backward", 64, 1024, "1,1", 32, 24, "fp32", "heads", norm=False,
                interleaved=True),
        # the decode step of 64 sequences x 16 heads at 4096 cached positions
        _weigh("weigh_decode", 64, (1, 1), (4095, 4095), 16, 16, 128, 64),
        # a chunk of a long prompt over what is cached of it, older scores fading
        _weigh("weigh_chunk", 1, (512, 512), (16384, 16384), 32, 4, 128, 16, decay=0.97),
        # whole prompts, scored by their last 32 tokens
        _weigh("weigh_window", 8, (700, 4096), (0, 0), 16, 16, 128, 64, last=32, lens=4),
        # fp32 regression streams, chunks of odd length over the stream so far
        _weigh("weigh_stream_fp32", 16, (1, 97), (200, 1024), 4, 4, 32, 16, dtype="fp32", lens=6),
        # long prompts cut to a bounded cache after their prefill
        _evict("evict_prompts", 8, (4097, 16000), 2048, 16, 128, 16, lens=7),
        # decoding requests: every 64 steps, back to 4096 positions
        _evict("evict_steady", 64, (4130, 4160), 4096, 16, 128, 64, recent=128, again=True, lens=8),
        # the pages of the 64 requests above
        _trim("trim_steady", 64, (4130, 4160), 4096, 64, lens=8),
        # many requests cut to 1000 positions, some of them ended, small pages
        _trim("trim_many", 512, (0, 8000), 1000, 16, ended=0.2, lens=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["rotary", "rotary", "rotary_backward", "rotary_backward", "weigh", "weigh", "weigh", "evict", "evict", "trim"])
    page, lens = rng.choice([8, 16, 32, 64, 128]), rng.randrange(1 << 30)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op.startswith("rotary"):
        d, layout = rng.choice([16, 32, 64, 128, 128]), rng.choice(["rows", "heads"])
        rot = rng.choice([d, d, d // 2, d // 4, 2 * rng.randrange(1, d // 2 + 1)])
        g = rng.choice([1, 2, 4, 8])
        heads = rng.choice(["%d" % g, "%d,%d" % (g * rng.choice([1, 2, 4]), g), "%d,%d,%d" % (g * 2, g, g * 2)])
        n = _log(rng, 1, 8000)
        return _rotary("", op, 1 if layout == "rows" else _log(rng, 1, 8), n, heads, d, rot, dtype, layout, rng.random() < 0.7,
                       rng.random() < 0.4, rng.choice(["none", "linear", "ntk", "parts"]), rng.choice([2.0, 4.0, 16.0]),
                       rng.choice([0, 0, 5000, 300000]), _log(rng, 1, 200) if layout == "rows" and rng.random() < 0.5 else 0,
                       rng.choice(["same", "fp32"]) if op == "rotary_backward" else "same")
    if op == "trim":
        return _trim("", _log(rng, 1, 512), (0, _log(rng, 10, 8000)), _log(rng, 1, 4000), page, rng.choice([0.0, 0.3]), lens)
    Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128, 128])
    if op == "evict":
        hi = _log(rng, 20, 16000)
        S = _log(rng, 1, max(1, min(48, 200000 // hi)))
        keep = _log(rng, 1, hi)
        return _evict("", S, (hi // 3, hi), keep, Hkv, d, page, dtype, rng.choice([0, 4, 9]), rng.choice([0, keep // 4, 40]),
                      rng.random() < 0.5, lens)
    G, kind = rng.choice([1, 1, 2, 3, 4, 6, 8]), rng.choice(["decode", "draft", "chunk", "window", "cross"])
    if kind == "decode":
        S, new, ctx = _log(rng, 1, 96), 1, _log(rng, 1, 8000)
    elif kind == "draft":
        S, new, ctx = _log(rng, 1, 48), rng.randrange(2, 9), _log(rng, 10, 8000)
    else:
        S, new, ctx = _log(rng, 1, 12), _log(rng, 9, 1200), _log(rng, 1, 6000)
    last = rng.choice([1, 16, 32, 100]) if kind == "window" else 0
    if dtype == "fp32" or d < 64:
        S, new, ctx = max(1, S // 2), min(new, 300), min(ctx, 3000)
    return _weigh("", S, (max(1, new // 8), new), (ctx // 20, ctx), Hkv * G, Hkv, d, page, dtype, last,
                  rng.choice([1.0, 1.0, 0.9, 0.0]), kind != "cross", lens)


def draw(rng):
    while True:                                          # no larger than the largest listed case
        case = {k: v for k, v in _draw(rng).items() if k != "name"}
        cost, small = work(case), case["op"] == "weigh" and (case["dtype"] == "fp32" or case["d"] < 64)
        if cost["bytes"] <= 1e9 and cost["flops"] <= (5e9 if small else 6e10):
            return case


def _lengths(case):
    """Positions cached before a step and its new tokens (in cross attention these are not among the keys)."""
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["S"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["S"])]
    return (ctx, new) if case["causal"] else ([max(c, 1) for c in ctx], new)


def _held(case):
    """Lengths before eviction, and what each sequence keeps."""
    rng = random.Random(case["lens"])
    held = [rng.randint(case["lo"], case["hi"]) for _ in range(case["S"])]
    return held, [0 if rng.random() < case.get("ended", 0.0) else case["keep"] for _ in held]


def _pages(n, page):
    return -(-n // page)


def _heads(case):
    return [int(h) for h in case["heads"].split(",")]


def work(case):
    if case["op"].startswith("rotary"):
        es, rows = (2 if case["dtype"] == "bf16" else 4), case["B"] * case["n"] * sum(_heads(case))
        elements = rows * case["d"]
        if case["op"] == "rotary":
            return {"bytes": 2 * elements * es + 4 * case["n"], "flops": elements * (7 if case["norm"] else 3)}
        dy = 4 if case["dy"] == "fp32" else es
        read = es if case["norm"] else 0                 # without normalisation the rotation alone is undone
        return {"bytes": elements * (dy + read + es) + 4 * case["n"], "flops": elements * (12 if case["norm"] else 3)}
    if case["op"] == "trim":
        held, keep = _held(case)
        freed = sum(_pages(x, case["page"]) - _pages(min(x, k), case["page"]) for x, k in zip(held, keep))
        return {"bytes": 20 * case["S"] + 8 * freed, "flops": 4 * case["S"]}
    es, d, Hkv = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hkv"]
    if case["op"] == "evict":
        held, keep = _held(case)
        read = moved = 0
        for x, k in zip(held, keep):
            if x > k:                                    # expected rows to move: kept positions lie anywhere among the free
                r = min(case["recent"], k)
                free, first = max(x - r - case["sinks"], 1), max(k - r - case["sinks"], 0)
                behind = max(min(x - r, x) - k, 0)
                moved += min(r, x - k) + first * behind / free
                read += x
        return {"bytes": 8 * case["S"] + int(Hkv * (8 * read + moved * (4 * d * es + 8))), "flops": Hkv * read}
    ctx, new = _lengths(case)
    kv = [c + n for c, n in zip(ctx, new)] if case["causal"] else ctx
    rows = [min(n, case["last"]) if case["last"] else n for n in new]
    if case["causal"]:
        pairs = sum(r * (k - r) + r * (r + 1) // 2 for r, k in zip(rows, kv))
    else:
        pairs = sum(r * k for r, k in zip(rows, kv))
    return {"bytes": sum(kv) * Hkv * (d * es + (8 if case["decay"] else 4)) + sum(rows) * case["Hq"] * (d * es + 4)
            + 4 * sum(_pages(k, case["page"]) for k in kv), "flops": 2 * d * case["Hq"] * pairs}


# ----------------------------------------------------------------------------------------- inputs
def _rows(gen, shape, dtype, norm):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if norm:
        x *= torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * norm
    return x.to(dtype)


_ROPE = {"base": 10000.0, "original": 4096, "low": 1.0, "high": 32.0}


def _frequencies(case):
    """(frequencies in float64, magnitude) of a table; "parts": wavelengths that turn fewer than `low` times over the
    original length are stretched by the factor, those with more than `high` turns kept, and a ramp lies between."""
    r, base, factor = case["rot"], _ROPE["base"], case["factor"]
    if case["scaling"] == "ntk":
        base *= factor ** (r / max(r - 2, 1))
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "parts":
        ramp = ((_ROPE["original"] * f / (2 * math.pi) - _ROPE["low"]) / (_ROPE["high"] - _ROPE["low"])).clamp(0, 1)
        return f * ramp + f / factor * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _prepare_rotary(case, gen):
    dt, d, B, n, heads = _DT[case["dtype"]], case["d"], case["B"], case["n"], _heads(case)
    st = SimpleNamespace(op=case["op"], eps=1e-6 if case["norm"] else None, interleaved=case["interleaved"], cu=None, shift=None)
    if case["layout"] == "rows":                         # slices of a fused projection, values behind them
        fused = torch.randn(n, (sum(heads) + heads[-1]) * d, generator=gen, device="cuda").to(dt)
        st.x = [t.reshape(n, h, d) for h, t in zip(heads, fused.split([h * d for h in heads] + [heads[-1] * d], 1))]
    else:
        st.x = [torch.randn(B, h, n, d, generator=gen, device="cuda").to(dt) for h in heads]
    st.positions = case["far"] + torch.arange(n, dtype=torch.int32, device="cuda")
    if case["seqs"]:
        cut = torch.sort(torch.randint(0, n + 1, (case["seqs"] - 1,), generator=gen, device="cuda")).values
        st.cu = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), n)]).int()
        st.shift = torch.randint(0, 3000, (case["seqs"],), generator=gen, device="cuda", dtype=torch.int32)
    st.gains = [1 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in heads] if case["norm"] else None
    f, st.magnitude = _frequencies(case)
    st.frequencies = f.cuda()
    if case["op"] == "rotary_backward":
        dy = torch.float32 if case["dy"] == "fp32" else dt
        st.dy = [torch.randn(x.shape, generator=gen, device="cuda").to(dy) for x in st.x]
    if own:
        import local_linear_attention_flashlla_gb300 as lla
        st.table = lla.rotary_table(case["rot"], _ROPE["base"], scaling=None if case["scaling"] == "none" else case["scaling"],
                                    factor=case["factor"], original=_ROPE["original"], low=_ROPE["low"], high=_ROPE["high"])
    return st


def _tables(gen, need, spare):
    """Page ids of every sequence in a table, ids that are left, and the number of pages."""
    pages, width = sum(need) + spare, max(max(need), 1) + 2
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    host, table, at = ids.cpu(), torch.full((len(need), width), -1, dtype=torch.int32), 0
    for s, k in enumerate(need):
        table[s, :k] = host[at: at + k]
        at += k
    return table.cuda(), ids[at:], pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"].startswith("rotary"):
        return _prepare_rotary(case, gen)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    page, S = case["page"], case["S"]
    st = SimpleNamespace(op=case["op"], page=page)
    if case["op"] in ("evict", "trim"):
        held, keep = _held(case)
        st.max_kv, st.max_keep = max(held), max(keep)
        st.kv, st.keep = i32(held), i32(keep)
        st.dropped = torch.randint(0, 5000, (S,), generator=gen, device="cuda", dtype=torch.int32)
    if case["op"] == "trim":
        st.table, spare, pages = _tables(gen, [_pages(k, page) for k in held], 40)
        st.free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        st.free[: spare.numel()] = spare
        st.free_count = i32([spare.numel()])
        return st
    Hkv, d, dt = case["Hkv"], case["d"], _DT[case["dtype"]]
    if case["op"] == "evict":
        kv = held
    else:
        ctx, new = _lengths(case)
        kv = [c + n for c, n in zip(ctx, new)] if case["causal"] else ctx
    st.table, _, pages = _tables(gen, [_pages(k, page) for k in kv], 5)
    st.k_cache = _rows(gen, (pages, Hkv, page, d), dt, 1.0)
    st.scores = torch.exp(2 * torch.randn(pages, Hkv, page, generator=gen, device="cuda"))
    st.scores_out = torch.zeros_like(st.scores)
    st.positions = torch.full((pages, Hkv, page), -1, dtype=torch.int32, device="cuda")
    if case["op"] == "evict":
        st.v_cache = _rows(gen, (pages, Hkv, page, d), dt, None)
        st.positions_out = st.positions.clone()
        st.sinks, st.recent = case["sinks"], case["recent"]
        j = torch.arange(max(held), device="cuda")
        if not case["again"]:
            st.dropped.zero_()
        for s in range(S):
            mine = (st.dropped[s] + j[: held[s]]).int().expand(Hkv, -1).clone()
            if case["again"]:                            # what earlier evictions left, in no order; the first and last stay
                old, span = min(held[s], case["keep"]), int(st.dropped[s]) + min(held[s], case["keep"])
                must = min(case["sinks"], old)
                late = min(case["recent"], old - must)
                rest = must + torch.rand(Hkv, span - must - late, generator=gen, device="cuda").argsort(1)[:, : old - must - late]
                mine[:, :must], mine[:, must: old - late] = j[:must], rest
                mine[:, old - late: old] = span - late + j[:late]
                mine[:, :old] = mine[:, torch.randperm(old, generator=gen, device="cuda")]
            at = st.table[s, j[: held[s]] // page].long()
            st.positions[at, :, j[: held[s]] % page] = mine.T
        return st
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st.cu, st.kv, st.max_new, st.max_kv = i32(cu), i32(kv), max(new), max(kv)
    st.q = _rows(gen, (cu[-1], case["Hq"], d), dt, 1.0)
    st.tau, st.causal, st.last, st.decay = 1.0 / math.sqrt(d), case["causal"], case["last"], case["decay"]
    st.dropped = torch.randint(0, 5000, (S,), generator=gen, device="cuda", dtype=torch.int32)
    st.lse = torch.empty(cu[-1], case["Hq"], device="cuda")
    for s in range(S):                                   # what the attention of the step wrote beside its output
        K = st.k_cache[st.table[s, : _pages(kv[s], page)].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, : kv[s]].float()
        q = st.q[cu[s]: cu[s + 1]].float().reshape(new[s], Hkv, -1, d).permute(1, 2, 0, 3)
        logit = torch.matmul(q, K.transpose(1, 2)[:, None]).mul_(st.tau)
        if st.causal:
            logit.masked_fill_(torch.ones(new[s], kv[s], dtype=torch.bool, device="cuda").triu(kv[s] - new[s] + 1), -math.inf)
        st.lse[cu[s]: cu[s + 1]] = torch.logsumexp(logit, -1).permute(2, 0, 1).reshape(new[s], -1)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _angles(st):
    pos = st.positions.double()
    if st.shift is not None:
        of = torch.searchsorted(st.cu.long(), torch.arange(pos.numel(), device="cuda"), right=True) - 1
        pos = pos + st.shift[of]
    a = pos[:, None] * st.frequencies
    return a.cos().float() * st.magnitude, a.sin().float() * st.magnitude


def _turn(x, c, s, interleaved):
    """The rotation of the leading columns of x by angles with cosines c and sines s."""
    r = 2 * c.shape[-1]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., r:]], -1)
    a, b = x[..., : r // 2], x[..., r // 2: r]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., r:]], -1)


def _plain_rotary(st):
    c, s = _angles(st)
    out = []
    for i, x in enumerate(st.x):
        cc, ss = (c[:, None], s[:, None]) if x.dim() == 3 else (c, s)
        y = x.float()
        if st.eps is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st.eps) * st.gains[i]
        out.append(_turn(y, cc, ss, st.interleaved).to(x.dtype))
    return out


def _plain_rotary_backward(st):
    c, s = _angles(st)
    dxs, dgains = [], []
    for i, (x, dy) in enumerate(zip(st.x, st.dy)):
        cc, ss = (c[:, None], s[:, None]) if x.dim() == 3 else (c, s)
        g = _turn(dy.float(), cc, -ss, st.interleaved)
        if st.eps is not None:
            y = x.float()
            rs = torch.rsqrt((y * y).mean(-1, keepdim=True) + st.eps)
            dgains.append((g * y * rs).flatten(0, -2).double().sum(0).float())
            g = g * st.gains[i]
            g = rs * (g - y * rs * rs * (g * y).mean(-1, keepdim=True))
        dxs.append(g.to(x.dtype))
    return dxs + dgains


def _slots(table, kv, most, page):
    """(page, row) of the first `most` slots of every sequence, and which of them it holds."""
    j = torch.arange(most, device="cuda")
    at = table[:, : _pages(most, page)].long().clamp(min=0).repeat_interleave(page, 1)[:, :most]
    return at, (j % page).expand_as(at), j < kv[:, None]


def _plain_weigh(st):
    Hkv, d = st.k_cache.shape[1], st.k_cache.shape[3]
    T, Hq = st.q.shape[:2]
    S, N, G = st.kv.numel(), min(st.max_new, st.last or st.max_new), Hq // Hkv
    cu, kv = st.cu.long(), st.kv.long()
    n_new = cu[1:] - cu[:-1]
    at, row, there = _slots(st.table, kv, st.max_kv, st.page)
    K = st.k_cache[at, :, row].permute(0, 2, 1, 3).float()                 # [S, Hkv, keys, d]
    tok = n_new[:, None] - N + torch.arange(N, device="cuda")              # the last N tokens of every sequence
    of = (cu[:-1, None] + tok).clamp(0, T - 1)
    j = torch.arange(st.max_kv, device="cuda")
    seen = there[:, None] & (tok >= 0)[:, :, None]
    if st.causal:
        seen = seen & (j <= (kv - n_new)[:, None, None] + tok[:, :, None])
    q = st.q[of].float().reshape(S, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(S, Hkv, N * G, d)
    lse = st.lse[of].reshape(S, N, Hkv, G).transpose(1, 2).reshape(S, Hkv, N * G, 1)
    p = torch.matmul(q, K.transpose(2, 3)).mul_(st.tau).sub_(lse).exp_()
    w = p.masked_fill_(~seen.repeat_interleave(G, 1)[:, None], 0.0).sum(2)  # [S, Hkv, keys]
    mine = there & (j >= (kv - n_new)[:, None]) if st.causal else torch.zeros_like(there)
    if st.decay:
        w += torch.where(mine[:, None], 0.0, st.decay * st.scores[at, :, row].transpose(1, 2))
    s, k = torch.nonzero(there, as_tuple=True)
    st.scores_out[at[s, k], :, row[s, k]] = w[s, :, k]
    s, k = torch.nonzero(mine, as_tuple=True)
    st.positions[at[s, k], :, row[s, k]] = (st.dropped[s] + k).int()[:, None].expand(-1, Hkv)
    return {"scores": st.scores_out, "positions": st.positions}


def _plain_evict(st):
    kv, keep = st.kv.long(), torch.minimum(st.kv, st.keep.clamp(min=0)).long()
    at, row, there = _slots(st.table, kv, st.max_kv, st.page)
    score = st.scores[at, :, row].transpose(1, 2)                          # [S, Hkv, slots]
    pos = st.positions[at, :, row].transpose(1, 2)
    must = (pos < st.sinks) | (pos >= (kv + st.dropped)[:, None, None] - st.recent)
    rank = torch.where(torch.isnan(score), -math.inf, score).double()
    rank = torch.where(must, math.inf, rank.clamp(max=1e300)).masked_fill(~there[:, None], -math.inf)
    # slots by falling score, equal ones by rising slot: the first `keep` of them stay
    order = torch.sort(rank, stable=True, dim=-1, descending=True).indices
    place = torch.empty_like(order).scatter_(-1, order, torch.arange(order.shape[-1], device="cuda").expand_as(order))
    kept = (place < keep[:, None, None]) & there[:, None]
    j = torch.arange(order.shape[-1], device="cuda")
    hole, move = ~kept & (j < keep[:, None, None]), kept & (j >= keep[:, None, None])
    (s, h, to), (_, _, frm) = torch.nonzero(hole, as_tuple=True), torch.nonzero(move, as_tuple=True)
    for cache in (st.k_cache, st.v_cache):
        cache[at[s, to], h, row[s, to]] = cache[at[s, frm], h, row[s, frm]]
    source = j.expand_as(order).clone()
    source[s, h, to] = frm
    s, h, k = torch.nonzero((j < keep[:, None, None]).expand_as(order), as_tuple=True)
    frm = source[s, h, k]
    for new, old in ((st.scores_out, st.scores), (st.positions_out, st.positions)):
        new[at[s, k], h, row[s, k]] = old[at[s, frm], h, row[s, frm]]
    return {"k_cache": st.k_cache, "v_cache": st.v_cache, "scores": st.scores_out, "positions": st.positions_out}


def _plain_trim(st):
    kv = st.kv.long()
    new = torch.minimum(kv, st.keep.long().clamp(min=0))
    first, held = (new + st.page - 1) // st.page, (kv + st.page - 1) // st.page
    col = torch.arange(st.table.shape[1], device="cuda")
    ids = st.table[(col >= first[:, None]) & (col < held[:, None])]
    st.free[st.free_count.long() + torch.arange(ids.numel(), device="cuda")] = ids
    return {"kv_lens": new.int(), "dropped": (st.dropped + kv - new).int(), "free_left": st.free_count + ids.numel(),
            "free_pages": st.free}


_PLAIN = {"rotary": _plain_rotary, "rotary_backward": _plain_rotary_backward, "weigh": _plain_weigh, "evict": _plain_evict,
          "trim": _plain_trim}


def run(st):
    if not own:
        return _PLAIN[st.op](st)
    import local_linear_attention_flashlla_gb300 as lla
    if st.op == "rotary":
        return list(lla.rotary(st.x, st.positions, st.table, gain=st.gains, eps=st.eps, interleaved=st.interleaved, cu_q=st.cu,
                               shift=st.shift))
    if st.op == "rotary_backward":
        dxs, dgains = lla.rotary_backward(st.dy, st.x, st.positions, st.table, gain=st.gains, eps=st.eps,
                                          interleaved=st.interleaved, cu_q=st.cu, shift=st.shift)
        return list(dxs) + list(dgains or ())
    if st.op == "weigh":
        lla.paged_weigh(st.q, st.lse, st.k_cache, st.scores, st.table, st.cu, st.kv, st.tau, st.max_new,
                        positions=st.positions, dropped=st.dropped, decay=st.decay, last=st.last, causal=st.causal,
                        out=st.scores_out)
        return {"scores": st.scores_out, "positions": st.positions}
    if st.op == "evict":
        lla.paged_evict(st.scores, st.k_cache, st.v_cache, st.table, st.kv, st.keep, positions=st.positions,
                        dropped=st.dropped, sinks=st.sinks, recent=st.recent, scores_out=st.scores_out,
                        positions_out=st.positions_out)
        return {"k_cache": st.k_cache, "v_cache": st.v_cache, "scores": st.scores_out, "positions": st.positions_out}
    r = lla.paged_trim(st.kv, st.keep, st.table, st.free, st.free_count, st.page, dropped=st.dropped)
    return {"kv_lens": r.kv_lens, "dropped": r.dropped, "free_left": r.free_left, "free_pages": st.free}


# ------------------------------------------------------------------------------------------ exact
def _matrix(st, case):
    """The rotation of every position as complex numbers, magnitude in: [n, rot / 2]."""
    pos = st.positions.tolist()
    if st.shift is not None:
        cu, shift = st.cu.tolist(), st.shift.tolist()
        for s, by in enumerate(shift):
            for t in range(cu[s], cu[s + 1]):
                pos[t] += by
    angle = torch.tensor(pos, dtype=torch.float64, device="cuda")[:, None] * st.frequencies
    return torch.polar(torch.full_like(angle, st.magnitude), angle)


def _as_complex(x, r, interleaved):
    pair = x[..., :r].unflatten(-1, (r // 2, 2)) if interleaved else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    return torch.view_as_complex(pair.contiguous())


def _as_real(z, rest, interleaved):
    pair = torch.view_as_real(z)
    return torch.cat([(pair if interleaved else pair.transpose(-1, -2)).flatten(-2), rest], -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("rotary"):
        z, r, d = _matrix(st, case), case["rot"], case["d"]
        out, gains = [], []
        for i, x in enumerate(st.x):
            x, zz = x.double(), z[:, None] if x.dim() == 3 else z
            scale = 1.0 / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + st.eps) if case["norm"] else 1.0
            gain = st.gains[i].double() if case["norm"] else 1.0
            if case["op"] == "rotary":
                u = x * scale * gain
                out.append(_as_real(_as_complex(u, r, st.interleaved) * zz, u[..., r:], st.interleaved))
                continue
            dy = st.dy[i].double()
            g = _as_real(_as_complex(dy, r, st.interleaved) * zz.conj(), dy[..., r:], st.interleaved)
            if case["norm"]:
                unit = x * scale                         # dx is g gain / rms without its part along the unit row
                gains.append((g * unit).reshape(-1, d).sum(0))
                g = g * gain
                g = scale * g - unit * scale * (g * unit).sum(-1, keepdim=True) / d
            out.append(g)
        return out + gains
    page = case["page"]
    if case["op"] == "weigh":
        ctx, new = _lengths(case)
        Hkv, G, d, at = case["Hkv"], case["Hq"] // case["Hkv"], case["d"], 0
        scores, positions = st.scores_out.double(), st.positions.clone()
        for s, n in enumerate(new):
            L = ctx[s] + n if case["causal"] else ctx[s]
            used = st.table[s, : _pages(L, page)].long()
            rows = min(n, case["last"]) if case["last"] else n
            slot = torch.arange(L, device="cuda")
            for h in range(Hkv):
                K, w = st.k_cache[used, h].reshape(-1, d)[:L].double(), torch.zeros(L, dtype=torch.float64, device="cuda")
                for g in range(h * G, (h + 1) * G):
                    logit = K @ st.q[at + n - rows: at + n, g].double().T * st.tau          # [L, rows]
                    weight = torch.exp(logit - st.lse[at + n - rows: at + n, g].double())
                    if case["causal"]:
                        weight[slot[:, None] > L - rows + torch.arange(rows, device="cuda")] = 0.0
                    w += weight.sum(1)
                old = st.scores[used, h].reshape(-1)[:L].double() * case["decay"]
                first = ctx[s] if case["causal"] else L
                w[:first] += old[:first]
                scores[used[slot // page], h, slot % page] = w
                if case["causal"]:
                    fresh = slot[ctx[s]:]
                    positions[used[fresh // page], h, fresh % page] = (int(st.dropped[s]) + fresh).int()
            at += n
        return {"scores": scores, "positions": positions}
    held, keep = _held(case)
    table = st.table.cpu().tolist()
    if case["op"] == "trim":
        free, count = st.free.cpu().tolist(), int(st.free_count)
        for s, (x, k) in enumerate(zip(held, keep)):
            for c in range(_pages(min(x, k), page), _pages(x, page)):
                free[count] = table[s][c]
                count += 1
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        dropped = [a + x - min(x, k) for a, x, k in zip(st.dropped.tolist(), held, keep)]
        return {"kv_lens": i32([min(x, k) for x, k in zip(held, keep)]), "dropped": i32(dropped), "free_left": i32([count]),
                "free_pages": i32(free)}
    if case["S"] * case["Hkv"] * max(held) > 8_000_000:
        return None
    score, where, dropped = st.scores.cpu(), st.positions.cpu(), st.dropped.tolist()
    kc, vc, so, po = (t.cpu() for t in (st.k_cache, st.v_cache, st.scores_out, st.positions_out))
    for s, (x, k) in enumerate(zip(held, keep)):
        slot = torch.arange(x)
        used, off = torch.tensor(table[s])[slot // page].long(), slot % page
        k = min(x, k)
        for h in range(case["Hkv"]):
            value, pos = score[used, h, off].tolist(), where[used, h, off].tolist()
            first = [p < case["sinks"] or p >= x + dropped[s] - case["recent"] for p in pos]
            best = sorted(range(x), key=lambda i: (not first[i], 0.0 if first[i] else -value[i], i))[:k]
            stay = set(best)
            to = [i for i in range(k) if i not in stay]
            frm = sorted(i for i in best if i >= k)
            src = torch.arange(k)
            src[to] = torch.tensor(frm, dtype=torch.int64)
            for new, old in ((so, score), (po, where)):
                new[used[:k], h, off[:k]] = old[used[src], h, off[src]]
            for cache in (kc, vc):
                cache[used[to], h, off[to]] = cache[used[frm], h, off[frm]]
    return {"k_cache": kc.double().cuda(), "v_cache": vc.double().cuda(), "scores": so.double().cuda(), "positions": po.cuda()}
