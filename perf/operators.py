"""Cases of the paged-cache operators: page planning, cache append and Parallax attention over pages.

The three run in this order in a serving step: ``paged_plan`` gives every request the pages its new
tokens need and maps token rows to cache slots, ``paged_append`` writes the tokens' keys and values
there, and ``paged_parallax`` attends from the new tokens to all cached positions of their request:

    p_j = exp(tau q.k_j - m),  w = sum_j p_j,  t_j = probe.k_j,  c = sum_j p_j t_j / w,
    out = sum_j p_j (1 - (t_j - c)) v_j / w        (softmax output minus Sigma_KV probe).

Caches are [pages, key heads, page, d]; token rows are packed request after request.
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def _plan(name, S, new, ctx, page, pad=0, lens=1, short=False):
    return {"name": name, "op": "plan", "S": S, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "page": page, "pad": pad, "lens": lens, "short": short}


def _append(name, S, new, ctx, Hkv, d, page, dtype="bf16", pad=0, lens=1):
    return {"name": name, "op": "append", "S": S, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hkv": Hkv, "d": d, "page": page, "dtype": dtype, "pad": pad, "lens": lens}


def _attend(name, S, new, ctx, Hq, Hkv, d, page, dtype="bf16", causal=True, pad=0, lens=1):
    return {"name": name, "op": "parallax", "S": S, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype, "causal": causal, "pad": pad,
            "lens": lens}


def listed():
    return [
        # one decode step of 64 requests: a page for those that cross a page border
        _plan("plan_decode", 64, (1, 1), (1, 4095), 64),
        # a step that mixes decoding requests with prompts, in a batch padded to its capacity
        _plan("plan_mixed", 512, (1, 250), (0, 8000), 16, pad=1000),
        # the new token of 64 decoding requests
        _append("append_decode", 64, (1, 1), (1, 4095), 16, 128, 64),
        # the prompts of a prefill step, odd lengths, with padding rows
        _append("append_prompts", 24, (40, 1500), (0, 2000), 8, 128, 16, pad=77),
        # the decode step of 64 sequences x 16 heads at 4096 cached positions
        _attend("decode_even", 64, (1, 1), (4095, 4095), 16, 16, 128, 64),
        # decoding requests of very different lengths, eight query heads to a key head, small pages
        _attend("decode_ragged", 96, (1, 1), (100, 16000), 32, 4, 128, 16, lens=2),
        # one user at a long context: latency
        _attend("decode_one_long", 1, (1, 1), (32767, 32767), 16, 2, 128, 64),
        # five drafted tokens of each request checked at once
        _attend("verify_drafts", 32, (5, 5), (300, 6000), 16, 4, 64, 32, lens=3),
        # a chunk of a long prompt over what is cached of it
        _attend("chunk_long", 1, (512, 512), (16384, 16384), 32, 4, 128, 16),
        # whole prompts, ragged, nothing cached before
        _attend("prefill", 8, (700, 4096), (0, 0), 16, 16, 128, 64, pad=100, lens=4),
        # decoder tokens to an encoder's cached states of another length
        _attend("cross_states", 16, (30, 200), (900, 1500), 8, 8, 64, 32, causal=False, lens=5),
        # fp32 regression streams, d = 32, chunks of odd length over the stream so far
        _attend("stream_fp32", 16, (1, 97), (200, 1024), 4, 4, 32, 16, dtype="fp32", pad=3, lens=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "parallax", "parallax", "parallax"])
    page = rng.choice([8, 16, 32, 64, 128])
    lens = rng.randrange(1 << 30)
    pad = rng.choice([0, 0, rng.randrange(1, 200)])
    if op == "plan":
        new = _log(rng, 1, 250)
        return {k: v for k, v in _plan("", _log(rng, 1, 512), (rng.choice([0, 1, new]), new), (0, _log(rng, 10, 8000)),
                                       page, pad, lens, rng.random() < 0.3).items() if k != "name"}
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "append":
        new = _log(rng, 1, 1500)
        return {k: v for k, v in _append("", _log(rng, 1, 24 if new > 8 else 128), (max(1, new // 30), new),
                                         (0, _log(rng, 10, 4000)), rng.choice([1, 2, 3, 4, 8]),
                                         rng.choice([16, 32, 64, 128]), page, dtype, pad, lens).items() if k != "name"}
    d = rng.choice([64, 128, 128]) if dtype == "bf16" and rng.random() < 0.85 else rng.choice([16, 32, 64, 128])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 3, 4, 6, 8])
    kind = rng.choice(["decode", "draft", "chunk", "cross"])
    if kind == "decode":
        S, new, ctx = _log(rng, 1, 96), 1, _log(rng, 1, 8000)
    elif kind == "draft":
        S, new, ctx = _log(rng, 1, 48), rng.randrange(2, 9), _log(rng, 10, 8000)
    else:
        S, new, ctx = _log(rng, 1, 12), _log(rng, 9, 1200), _log(rng, 1, 6000)
    if dtype == "fp32" or d < 64:
        S, new, ctx = max(1, S // 2), min(new, 300), min(ctx, 3000)
    while True:                                          # no larger than the largest listed case
        case = {k: v for k, v in _attend("", S, (max(1, new // 8), new), (ctx // 20, ctx), Hkv * G, Hkv, d, page, dtype,
                                         kind != "cross", pad, lens).items() if k != "name"}
        cost = work(case)
        if cost["bytes"] <= 2e9 and cost["flops"] <= (2.5e11 if dtype == "bf16" and d >= 64 else 1e10):
            return case
        S, new, ctx = max(1, S * 2 // 3), max(1, new * 4 // 5), max(1, ctx * 4 // 5)


def _lengths(case):
    """Positions cached before the step and new tokens of every request (new tokens are not part of the
    keys in cross attention)."""
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["S"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["S"])]
    if case["op"] == "parallax" and not case["causal"]:
        return [max(c, 1) for c in ctx], new
    return ctx, new


def _pages(n, page):
    return -(-n // page)


def _key_lengths(case):
    ctx, new = _lengths(case)
    if case["op"] == "parallax" and not case["causal"]:
        return ctx
    return [c + n for c, n in zip(ctx, new)]


def work(case):
    ctx, new = _lengths(case)
    kv, page, S = _key_lengths(case), case["page"], case["S"]
    rows = sum(new)
    if case["op"] == "plan":
        fresh = sum(_pages(k, page) - _pages(c, page) for k, c in zip(kv, ctx))
        touched = sum(_pages(k, page) - c // page for k, c in zip(kv, ctx) if k > c)
        return {"bytes": 20 * S + 12 * (rows + case["pad"]) + 8 * fresh + 4 * (touched - fresh), "flops": 4 * rows}
    es, d, Hkv = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hkv"]
    if case["op"] == "append":
        return {"bytes": 4 * rows * Hkv * d * es + 8 * (rows + case["pad"]), "flops": 0}
    if case["causal"]:
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    else:
        pairs = sum(n * k for n, k in zip(new, kv))
    return {"bytes": 2 * sum(kv) * Hkv * d * es + 3 * rows * case["Hq"] * d * es + 4 * sum(_pages(k, page) for k in kv),
            "flops": 8 * d * case["Hq"] * pairs}


# ----------------------------------------------------------------------------------------- inputs
def _rows(gen, shape, dtype, norm):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if norm:
        x *= torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * norm
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx, new = _lengths(case)
    kv, page, S = _key_lengths(case), case["page"], case["S"]
    need = [_pages(k, page) for k in kv]
    width = max(need) + 2
    pages = sum(need) + 5
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32)
    held = [_pages(c, page) for c in ctx] if case["op"] == "plan" else need
    ids_host, at = ids.cpu(), 0
    for s in range(S):
        table[s, : held[s]] = ids_host[at: at + held[s]]
        at += held[s]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1] + case["pad"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = SimpleNamespace(op=case["op"], page=page, T=T, table=table.cuda(), case=case, max_new=max(new), max_kv=max(kv))
    if case["op"] == "plan":
        st.ctx, st.new, st.free = i32(ctx), i32(new), ids[at:].contiguous()
        fresh = sum(need) - sum(held)
        st.free_count = i32([max(1, fresh * 7 // 10) if case["short"] else len(ids_host) - at])
        return st
    dt, d, Hkv = _DT[case["dtype"]], case["d"], case["Hkv"]
    st.k_cache = _rows(gen, (pages, Hkv, page, d), dt, 1.0)
    st.v_cache = _rows(gen, (pages, Hkv, page, d), dt, None)
    if case["op"] == "append":
        slots = torch.full((T,), -1, dtype=torch.int64)
        for s in range(S):
            pos = torch.arange(ctx[s], kv[s])
            slots[cu[s]: cu[s + 1]] = table[s, pos // page].long() * page + pos % page
        st.slots = slots.cuda()
        st.k_new = _rows(gen, (T, Hkv, d), dt, 1.0)
        st.v_new = _rows(gen, (T, Hkv, d), dt, None)
        return st
    st.cu, st.kv = i32(cu), i32(kv)
    st.q = _rows(gen, (T, case["Hq"], d), dt, 1.0)
    st.probe = _rows(gen, (T, case["Hq"], d), dt, 1.0 / math.sqrt(d))
    st.out = torch.zeros_like(st.q)
    st.tau, st.causal = 1.0 / math.sqrt(d), case["causal"]
    return st


# ------------------------------------------------------------------------------------ plain forms
def _plain_plan(st):
    ctx, new, page, table = st.ctx.long(), st.new.long(), st.page, st.table
    S, width = table.shape
    total = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros_like(total[:1]), total]).clamp(max=st.T)
    held = (ctx + page - 1) // page
    fits = (ctx + new <= width * page) & (total <= st.T)
    need = torch.where(fits, (ctx + new + page - 1) // page - held, 0)
    incl = torch.cumsum(need, 0)
    count = st.free_count.long()
    granted = fits & ((need == 0) | (incl <= count))
    left = count - torch.where(granted, incl * (need > 0), 0).max()
    kv = ctx + torch.where(granted, new, 0)
    j = torch.arange(width, device="cuda") - held[:, None]
    fresh = granted[:, None] & (j >= 0) & (j < need[:, None])
    pick = (count - 1 - ((incl - need)[:, None] + j)).clamp(0, st.free.numel() - 1)
    table.copy_(torch.where(fresh, st.free[pick], table))
    t = torch.arange(st.T, device="cuda")
    s = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=S - 1)
    there = t < cu[-1]
    pos = torch.where(there, ctx[s] + t - cu[s], 0)
    ok = there & granted[s]
    slot = table[s, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    return {"kv_lens": kv.int(), "cu_q": cu.int(), "slots": torch.where(ok, slot, -1), "positions": pos.int(),
            "granted": granted.int(), "free_left": left.int(), "table": table}


def _plain_append(st):
    # padding rows (slot -1) write the position that row 0 holds in the cache back to itself: no row is
    # read by the host, and a real row never shares a slot with another
    ok = st.slots >= 0
    at = torch.where(ok, st.slots, st.slots[0])
    for cache, new in ((st.k_cache, st.k_new), (st.v_cache, st.v_new)):
        cache[at // st.page, :, at % st.page] = torch.where(ok[:, None, None], new, new[0])
    return {"k_cache": st.k_cache, "v_cache": st.v_cache}


def _plain_parallax(st):
    P, Hkv, page, d = st.k_cache.shape
    T, Hq = st.q.shape[:2]
    S, N, G = st.kv.numel(), st.max_new, Hq // Hkv
    cu, kv = st.cu.long(), st.kv.long()
    n_new = cu[1:] - cu[:-1]
    cols = st.table[:, : -(-st.max_kv // page)].long().clamp(0, P - 1)
    K = st.k_cache[cols].transpose(1, 2).reshape(S, Hkv, -1, d).float()
    V = st.v_cache[cols].transpose(1, 2).reshape(S, Hkv, -1, d).float()
    at = (cu[:-1, None] + torch.arange(N, device="cuda")).clamp(max=T - 1)

    def heads(x):                                         # [T, Hq, d] -> [S, Hkv, N * G, d]
        return x[at].float().reshape(S, N, Hkv, G, d).transpose(1, 2).reshape(S, Hkv, N * G, d)

    j = torch.arange(K.shape[2], device="cuda")
    seen = j < kv[:, None, None]
    if st.causal:
        pos = (kv - n_new)[:, None] + torch.arange(N, device="cuda")
        seen = seen & (j <= pos[:, :, None])
    else:
        seen = seen.expand(S, N, -1)
    seen = seen.repeat_interleave(G, 1)[:, None]
    s = torch.matmul(heads(st.q), K.transpose(2, 3)).mul_(st.tau).masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isfinite(m), m, 0.0)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30))
    t = torch.matmul(heads(st.probe), K.transpose(2, 3))
    c = (p * t).sum(-1, keepdim=True)
    o = torch.matmul(p.mul_(1.0 - t.sub_(c)), V)
    o = o.reshape(S, Hkv, N, G, d).transpose(1, 2).reshape(S, N, Hq, d)
    row = torch.arange(T, device="cuda")
    of = (torch.searchsorted(cu, row, right=True) - 1).clamp(max=S - 1)
    mine = (row < cu[-1])[:, None, None]
    st.out.copy_(torch.where(mine, o[of, (row - cu[of]).clamp(max=N - 1)].to(st.out.dtype), st.out))
    return {"out": st.out}


def run(st):
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "parallax": _plain_parallax}[st.op](st)
    import local_linear_attention_flashlla_gb300 as lla
    if st.op == "plan":
        r = lla.paged_plan(st.ctx, st.new, st.table, st.free, st.free_count, st.page, st.T)
        return {"kv_lens": r.kv_lens, "cu_q": r.cu_q, "slots": r.slots, "positions": r.positions, "granted": r.granted,
                "free_left": r.free_left, "table": st.table}
    if st.op == "append":
        lla.paged_append(st.k_new, st.v_new, st.slots, st.k_cache, st.v_cache)
        return {"k_cache": st.k_cache, "v_cache": st.v_cache}
    lla.paged_parallax(st.q, st.probe, st.k_cache, st.v_cache, st.table, st.cu, st.kv, st.tau, st.max_new,
                       causal=st.causal, out=st.out)
    return {"out": st.out}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    ctx, new = _lengths(case)
    kv, page = _key_lengths(case), case["page"]
    if case["op"] == "plan":
        table, free, left = st.table.cpu().tolist(), st.free.cpu().tolist(), int(st.free_count)
        width, rows, asked, first = len(table[0]), 0, 0, left
        out = {"kv_lens": [], "cu_q": [0], "slots": [], "positions": [], "granted": []}
        for s, (c, n) in enumerate(zip(ctx, new)):
            rows += n
            held, total = -(-c // page), -(-(c + n) // page)
            fits = c + n <= width * page and rows <= st.T
            asked += total - held if fits else 0
            ok = fits and (total == held or asked <= first)
            for col in range(held, total if ok else held):
                left -= 1
                table[s][col] = free[left]
            out["cu_q"].append(min(rows, st.T))
            out["granted"].append(int(ok))
            out["kv_lens"].append(c + n if ok else c)
            for x in range(c, c + min(n, st.T - (rows - n))):
                out["positions"].append(x)
                out["slots"].append(table[s][x // page] * page + x % page if ok else -1)
        out["positions"] += [0] * (st.T - len(out["positions"]))
        out["slots"] += [-1] * (st.T - len(out["slots"]))
        out = {k: torch.tensor(v, dtype=torch.int64 if k == "slots" else torch.int32, device="cuda") for k, v in out.items()}
        out["free_left"] = torch.tensor([left], dtype=torch.int32, device="cuda")
        out["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        return out
    if case["op"] == "append":
        for cache, rows in ((st.k_cache, st.k_new), (st.v_cache, st.v_new)):
            at = 0
            for s, n in enumerate(new):
                for x in range(ctx[s], kv[s], page):
                    y = min((x // page + 1) * page, kv[s])    # to the end of the page that x lies in
                    for lo, hi in ((x, y), (y, min(x + page, kv[s]))):
                        if hi > lo:
                            i = at + lo - ctx[s]
                            cache[int(st.table[s, lo // page]), :, lo % page: lo % page + hi - lo] = \
                                rows[i: i + hi - lo].transpose(0, 1)
                at += n
        return {"k_cache": st.k_cache.double(), "v_cache": st.v_cache.double()}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    out, at = torch.zeros(st.q.shape, dtype=torch.float64, device="cuda"), 0
    for s, n in enumerate(new):
        used = st.table[s, : _pages(kv[s], page)].long()
        for h in range(Hkv):
            K = st.k_cache[used, h].reshape(-1, d)[: kv[s]].double()
            V = st.v_cache[used, h].reshape(-1, d)[: kv[s]].double()
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                logit = st.q[at: at + n, g].double() @ K.T * st.tau
                if case["causal"]:
                    hide = torch.ones(n, kv[s], dtype=torch.bool, device="cuda").triu(kv[s] - n + 1)
                    logit.masked_fill_(hide, -math.inf)
                w = torch.softmax(logit, -1)
                r = st.probe[at: at + n, g].double()
                mean_k, mean_v = w @ K, w @ V
                lean = r @ K.T - (mean_k * r).sum(-1, keepdim=True)            # (k_j - kbar).probe
                slope = (w * lean) @ V - (w * lean).sum(-1, keepdim=True) * mean_v
                out[at: at + n, g] = mean_v - slope
        at += n
    return {"out": out}
