"""Float64 / integer references of the paged-cache operators (numpy, no torch, no GPU).

``paged_plan_ref`` walks the sequences one by one with a Python list as the free stack.
``paged_parallax_ref`` attends token by token group to the keys gathered from the pages: softmax output
minus the softmax-weighted value/key covariance times the probe, the covariance taken with both factors
centred on their means.  It also returns, per output entry, the magnitudes that rounding-error bounds of
any one-pass evaluation need.
"""
from __future__ import annotations

import numpy as np

__all__ = ["paged_plan_ref", "gather_pages", "paged_parallax_ref"]


def paged_plan_ref(ctx, new, table, free, count, page, T):
    """Returns dict(kv_lens, cu_q, slots, positions, granted, free_left, table); inputs are not changed."""
    table = np.array(table, dtype=np.int64)
    count = min(max(int(count), 0), len(free))
    stack = [int(x) for x in free[:count]]
    width = table.shape[1]
    out = dict(kv_lens=[], cu_q=[0], granted=[], slots=np.full(T, -1, np.int64), positions=np.zeros(T, np.int64))
    row, asked = 0, 0
    for s, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        first, row = row, row + n
        held, total = -(-c // page), -(-(c + n) // page)
        fits = c + n <= width * page and row <= T
        asked += total - held if fits else 0
        ok = fits and (total == held or asked <= count)
        if ok:
            for lp in range(held, total):
                table[s, lp] = stack.pop()
        for i in range(n):
            if first + i < T:
                out["positions"][first + i] = c + i
                if ok and table[s, (c + i) // page] >= 0:
                    out["slots"][first + i] = table[s, (c + i) // page] * page + (c + i) % page
        out["granted"].append(int(ok))
        out["kv_lens"].append(c + n if ok else c)
        out["cu_q"].append(min(row, T))
    out["free_left"] = len(stack)
    out["table"] = table
    return out


def gather_pages(cache, table_row, n):
    """[num_pages, Hkv, page, d] cache, one sequence's table row -> its first n rows [Hkv, n, d]."""
    page = cache.shape[2]
    ids = [int(x) for x in table_row[: -(-n // page)]]
    if not ids:
        return np.zeros((cache.shape[1], 0, cache.shape[3]))
    return np.concatenate([np.asarray(cache[i], np.float64) for i in ids], axis=1)[:, :n]


def paged_parallax_ref(q, probe, k_cache, v_cache, table, cu_q, kv_lens, tau, causal=True, seqs=None):
    """Returns (out, mag, keys): out [T, Hq, d]; mag [T, Hq, d] = (1 + M) sum_j p_j |v_j| +
    sum_j p_j |t_j - c| |v_j| with M = max_j |t_j - c| over the keys that carry weight; keys [T] their
    number.  Rows of no sequence (or of one not in seqs) are NaN in out."""
    q, probe = np.asarray(q, np.float64), np.asarray(probe, np.float64)
    T, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    out, mag, keys = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d)), np.zeros(T, np.int64)
    for s in range(len(kv_lens)) if seqs is None else seqs:
        lo, hi, L = int(cu_q[s]), int(cu_q[s + 1]), int(kv_lens[s])
        if hi == lo:
            continue
        K, V = gather_pages(k_cache, table[s], L), gather_pages(v_cache, table[s], L)
        n = hi - lo
        sees = np.full(n, L) if not causal else np.clip(L - n + np.arange(n) + 1, 0, L)
        keys[lo:hi] = sees
        hide = np.arange(L)[None, :] >= sees[:, None]
        for h in range(Hq):
            k, v = K[h // G], V[h // G]
            logit = np.where(hide, -np.inf, tau * (q[lo:hi, h] @ k.T))
            some = sees > 0
            w = np.zeros((n, L))
            if some.any():
                w[some] = np.exp(logit[some] - logit[some].max(axis=1, keepdims=True))
                w[some] /= w[some].sum(axis=1, keepdims=True)
            kbar, vbar = w @ k, w @ v
            lean = np.where(hide, 0.0, probe[lo:hi, h] @ k.T - (kbar * probe[lo:hi, h]).sum(1, keepdims=True))
            # sum_j w_j (v_j - vbar) ((k_j - kbar).probe)
            slope = (w * lean) @ v - (w * lean).sum(1, keepdims=True) * vbar
            out[lo:hi, h] = vbar - slope
            M = np.abs(lean).max(axis=1, keepdims=True) if L else np.zeros((n, 1))
            mag[lo:hi, h] = (1.0 + M) * (w @ np.abs(v)) + (w * np.abs(lean)) @ np.abs(v)
    return out, mag, keys
