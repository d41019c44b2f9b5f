"""Float64 / integer references of rotary positions and of cache eviction (numpy, no torch, no GPU).

``rotary_ref`` and ``rotary_backward_ref`` turn column pairs as complex numbers; angles come from integer products of
positions with the table's 64-bit turns, so that far positions are exact.  ``paged_weigh_ref`` walks sequence by sequence
and head by head over the keys gathered from the pages, ``paged_evict_ref`` sorts every (sequence, key head) by itself,
``paged_trim_ref`` pushes page by page onto a Python list.  Inputs are not changed.
"""
from __future__ import annotations

import numpy as np

from .paged_ref import gather_pages

__all__ = ["frequencies", "turn_angles", "rotary_ref", "rotary_backward_ref", "paged_weigh_ref", "paged_evict_ref",
           "paged_trim_ref"]


def frequencies(dim, base=10000.0, scaling=None, factor=1.0, original=4096, low=1.0, high=32.0):
    """(frequencies in radians per position, magnitude)."""
    i = np.arange(0, dim, 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (dim / max(dim - 2, 1))
    f = base ** (-i / dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        turns = original * f / (2 * np.pi)
        keep = np.clip((turns - low) / (high - low), 0, 1)
        return keep * f + (1 - keep) * f / factor, 0.1 * np.log(factor) + 1.0
    return f, 1.0


def turn_angles(positions, turns):
    """Angles in radians [..., rot / 2] of integer positions, the whole turns taken off exactly."""
    out = np.empty((*np.shape(positions), len(turns)))
    flat = out.reshape(-1, len(turns))
    for a, p in enumerate(np.asarray(positions, dtype=object).reshape(-1)):
        for b, t in enumerate(turns):
            whole = (int(p) * int(t)) % 2 ** 64
            flat[a, b] = 2 * np.pi * ((whole - 2 ** 64 if whole >= 2 ** 63 else whole) / 2.0 ** 64)
    return out


def _turned(u, angles, interleaved, sign):
    """u [..., d] with its first columns turned by sign * angles [..., rot / 2]."""
    half = angles.shape[-1]
    y = u.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    z = (u[..., a] + 1j * u[..., b]) * np.exp(1j * sign * angles)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _scaled(y, half, magnitude):
    y = y.copy()
    y[..., : 2 * half] *= magnitude
    return y


def rotary_ref(x, angles, gain=None, eps=None, interleaved=False, magnitude=1.0):
    """x [..., d] float64, angles broadcastable to [..., rot / 2]."""
    u = np.asarray(x, np.float64)
    if eps is not None:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * (1.0 if gain is None else gain)
    angles = np.broadcast_to(angles, (*u.shape[:-1], angles.shape[-1]))
    return _scaled(_turned(u, angles, interleaved, 1), angles.shape[-1], magnitude)


def rotary_backward_ref(dy, x, angles, gain=None, eps=None, interleaved=False, magnitude=1.0):
    """(dx, dgain or None): the transpose of the rotation, then of the normalisation's Jacobian."""
    dy = np.asarray(dy, np.float64)
    angles = np.broadcast_to(angles, (*dy.shape[:-1], angles.shape[-1]))
    g = _turned(_scaled(dy, angles.shape[-1], magnitude), angles, interleaved, -1)
    if eps is None:
        return g, None
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    s = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dgain = (g * x / s).reshape(-1, d).sum(0)
    h = g * (1.0 if gain is None else gain)
    return h / s - x * (h * x).sum(-1, keepdims=True) / (d * s ** 3), dgain


def paged_weigh_ref(q, lse, k_cache, scores, table, cu_q, kv_lens, tau, decay=1.0, last=0, causal=True, positions=None,
                    dropped=None):
    """Returns (scores, positions or None, mag): mag holds each score's sum of weights alone."""
    q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
    scores = np.array(scores, np.float64)
    positions = None if positions is None else np.array(positions)
    mag = np.zeros_like(scores)
    page, Hkv, G = k_cache.shape[2], k_cache.shape[1], q.shape[1] // k_cache.shape[1]
    for s, L in enumerate(int(x) for x in kv_lens):
        lo, hi = int(cu_q[s]), int(cu_q[s + 1])
        n = hi - lo
        if n == 0:
            continue
        K = gather_pages(k_cache, table[s], L)
        first = max(n - last, 0) if last else 0
        tok = np.arange(first, n)
        sees = np.clip(L - n + tok + 1, 0, L) if causal else np.full(len(tok), L)
        hide = np.arange(L)[None, :] >= sees[:, None]
        for h in range(Hkv):
            w = np.zeros(L)
            for g in range(h * G, (h + 1) * G):
                e = lse[lo + first: hi, g][:, None]
                logit = tau * (q[lo + first: hi, g] @ K[h].T)
                skip = hide | np.isneginf(e)
                w += np.where(skip, 0.0, np.exp(np.where(skip, 0.0, logit - np.where(np.isneginf(e), 0.0, e)))).sum(0)
            for j in range(L):
                at = int(table[s][j // page]), h, j % page
                fresh = causal and j >= L - n
                mag[at] = w[j]
                scores[at] = w[j] + (0.0 if fresh or decay == 0 else decay * scores[at])
                if fresh and positions is not None:
                    positions[at] = j + (0 if dropped is None else int(dropped[s]))
    return scores, positions, mag


def paged_evict_ref(scores, table, kv_lens, keep, page, Hkv, positions=None, dropped=None, sinks=0, recent=0):
    """For every (sequence, key head): the slot whose row each of its first min(L, keep) slots holds afterwards.  A slot whose
    page is not in the cache holds no row and takes none: that many fewer positions are kept."""
    out, pages = {}, len(scores)
    for s, L in enumerate(int(x) for x in kv_lens):
        b = min(L, max(int(keep[s]), 0))
        for h in range(Hkv):
            at = [(int(table[s][j // page]), h, j % page) for j in range(L)]
            there = [j for j in range(L) if 0 <= at[j][0] < pages]
            value = {j: float(scores[at[j]]) for j in there}
            value = {j: -np.inf if np.isnan(v) else v for j, v in value.items()}
            must = dict.fromkeys(there, False)
            if positions is not None:
                newest = L + (0 if dropped is None else int(dropped[s]))
                must = {j: int(positions[at[j]]) < sinks or int(positions[at[j]]) >= newest - recent for j in there}
            order = sorted(there, key=lambda j: (not must[j], 0.0 if must[j] else -value[j], j))
            places = sum(j < b for j in there)
            stay = sorted(order[:places])
            source, kept = list(range(b)), set(stay)
            holes = [j for j in there if j < b and j not in kept]
            for hole, j in zip(holes, [j for j in stay if j >= b]):
                source[hole] = j
            out[s, h] = source
    return out


def paged_trim_ref(kv_lens, keep, table, free, count, page, dropped=None):
    """dict(kv_lens, dropped, free_left, free_pages, full): full where a page found no room on the free stack."""
    free, capacity = [int(x) for x in free], len(free)
    count, full = min(max(int(count), 0), capacity), False
    out = dict(kv_lens=[], dropped=[])
    for s, L in enumerate(max(int(x), 0) for x in kv_lens):
        b = min(L, max(int(keep[s]), 0))
        for c in range(-(-b // page), -(-L // page)):
            if int(table[s][c]) < 0:
                continue
            if count < capacity:
                free[count] = int(table[s][c])
                count += 1
            else:
                full = True
        out["kv_lens"].append(b)
        out["dropped"].append(L - b + (0 if dropped is None else int(dropped[s])))
    out.update(free_left=count, free_pages=free, full=full)
    return out
