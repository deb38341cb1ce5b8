"""What a decoder's step does with its quantized cache, in float64 (and float32
where a definition rounds): page tables and slot maps, heads normed and rotated,
attention.  Plain numpy, one step after another."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["cache_extend", "rope_heads", "cache_attention"]


def cache_extend(lens, added, pages, free_pages, free_count, page_tokens, T):
    """One sequence after another, one page after another.  Returns a dict of
    lens_out, free_count_out, offsets, positions, slots, pages, free_pages."""
    lens = [-1 - int(n) if n < 0 else int(n) for n in lens]
    pages, free = np.array(pages), np.array(free_pages)
    max_pages, top = pages.shape[1], min(max(int(free_count), 0), len(free))

    def held(n):
        return min(-(-n // page_tokens), max_pages)

    for i, a in enumerate(added):
        if a < 0:
            for k in range(held(lens[i])):
                if top < len(free):
                    free[top] = pages[i, k]
                    top += 1
    out, offsets, positions, slots = [], [0], [], []
    # (the running sum of what is asked for goes on past a sequence that is refused)
    asked, stack = 0, top
    for i, (n, a) in enumerate(zip(lens, added)):
        a = int(a)
        if a < 0:
            out.append(0)
            offsets.append(offsets[-1])
            continue
        end = offsets[-1] + a
        need = -(-(n + a) // page_tokens) - held(n)
        ok = -(-(n + a) // page_tokens) <= max_pages and end <= T and n + a <= 2 ** 31 - 1
        if ok:
            asked += need
            ok = need == 0 or asked <= stack
        if ok or a == 0:
            for k in range(need if ok else 0):
                top -= 1
                pages[i, held(n) + k] = free[top]
            out.append(n + a)
        else:
            out.append(-1 - n)
        for q in range(n, n + a if end <= T else n + max(0, T - offsets[-1])):
            positions.append(q)
            slots.append(int(pages[i, q // page_tokens]) * page_tokens + q % page_tokens
                         if ok else -1)
        offsets.append(end)
    positions += [0] * (T - len(positions))
    slots += [-1] * (T - len(slots))
    return dict(lens_out=np.array(out, np.int64), free_count_out=top,
                offsets=np.minimum(np.array(offsets, np.int64), T),
                positions=np.array(positions, np.int64), slots=np.array(slots, np.int64),
                pages=pages, free_pages=free)


def rope_heads(x32, weight, eps, inv_freq, positions, interleaved=False):
    """Float32 heads [T, n, head_dim], normed (weight None: not) and rotated, float32:
    every operation rounded, r and the angles in float64 first."""
    f = np.float32
    y = np.asarray(x32, f)
    if weight is not None:
        x64 = y.astype(np.float64)
        r = (1.0 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)).astype(f)
        y = (y * r) * np.asarray(weight, f)
    out = y.copy()
    half = 0 if inv_freq is None else len(inv_freq)
    if half:
        angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, f).astype(np.float64)
        c, s = np.cos(angle).astype(f)[:, None], np.sin(angle).astype(f)[:, None]
        first = np.arange(half) * 2 if interleaved else np.arange(half)
        second = first + 1 if interleaved else first + half
        a, b = y[..., first], y[..., second]
        out[..., first] = a * c - b * s
        out[..., second] = b * c + a * s
    return out


def cache_attention(Q, K, V, pos, scale, window=0):
    """Causal attention of one sequence, float64: Q [n, heads, hd], K and V [len,
    kv_heads, hd], pos [n] the rows' positions.  A row that sees no key is 0."""
    Q, K, V = (np.asarray(t, np.float64) for t in (Q, K, V))
    n, H, hd = Q.shape
    G = H // K.shape[1]
    out = np.zeros_like(Q)
    keys = np.arange(K.shape[0])
    for r in range(n):
        seen = keys <= pos[r]
        if window:
            seen &= keys > pos[r] - window
        if not seen.any():
            continue
        for h in range(H):
            t = scale * (K[seen, h // G] @ Q[r, h])
            p = np.exp(t - t.max())
            out[r, h] = p @ V[seen, h // G] / math.fsum(p)
    return out
