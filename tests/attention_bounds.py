"""Float64 attention of one sequence and the bound of its error, each key by what its own
roundings may do (tests/attention_util.py takes the worst of them for all)."""
import math

import torch

F16, F32, BF16 = 2.0 ** -11, 2.0 ** -24, 2.0 ** -8


def _sizes(cache, rows, which):
    """Of rows of K (0) or V (1): |values|, |s (c - mid)|, |middle|, the largest of a
    group, [n, KV, hd], and per channel what D^{-1/2} multiplies."""
    sc, m = cache.parts(rows, which)
    mid = cache.middle(rows, which)
    group = min(cache.group, cache.hd)
    part, b = (sc - mid).abs(), (m + mid).abs()
    dhi = cache.dhi[which]
    at = (cache.first, cache.v_first)[which]
    d = torch.ones(cache.KV, cache.hd, dtype=torch.float64, device=sc.device) if dhi is None else \
        dhi.double()[at:at + cache.KV * cache.hd].view(cache.KV, cache.hd)
    # the unit goes with the codes' range, before D^{-1/2}: s mid or |b|
    if cache.how["qformat"] == "fp8":
        s = (cache.two if which and cache.two else cache.one)[1][rows].double().repeat_interleave(cache.group, 1)
        most = 448 * s[:, at:at + cache.KV * cache.hd].unflatten(1, (cache.KV, cache.hd))
    else:
        most = torch.maximum(mid, b) / d
    top = most.unflatten(2, (-1, group)).amax(3, keepdim=True).expand(-1, -1, -1, group).flatten(2) * d
    return sc + m, part, b, sc.abs(), top


def by_key(cache, Q, rows, shift, scale, window=0, tile=False):
    """Row r of Q [n, H, hd] at position shift + r over cache rows `rows`.

    Key j's weight is off by a factor e^x with |x| at most
      2^-11 + 2^-25 / p_j         p_j in fp16, p of the largest score in [1, 2^8)
      + scale sum_i |q_i| dk_ij   dk: tile: three roundings of 2^-11, of s (c - mid), of
                                  the middle and of their sum, and 2^-16 of the group's
                                  largest value where fp16 is subnormal; else none
      + (2^-11 if D, + 2 (hd + 8) 2^-24) scale sum_i |q_i| (|s c| + |m|)   q' in fp16;
                                  float32 sums and products,
    and its v by dv: tile: as dk; else 2^-11 of s c twice (p s in fp16, s made up for in
    the middle: 2^-11 of s (c - mid)) and 2^-16 of the group's largest.  The result is
    rounded to bf16."""
    n, H, hd = Q.shape
    G = H // cache.KV
    (k, kp, kb, ks, kt), (v, vp, vb, vs, vt) = (_sizes(cache, rows, w) for w in (0, 1))
    at = torch.arange(rows.numel(), device=rows.device)
    pos = shift + torch.arange(n, device=rows.device)[:, None]
    seen = at <= pos
    if window:
        seen &= at > pos - window
    out, tol = (torch.zeros(n, H, hd, dtype=torch.float64, device=rows.device) for _ in range(2))
    for h in range(H):
        g = h // G
        q, qa = Q[:, h].double(), Q[:, h].double().abs()
        t = torch.where(seen, scale * q @ k[:, g].T, -math.inf)
        top = t.amax(1, keepdim=True)
        w = torch.softmax(t, 1)
        dk = F16 * (kp + kb + k.abs())[:, g] + 2.0 ** -16 * kt[:, g] if tile else torch.zeros_like(k[:, g])
        few = (F16 if cache.dhi[0] is not None else 0.0) + 2 * (hd + 8) * F32
        x = abs(scale) * (qa @ dk.T + few * qa @ (ks + (k - kp - kb).abs() + kb + kp)[:, g].T)
        x = x + F16 + 2.0 ** -25 * torch.exp((top - t).clamp(max=40)) + 2.0 ** -22 * t.abs().clamp(max=1e30)
        x = torch.where(seen, x, 0.0)
        f = torch.where(seen, w * torch.expm1(x.clamp(max=50)), 0.0)
        left = (w * torch.exp(-x)).sum(1, keepdim=True)
        o = w @ v[:, g]
        dv = F16 * (vp + vb + v.abs())[:, g] if tile else F16 * (2 * vs + vp)[:, g]
        dv = dv + 2.0 ** -16 * vt[:, g]
        # sum_j f_j |v_j - o|, a row at a time (it is [n, keys, hd])
        e = torch.stack([f[i] @ (v[:, g] - o[i]).abs() for i in range(n)]) / left + (w + f) @ dv / left
        out[:, h], tol[:, h] = o, e + BF16 * (o.abs() + e)
    none = ~seen.any(1)
    out[none], tol[none] = 0, 0
    return out, tol


def sized_cache(cache, g, k_spread, v_spread, rows=None):
    """The cache's rows written again, the K and V of a token times powers of two of
    these spreads; returns them."""
    import online_activation_aware_ttq_amd as ttq
    n = cache.one[0].shape[0]
    width = cache.KV * cache.hd
    for which, c in enumerate((cache.one, cache.two) if cache.two else (cache.one,)):
        x = torch.randn(n, cache.d, generator=g, device="cuda")
        x = x + 0.5 * torch.randn(cache.d, generator=g, device="cuda")
        for at, spread, there in ((cache.first, k_spread, which == 0),
                                  (cache.v_first, v_spread, which == 1 or not cache.two)):
            if there:
                x[:, at:at + width] *= torch.exp2(spread * torch.randn(n, 1, generator=g, device="cuda"))
        ttq.ttq_cache_write(x, torch.arange(n, device="cuda"), *c, dhalf=cache.dh[which], **cache.how)
