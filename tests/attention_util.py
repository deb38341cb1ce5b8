"""A quantized cache of random rows, its attention in float64, and how far a row of
the kernel's may be from it."""
import math

import torch

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


class Cache:
    """K and V of `heads` K/V heads, written by ttq_cache_write into one cache (K, then
    V, from channel `first` on) or two; .k, .v: what its rows stand for, float64."""

    def __init__(self, g, n_slots, KV, hd, bits, group, fmt, dhalf=False, two=False, first=0,
                 spread=0.0, rows=None):
        import online_activation_aware_ttq_amd as ttq
        self.how = dict(bits=bits, group=group, qformat=fmt)
        width = KV * hd
        d = first + (width if two else 2 * width)
        d += -d % group
        rb = d * (4 if bits in (3, 4) else 8) // 8

        def empty():
            return (torch.zeros(n_slots, rb, dtype=torch.uint8, device="cuda"),
                    torch.zeros(n_slots, d // group, device="cuda"),
                    torch.zeros(n_slots, d // group, device="cuda"))

        self.one, self.KV, self.hd, self.group, self.d = empty(), KV, hd, group, d
        self.two = empty() if two else None
        self.first, self.v_first = first, (first if two else first + width)
        self.dh = [(0.3 + torch.rand(d, generator=g, device="cuda")) if dhalf else None for _ in range(2)]
        if not two:
            self.dh[1] = self.dh[0]
        self.dhi = [None if v is None else 1.0 / v for v in self.dh]
        at = torch.arange(n_slots, device="cuda") if rows is None else rows
        for c, dh in zip((self.one, self.two), self.dh):
            if c is None:
                continue
            x = torch.randn(at.numel(), d, generator=g, device="cuda")
            x = x + 0.5 * torch.randn(d, generator=g, device="cuda")  # channels have means
            x = x * torch.exp2(spread * torch.randn(at.numel(), 1, generator=g, device="cuda"))
            ttq.ttq_cache_write(x, at, *c, dhalf=dh, **self.how)

    def kwargs(self):
        return dict(kv_heads=self.KV, k_first=self.first, v_first=self.v_first, v_cache=self.two,
                    dhalf_inv=self.dhi[0], v_dhalf_inv=self.dhi[1] if self.two else None, **self.how)

    def parts(self, rows, which):
        """(s c D^{-1/2}, m D^{-1/2}) of K (0) or V (1) of cache rows [n], float64
        [n, KV, hd]; E4M3: its m is 0."""
        codes, s, m = self.two if which and self.two else self.one
        at = (self.first, self.v_first)[which]
        b = codes[rows]
        if self.how["qformat"] == "fp8":
            q = b.view(torch.float8_e4m3fn).double()
        elif self.how["bits"] > 4:
            q = b.double()
        else:
            q = torch.stack((b & 15, b >> 4), -1).flatten(-2).double()
        rep = lambda t: t[rows].double().repeat_interleave(self.group, 1)
        dhi = 1.0 if self.dhi[which] is None else self.dhi[which].double()
        cut = slice(at, at + self.KV * self.hd)
        return [(v * dhi)[:, cut].unflatten(1, (self.KV, self.hd)) for v in (rep(s) * q, rep(m).clone())]


    def middle(self, rows, which):
        """What the middle of the codes, 2^(bits - 1), stands for without m: s mid D^{-1/2},
        as .parts; E4M3: 0."""
        s = (self.two if which and self.two else self.one)[1]
        at = (self.first, self.v_first)[which]
        mid = 0.0 if self.how["qformat"] == "fp8" else 2.0 ** (self.how["bits"] - 1)
        v = mid * s[rows].double().repeat_interleave(self.group, 1)
        v = v * (1.0 if self.dhi[which] is None else self.dhi[which].double())
        return v[:, at:at + self.KV * self.hd].unflatten(1, (self.KV, self.hd))


def reference(cache, Q, rows, n_keys, shift, scale, window=0, tile=False):
    """Float64 attention of one sequence's rows Q [n, H, hd] over cache rows `rows`
    (its keys, -1: not there), row r at position shift + r; and the bound of the error.

    The bound: (a) the result is rounded once to bf16.  (b) p is rounded to fp16 in
    the sum and the divisor alike, and for p < 2^-14 by 2^-25.
    (c) V's scales, offsets and the products of scales and codes are rounded to fp16
    (2^-11 each; and 2^-20 of the largest for values far below it, which fp16 holds as
    subnormals); what the scale's rounding leaves out is added for the middle of the
    codes, so that it is off by 2^-11 of s (c - mid), at most s c or s mid.
    (d) scores: q' is rounded to fp16 (exactly where it is bf16 and no D^{-1/2}
    enters, but for values 2^-14 below its largest), and hd + 8 float32 operations on
    terms s c q and m sum q; their error moves p by as much relatively.
    (e) tile (many rows share decoded keys): K is fp16(fp16(s) (c - mid) + fp16(m +
    mid s)), three roundings of 2^-11 of s (c - mid), of m + mid s and of their sum,
    where (d) has them exact; and its unit is such that the largest scale is 2^11 or
    more of the code's 2^-24, so what fp16 holds as a subnormal is off by 2^-25 of
    that, 2^-12 of the scale.  V alike."""
    n, H, hd = Q.shape
    G = H // cache.KV
    out, tol = torch.zeros(n, H, hd, dtype=torch.float64), torch.zeros(n, H, hd, dtype=torch.float64)
    rows = rows[:max(0, n_keys)]
    if rows.numel() == 0 or n == 0:
        return out, tol
    there = rows >= 0
    at = torch.arange(rows.numel(), device=rows.device)
    (ka, km), (va, vm) = (cache.parts(rows.clamp(min=0), w) for w in (0, 1))
    k_mid, v_mid = (cache.middle(rows.clamp(min=0), w) for w in (0, 1))
    pos = shift + torch.arange(n, device="cuda")[:, None]
    seen = (at <= pos) & there
    if window:
        seen &= at > pos - window
    any_seen = seen.any(1)
    for h in range(H):
        q = Q[:, h].double()
        K, V = ka[:, h // G] + km[:, h // G], va[:, h // G] + vm[:, h // G]
        t = scale * q @ K.T
        t = torch.where(seen, t, -math.inf)
        p = torch.softmax(t, 1)
        p = torch.where(seen, p, 0.0)
        o = p @ V
        top = torch.where(seen, t, -math.inf).amax(1, keepdim=True)
        e_p = 2 * HALF["f16"] * (p @ V.abs() + o.abs())
        e_p = e_p + 2.0 ** -24 * torch.where(seen, torch.exp(top * 0), 0.0).double() @ V.abs() \
            / torch.exp(t - top).sum(1, keepdim=True)
        e_v = HALF["f16"] * p @ (2 * va[:, h // G].abs() + vm[:, h // G].abs() + v_mid[:, h // G])
        qa = q.abs()
        terms = qa @ ka[:, h // G].abs().T + qa.sum(1, keepdim=True) * km[:, h // G].abs().amax(1)
        e_t = abs(scale) * ((HALF["f16"] if cache.dhi[0] is not None else 0.0) * 2 * terms
                       + (hd + 8) * HALF["f32"] * 2 * terms
                       + 2.0 ** -24 * qa.amax(1, keepdim=True) * (ka[:, h // G].abs() + km[:, h // G].abs()).sum(1))
        if tile:
            e_v = HALF["f16"] * p @ ((va - v_mid).abs() + (vm + v_mid).abs() + (va + vm).abs())[:, h // G]
            dhi = 1.0 if cache.dhi[0] is None else cache.dhi[0].double()[cache.first + h // G * hd:][:hd]
            top_s = cache.one[1].double().nan_to_num(0.0).amax()
            e_t = e_t + abs(scale) * (HALF["f16"] * qa @ ((ka - k_mid).abs() + (km + k_mid).abs() + (ka + km).abs())[:, h // G].T
                                      + 2.0 ** -12 * top_s * (qa * dhi).sum(1, keepdim=True))
        e_v = e_v + 2.0 ** -20 * torch.where(seen, V.abs().amax(1), 0.0).amax(1, keepdim=True)
        e_t = torch.where(seen, e_t + 2.0 ** -22 * t.abs(), 0.0)
        w = p * torch.expm1(2 * e_t.amax(1, keepdim=True))
        e_s = w @ V.abs() + w.sum(1, keepdim=True) * o.abs()
        o[~any_seen] = 0
        e = e_p + e_v + e_s
        e = e + HALF["bf16"] * (o.abs() + e)
        e[~any_seen] = 0
        out[:, h], tol[:, h] = o.cpu(), e.cpu()
    return out, tol
