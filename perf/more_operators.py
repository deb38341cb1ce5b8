"""Cases of the attention of a decoder whose K and V rows are kept quantized:
page tables and slot maps of a step from its request lengths
(``ttq_cache_extend``), norms and rotation of the query and key heads with the
K and V rows quantized into the cache in the same pass (``ttq_cache_rope``),
and attention over that cache (``ttq_cache_attention``).

``own`` false: the plain form, in elementary torch operations.  ``own`` true:
the library's entry points.  ``exact`` gives the same from the definition in
64 bits.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of eight requests, one of them ended: a step's first call
        dict(name="extend_step_8", op="extend", S=8, ctx=4096, prompts=False, page=16, T=8),
        # a batch of prompts that arrive together, packed into 65536 rows
        dict(name="extend_prompts_65536", op="extend", S=100, ctx=1500, prompts=True, page=16,
             T=65536),
        # one token of one request: latency of a call
        dict(name="rope_token", op="rope", T=1, H=32, KV=8, hd=128, rot=128, inter=False,
             norm=True, x="f32", bits=4, group=128, fmt="asym", dhalf=False, far=4096),
        # a decode step of 64 requests on a 7B-class layer (as many key heads as
        # query heads), no norms, codes of K D^{1/2}
        dict(name="rope_step_64", op="rope", T=64, H=32, KV=32, hd=128, rot=128, inter=False,
             norm=False, x="f32", bits=4, group=64, fmt="asym", dhalf=True, far=8192),
        # a prompt of 4096 tokens
        dict(name="rope_prompt_4096", op="rope", T=4096, H=32, KV=8, hd=128, rot=128,
             inter=False, norm=True, x="bf16", bits=4, group=128, fmt="asym", dhalf=False,
             far=4096),
        # an odd number of rows far into a context, small heads, half of each
        # rotated, neighbouring channels as pairs, E4M3 codes
        dict(name="rope_odd_1021", op="rope", T=1021, H=20, KV=5, hd=64, rot=32, inter=True,
             norm=True, x="f32", bits=8, group=32, fmt="fp8", dhalf=False, far=1000000),
        # one token of a small model: latency of a call
        dict(name="attention_token_500", op="attention", S=1, ctx=500, new=1, H=8, KV=2, hd=64,
             page=16, bits=4, group=64, fmt="asym", dhalf=False, window=0),
        # eight requests' decode step on a 7B-class layer, a key head a query head
        dict(name="attention_step_8", op="attention", S=8, ctx=4096, new=1, H=32, KV=32, hd=128,
             page=16, bits=4, group=128, fmt="asym", dhalf=False, window=0),
        # a large decode batch, four query heads a key head
        dict(name="attention_step_64", op="attention", S=64, ctx=8192, new=1, H=32, KV=8, hd=128,
             page=32, bits=4, group=128, fmt="asym", dhalf=False, window=0),
        # one request with a long context, codes of K D^{1/2} in groups of 64
        dict(name="attention_long_131071", op="attention", S=1, ctx=131071, new=1, H=64, KV=8,
             hd=128, page=64, bits=4, group=64, fmt="sym", dhalf=True, window=0),
        # prompts packed one after another, each attending to itself
        dict(name="attention_prompts_2047", op="attention", S=4, ctx=2047, new=2047, H=32, KV=8,
             hd=128, page=16, bits=4, group=128, fmt="asym", dhalf=False, window=0),
        # chunks of long prompts on a layer with a sliding window, E4M3 codes
        dict(name="attention_chunk_fp8", op="attention", S=2, ctx=16000, new=500, H=32, KV=8,
             hd=128, page=64, bits=8, group=32, fmt="fp8", dhalf=False, window=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _code(rng):
    fmt = rng.choice(("asym", "asym", "sym", "intzp", "fp8"))
    bits = 8 if fmt == "fp8" else rng.choice((3, 4, 4, 4, 8))
    return dict(fmt=fmt, bits=bits, group=rng.choice((32, 64, 128)), dhalf=rng.random() < 0.4)


def draw(rng):
    op = rng.choice(("extend", "rope", "attention", "attention"))
    if op == "extend":
        prompts = rng.random() < 0.5
        S = _log(rng, 1, 100 if prompts else 500)
        ctx = _log(rng, 2, 600)
        return dict(op=op, S=S, ctx=ctx, prompts=prompts, page=rng.choice((1, 8, 16, 32, 64)),
                    T=min(65536, S * ctx) if prompts else S + rng.choice((0, 3)))
    KV = rng.choice((1, 2, 4, 5, 8))
    heads = dict(KV=KV, H=KV * rng.choice((1, 1, 3, 4, 4, 8)), hd=rng.choice((64, 128, 128, 128, 256)))
    code = _code(rng)
    while KV * heads["hd"] % code["group"]:
        code["group"] //= 2
    if op == "rope":
        hd = heads["hd"]
        return dict(op=op, T=_log(rng, 1, 2048), **heads, rot=rng.choice((hd, hd, hd // 2, 48)),
                    inter=rng.random() < 0.3, norm=rng.random() < 0.6, x=rng.choice(("bf16", "f32")),
                    far=_log(rng, 100, 1000000), **code)
    S = _log(rng, 1, 32)
    ctx = _log(rng, 1, 65536 // S)
    new = 1 if rng.random() < 0.6 else _log(rng, 1, min(ctx, 1024))
    while S * new * ctx * heads["H"] > 2 ** 28:
        new = max(1, new // 2)
        ctx = ctx * 3 // 4 if new == 1 else ctx
    return dict(op=op, S=S, ctx=ctx, new=new, **heads, page=rng.choice((8, 16, 32, 64)),
                window=rng.choice((0, 0, 1 + ctx // 3)), **code)


def _lens(c):
    """Context lengths of a case: ragged, the first one the longest."""
    return [max(1, c["ctx"] - (i * 997) % (c["ctx"] // 2 + 1)) for i in range(c["S"])]


def _news(c):
    """Rows of this step of an attention case: ragged where they are several."""
    return [n if c["new"] >= c["ctx"] else min(n, max(1, c["new"] - (i * 61) % (c["new"] // 2 + 1)))
            for i, n in enumerate(_lens(c))]


def _container(bits):
    return 1 if bits <= 1 else 2 if bits <= 2 else 4 if bits <= 4 else 8


# ------------------------------------------------------- plain quantizer
def _bf16(x):
    return x.to(torch.bfloat16)


def _encode(u, bits, group, fmt):
    """Float32 rows [N, C] -> codes (integers; E4M3 patterns for fp8), scales
    and offsets by the group, float32, no fused operations."""
    v = u.reshape(u.shape[0], -1, group)
    mn, mx = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    N, Z = float(2 ** bits - 1), float(2 ** (bits - 1) - 1)
    zero = torch.zeros((), device=u.device)
    if fmt == "asym":
        s = (mx - mn) / N
    elif fmt == "intzp":
        s = (torch.maximum(mx, zero) - torch.minimum(mn, zero)) / N
    else:
        s = torch.maximum(-mn, mx) / (Z if fmt == "sym" else 448.0)
    inv = torch.where(s > 0, 1.0 / s, zero)
    if fmt == "asym":
        q, m = ((v - mn) * inv).round().clamp(0, N), mn
    elif fmt == "sym":
        q, m = (v * inv).round().clamp(-Z, Z) + Z, -(Z * s)
    elif fmt == "intzp":
        z = (torch.minimum(mn, zero) * inv).round()
        q, m = ((v * inv).round() - z).clamp(0, N), z * s
    else:
        q, m = (v * inv).clamp(-448, 448).to(F8).view(torch.uint8), torch.zeros_like(s)
    return q.reshape(u.shape).to(torch.uint8), s[..., 0], m[..., 0]


def _pack(q, bits):
    c = _container(bits)
    if c == 8:
        return q
    sh = torch.arange(8 // c, device=q.device, dtype=torch.int32) * c
    return (q.to(torch.int32).reshape(*q.shape[:-1], -1, 8 // c) << sh).sum(-1).to(torch.uint8)


def _decode(packed, s, m, dhi, c):
    """Rows of packed codes with their scales and offsets -> float32 values."""
    if c["fmt"] == "fp8":
        q = packed.view(F8).float()
    else:
        n = _container(c["bits"])
        sh = torch.arange(8 // n, device=packed.device, dtype=torch.uint8) * n
        q = ((packed[..., None] >> sh) & (2 ** n - 1)).flatten(-2).float()
    w = q.unflatten(-1, (-1, c["group"])).mul_(s[..., None]).add_(m[..., None]).flatten(-2)
    return w if dhi is None else w.mul_(dhi)


# --------------------------------------------------------------- prepare
def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == "extend":
        S, page, T, lens = c["S"], c["page"], c["T"], _lens(c)
        # prompts: empty sequences get what their request brings; else each gets
        # one token, but for one in eight, which has ended
        jitter = torch.randint(0, 5, (S,), generator=g, device=dev).tolist()
        lens = [max(1, n - j) for n, j in zip(lens, jitter)]
        added = [n if c["prompts"] else -1 if i % 8 == 5 else 1 for i, n in enumerate(lens)]
        lens = [0] * S if c["prompts"] else lens
        P = -(-c["ctx"] // page) + 1
        n_pages = S * P + 8
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        pages = torch.full((S, P), -1, dtype=torch.int32, device=dev)
        held = i32([-(-n // page) for n in lens])
        live = torch.arange(P, device=dev) < held[:, None]
        pages[live] = order[:int(live.sum())]
        rest = order[int(live.sum()):]
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        free[:rest.numel()] = rest

        def empty(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=dev)

        return dict(case=c, lens=i32(lens), added=i32(added), pages=pages, free=free,
                    count=i32([rest.numel()]),
                    out=(empty(S), empty(1), empty(S + 1), empty(T), empty(T, torch.int64)))

    H, KV, hd, bits, group, fmt = (c[k] for k in ("H", "KV", "hd", "bits", "group", "fmt"))
    C = 2 * KV * hd  # K and V of a token side by side
    dh = (0.2 + randn(C).abs()) ** 0.25 if c["dhalf"] else None

    def cache(n):
        return [torch.zeros(n, C * _container(bits) // 8, dtype=torch.uint8, device=dev),
                torch.zeros(n, C // group, device=dev), torch.zeros(n, C // group, device=dev)]

    if c["op"] == "rope":
        T = c["T"]
        X = randn(T, (H + 2 * KV) * hd)  # as the projection leaves Q, K and V
        n_slots = -(-T // 16) * 16 + 32
        slots = torch.randperm(n_slots // 16, generator=g, device=dev)[:, None] * 16 \
            + torch.arange(16, device=dev)
        slots = slots.reshape(-1)[:T].contiguous()
        first = int(torch.randint(0, c["far"], (1,), generator=g, device=dev))
        return dict(case=c, X=_bf16(X) if c["x"] == "bf16" else X, slots=slots,
                    positions=(first + torch.arange(T, device=dev)).to(torch.int32),
                    inv_freq=(10000.0 ** (-torch.arange(0, c["rot"], 2, device=dev).double()
                                          / c["rot"])).float(),
                    wq=1 + 0.1 * randn(hd) if c["norm"] else None,
                    wk=1 + 0.1 * randn(hd) if c["norm"] else None,
                    cache=cache(n_slots), dh=dh, dhi=None if dh is None else 1.0 / dh,
                    pages=slots.to(torch.int32)[None].contiguous(), lens=i32([T]),
                    out=torch.empty(T, H, hd, dtype=torch.bfloat16, device=dev))

    S, page, lens, news = c["S"], c["page"], _lens(c), _news(c)
    P = -(-c["ctx"] // page)
    pages = torch.randperm(S * P, generator=g, device=dev).view(S, P).to(torch.int32)
    kv = cache(S * P * page)
    for k in range(0, S * P * page, 16384):  # every row of the cache is some token's
        n = min(16384, S * P * page - k)
        x = _bf16(randn(n, C)).float()
        q, s, m = _encode(x if dh is None else x * dh, bits, group, fmt)
        for t, v in zip(kv, (_pack(q, bits), s, m)):
            t[k:k + n] = v
    T = sum(news)
    return dict(case=c, Q=_bf16(2 * randn(T, H, hd)), cache=kv, pages=pages, lens=i32(lens),
                offsets=torch.cat((i32([0]), i32(news).cumsum(0).to(torch.int32))),
                dhi=None if dh is None else 1.0 / dh,
                out=torch.empty(T, H, hd, dtype=torch.bfloat16, device=dev))


# ----------------------------------------------------------------- plain
def _plain_extend(st):
    c, pages, free = st["case"], st["pages"], st["free"]
    page, T, (S, P) = c["page"], c["T"], pages.shape
    dev, n_pages = pages.device, free.numel()
    lens, added, c0 = st["lens"].long(), st["added"].long(), st["count"].long().clamp(0, n_pages)
    zero = torch.zeros((), dtype=torch.int64, device=dev)
    lens = torch.where(lens < 0, -1 - lens, lens)
    held, ends, adds = torch.clamp((lens + page - 1) // page, max=P), added < 0, added.clamp(min=0)
    k = torch.arange(P, device=dev)

    def scattered(into, at, value, where):
        """into[at] = value where it says so (the others go to a cell behind)."""
        more = torch.cat((into.reshape(-1), into.reshape(-1)[:1]))
        more[torch.where(where, at, into.numel())] = value
        return more[:-1].view_as(into)

    # the pages of sequences that end, on top of the free ones
    gone = torch.where(ends, held, zero)
    at = c0 + (gone.cumsum(0) - gone)[:, None] + k
    stack = scattered(free, at, pages, (k < gone[:, None]) & (at < n_pages))
    top = torch.clamp(c0 + gone.sum(), max=n_pages)
    # what the others need, the first ones first
    rows = adds.cumsum(0)
    want = (lens + adds + page - 1) // page
    too = ends | (want > P) | (rows > T)
    need = torch.where(too, zero, want - held)
    got = need.cumsum(0)
    refused = ((too & ~ends) | ((got > top) & (need > 0))) & (adds > 0)
    need = torch.where(refused, zero, need)
    new = (k >= held[:, None]) & (k < (held + need)[:, None])
    at = top - 1 - ((got - need)[:, None] + k - held[:, None])
    table = torch.where(new, stack[at.clamp(0, n_pages - 1)], pages)
    t = torch.arange(T, device=dev)
    i = torch.searchsorted(rows, t, right=True).clamp(max=S - 1)
    live = t < rows[-1]
    pos = torch.where(live, lens[i] + t - (rows[i] - adds[i]), zero)
    slot = table[i, (pos // page).clamp(max=P - 1)].long() * page + pos % page
    pages.copy_(table)
    free.copy_(stack)
    lens_out, count, offsets, positions, slots = st["out"]
    lens_out.copy_(torch.where(ends, zero, torch.where(refused, -1 - lens, lens + adds)))
    count.copy_(top - need.sum())
    offsets.copy_(torch.cat((zero[None], rows)).clamp(max=T))
    positions.copy_(pos)
    slots.copy_(torch.where(live & ~refused[i], slot, -1))
    return st["out"] + (pages, free)


def _plain_rope(st):
    c = st["case"]
    T, H, KV, hd, rot = (c[k] for k in ("T", "H", "KV", "hd", "rot"))
    X = st["X"].float().view(T, H + 2 * KV, hd)

    def normed(x, w):
        if w is None:
            return x
        r = (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt().float()
        return x * r * w

    angle = st["positions"].double()[:, None, None] * st["inv_freq"].double()
    co, si = angle.cos().float(), angle.sin().float()

    def rotated(x):
        x, rest = x[..., :rot], x[..., rot:]
        a, b = (x[..., ::2], x[..., 1::2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:])
        y = (a * co - b * si, b * co + a * si)
        y = torch.stack(y, -1).flatten(-2) if c["inter"] else torch.cat(y, -1)
        return torch.cat((y, rest), -1)

    st["out"].copy_(rotated(normed(X[:, :H], st["wq"])))
    kv = torch.cat((rotated(normed(X[:, H:H + KV], st["wk"])), X[:, H + KV:]), 1).flatten(1)
    q, s, m = _encode(kv if st["dh"] is None else kv * st["dh"], c["bits"], c["group"], c["fmt"])
    for t, v in zip(st["cache"], (_pack(q, c["bits"]), s, m)):
        t[st["slots"]] = v
    return st["out"], _bf16(_decode(*[t[st["slots"]] for t in st["cache"]], st["dhi"], c))[None]


def _plain_attention(st):
    c = st["case"]
    S, H, KV, hd, page, ctx = (c[k] for k in ("S", "H", "KV", "hd", "page", "ctx"))
    dev, off, lens = st["Q"].device, st["offsets"].long(), st["lens"].long()
    t = torch.arange(ctx, device=dev)
    rows = st["pages"].long()[:, t // page] * page + t % page
    kv = _decode(*[v[rows] for v in st["cache"]], st["dhi"], c).view(S, ctx, 2, KV, hd)
    # the rows of each sequence, padded to as many
    N = max(_news(c))
    n, j = off[1:] - off[:-1], torch.arange(N, device=dev)
    at = (off[:-1, None] + j).clamp(max=st["Q"].shape[0] - 1)
    Q = st["Q"][at].float().view(S, N, KV, H // KV, hd)
    p = torch.matmul(Q.permute(0, 2, 3, 1, 4).reshape(S, KV, -1, hd),
                     kv[:, :, 0].permute(0, 2, 3, 1)).view(S, KV, H // KV, N, ctx)
    p *= hd ** -0.5
    pos = (lens - n)[:, None] + j
    seen = (t <= pos[..., None]) & (j < n[:, None])[..., None]
    if c["window"]:
        seen &= t > pos[..., None] - c["window"]
    seen = seen[:, None, None]
    p = p.masked_fill_(~seen, -math.inf)
    p = (p - p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, KV, -1, ctx), kv[:, :, 1].permute(0, 2, 1, 3).contiguous())
    o = o.view(S, KV, H // KV, N, hd) / total.clamp(min=1e-37)
    seq = torch.searchsorted(off[1:], torch.arange(st["Q"].shape[0], device=dev), right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, N, H, hd)
    st["out"].copy_(o[seq, torch.arange(st["Q"].shape[0], device=dev) - off[seq]])
    return st["out"]


def run(state):
    op = state["case"]["op"]
    if not own:
        return dict(extend=_plain_extend, rope=_plain_rope, attention=_plain_attention)[op](state)
    import online_activation_aware_ttq_amd as ttq
    st, c = state, state["case"]
    if op == "extend":
        lens, count, offsets, positions, slots = st["out"]
        ttq.ttq_cache_extend(st["lens"], st["added"], st["pages"], st["free"], st["count"],
                             page_tokens=c["page"], lens_out=lens, free_count_out=count,
                             offsets=offsets, positions=positions, slots=slots)
        return st["out"] + (st["pages"], st["free"])
    how = dict(bits=c["bits"], group=c["group"], qformat=c["fmt"])
    if op == "rope":
        a, b = c["H"] * c["hd"], (c["H"] + c["KV"]) * c["hd"]
        X = st["X"]
        ttq.ttq_cache_rope(X[:, :a], X[:, a:b], X[:, b:], st["positions"], st["slots"],
                           *st["cache"], head_dim=c["hd"], inv_freq=st["inv_freq"],
                           interleaved=c["inter"], q_weight=st["wq"], k_weight=st["wk"],
                           eps=1e-6, dhalf=st["dh"], out=st["out"], **how)
        return st["out"], ttq.ttq_cache_read(*st["cache"], st["pages"], st["lens"], page_tokens=1,
                                             dhalf_inv=st["dhi"], dtype=torch.bfloat16, **how)
    return ttq.ttq_cache_attention(st["Q"], st["pages"], st["lens"], *st["cache"],
                                   kv_heads=c["KV"], page_tokens=c["page"],
                                   offsets=None if c["new"] == 1 else st["offsets"],
                                   window=c["window"], dhalf_inv=st["dhi"], out=st["out"], **how)


# ------------------------------------------------------------------ work
def _seen(c):
    """Per sequence: its rows, the keys that any of them sees, and the pairs."""
    for n, new in zip(_lens(c), _news(c)):
        w = c["window"] or n
        yield new, min(n, new - 1 + w), sum(min(p + 1, w) for p in range(n - new, n))


def work(case):
    c = case
    if c["op"] == "extend":
        rows = min(c["T"], sum(_lens(c)) if c["prompts"] else c["S"])
        return dict(bytes=12 * c["T"] + 16 * c["S"] + 8 * (rows // c["page"] + c["S"]), flops=0)
    per = _container(c["bits"]) / 8 + 8 / c["group"]  # bytes a channel of a cache row
    C = 2 * c["KV"] * c["hd"]
    if c["op"] == "rope":
        size, w = dict(bf16=2, f32=4)[c["x"]], c["H"] * c["hd"]
        return dict(bytes=c["T"] * ((w + C) * size + 2 * w + 2 * C * per + 2 * C + 12),
                    flops=c["T"] * 12 * (w + C))
    rows = [v for v in _seen(c)]
    return dict(bytes=sum(k for _, k, _ in rows) * C * per + sum(r for r, _, _ in rows) * 4 * c["H"] * c["hd"],
                flops=4 * c["H"] * c["hd"] * sum(p for _, _, p in rows))


# ----------------------------------------------------------------- exact
def _r(x):
    """One float32 rounding of a value in 64 bits."""
    return x.float().double()


def _levels64(packed, bits, fmt):
    b = packed.long()
    if fmt == "fp8":
        mag, e = (b & 7).double(), ((b >> 3) & 15)
        v = torch.where(e > 0, (8 + mag) * 2.0 ** (e.double() - 10), mag * 2.0 ** -9)
        return torch.where(b >= 128, -v, v)
    n = _container(bits)
    return torch.stack([(b >> (n * i)) & ((1 << n) - 1) for i in range(8 // n)], -1).flatten(-2).double()


def _requantized64(u, bits, group, fmt):
    """What the quantizer leaves of rows u: its definition decides the codes in
    float32 operations, each rounded once, so that a value next to a border has
    one answer; what the codes stand for is 64 bits."""
    v = _r(u).unflatten(-1, (-1, group))
    lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    top, Z = 2 ** bits - 1, 2 ** (bits - 1) - 1
    # the range times the float32 nearest to one part of it
    part = float(_r(torch.tensor(1.0 / {"sym": Z, "fp8": 448}.get(fmt, top), dtype=torch.float64)))
    if fmt == "asym":
        s = _r(_r(hi - lo) * part)
    elif fmt == "intzp":
        s = _r(_r(hi.clamp(min=0) - lo.clamp(max=0)) * part)
    else:
        s = _r(v.abs().max(-1, keepdim=True).values * part)
    inv = _r(1 / torch.where(s > 0, s, torch.inf))
    t = _r(_r(v - lo) * inv) if fmt == "asym" else _r(v * inv)
    if fmt == "asym":
        w = lo + s * torch.round(t).clamp(0, top)
    elif fmt == "sym":
        w = s * torch.round(t).clamp(-Z, Z)
    elif fmt == "intzp":
        z = torch.round(_r(lo.clamp(max=0) * inv))
        w = s * torch.round(t).clamp(min=z, max=z + top)
    else:
        t = t.clamp(-448, 448)
        step = 2.0 ** (torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        w = s * torch.round(t / step) * step
    return w.flatten(-2)


def _exact_extend(st):
    """One sequence after another, one page after another, on the host."""
    c = st["case"]
    page, T = c["page"], c["T"]
    lens, added, table, free = (st[k].tolist() for k in ("lens", "added", "pages", "free"))
    top, cap = int(st["count"]), len(free)
    lens = [-1 - n if n < 0 else n for n in lens]
    for i, a in enumerate(added):
        if a < 0:
            for p in table[i][:-(-lens[i] // page)]:
                if top < cap:
                    free[top] = p
                    top += 1
    lens_out, offsets, positions, slots, short = [], [0], [], [], False
    for i, (n, a) in enumerate(zip(lens, added)):
        if a < 0:
            lens_out.append(0)
            offsets.append(offsets[-1])
            continue
        fits = -(-(n + a) // page) <= len(table[i]) and len(positions) + a <= T
        need = -(-(n + a) // page) - -(-n // page) if fits else 0
        short = short or need > top
        fits = fits and not (short and need)
        for k in range(need if fits else 0):
            top -= 1
            table[i][-(-n // page) + k] = free[top]
        for q in range(n, n + a):
            positions.append(q)
            slots.append(table[i][q // page] * page + q % page if fits else -1)
        lens_out.append(n + a if fits or a == 0 else -1 - n)
        offsets.append(len(positions))
    positions, slots = ((v + [e] * T)[:T] for v, e in ((positions, 0), (slots, -1)))
    dev = st["lens"].device
    outs = [torch.tensor(v, device=dev) for v in (lens_out, [top], [min(o, T) for o in offsets],
                                                  positions, slots, table, free)]
    return tuple(v.to(torch.int64 if k == 4 else torch.int32) for k, v in enumerate(outs))


def _exact_rope(st):
    c = st["case"]
    T, H, KV, hd, rot = (c[k] for k in ("T", "H", "KV", "hd", "rot"))
    X, pairs = st["X"].double().view(T, H + 2 * KV, hd), torch.arange(rot // 2, device="cuda")
    first = 2 * pairs if c["inter"] else pairs
    second = first + (1 if c["inter"] else rot // 2)
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    co, si = torch.cos(angle)[:, None], torch.sin(angle)[:, None]

    def heads(x, w, r):
        """r: what the definition rounds to float32 before the codes are decided
        (for the queries, which are only rounded once more, nothing)."""
        if w is not None:
            x = r(r(x * r(1 / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + 1e-6))) * w.double())
        y = x.clone()
        a, b = x[..., first], x[..., second]
        y[..., first] = r(r(a * r(co)) - r(b * r(si)))
        y[..., second] = r(r(b * r(co)) + r(a * r(si)))
        return y

    Q = heads(X[:, :H], st["wq"], lambda x: x)
    kv = torch.cat((heads(X[:, H:H + KV], st["wk"], _r), X[:, H + KV:]), 1).flatten(1)
    got = _requantized64(kv if st["dh"] is None else kv * st["dh"].double(), c["bits"], c["group"], c["fmt"])
    return Q, (got if st["dhi"] is None else got * st["dhi"].double())[None]


def _exact_attention(st):
    c = st["case"]
    H, KV, hd, page, G = c["H"], c["KV"], c["hd"], c["page"], c["H"] // c["KV"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device="cuda")
    done = 0
    for i, (n, new) in enumerate(zip(_lens(c), _news(c))):
        t = torch.arange(n, device="cuda")
        at = st["pages"][i].long()[torch.div(t, page, rounding_mode="floor")] * page + t % page
        codes, s, m = (v[at] for v in st["cache"])
        kv = m.double()[..., None] + s.double()[..., None] * _levels64(codes, c["bits"], c["fmt"]).unflatten(
            -1, (-1, c["group"]))
        kv = kv.flatten(-2) if st["dhi"] is None else kv.flatten(-2) * st["dhi"].double()
        for h in range(H):
            K, V = (kv[:, (b * KV + h // G) * hd:(b * KV + h // G + 1) * hd] for b in (0, 1))
            for lo in range(0, new, 2048):
                hi = min(new, lo + 2048)
                w = st["Q"][done + lo:done + hi, h].double() @ K.t() / math.sqrt(hd)
                pos = n - new + torch.arange(lo, hi, device="cuda")[:, None]
                seen = (t <= pos) & (t > pos - (c["window"] or n))
                out[done + lo:done + hi, h] = torch.softmax(torch.where(seen, w, -math.inf), 1) @ V
        done += new
    return out


def exact(case, seed):
    return dict(extend=_exact_extend, rope=_exact_rope,
                attention=_exact_attention)[case["op"]](prepare(case, seed))
