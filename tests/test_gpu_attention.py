"""ttq_cache_attention on the GPU against float64 attention over what the stored
codes stand for, within the bound that tests/attention_util.py derives from the
kernel's roundings."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _i32(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(case, seed=0, spread=0.0, q_sigma=2.0, **kw):
    """One call and the largest error in units of its bound."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache, reference
    H, KV, hd, bits, group, fmt, page, lens, news, window, dhalf, two = case
    print(f"[case] attention H={H}/{KV} hd={hd} b{bits} g{group} {fmt} page={page} lens={lens} "
          f"news={news} window={window}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(seed + sum(lens) + hd)
    S = len(lens)
    P = max(1, -(-max(max(lens), 1) // page)) + 1
    n_slots = S * P * page
    pages = torch.randperm(S * P, generator=g, device="cuda").view(S, P).to(torch.int32)
    cache = Cache(g, n_slots, KV, hd, bits, group, fmt, dhalf, two, first=group, spread=spread)
    T = sum(news)
    wide = torch.randn(T + 2, H * hd + 64, generator=g, device="cuda").mul_(q_sigma).bfloat16()
    Q = wide[:T + 2, 32:32 + H * hd].unflatten(1, (H, hd))  # rows apart, two of no sequence
    off = _i32(np.concatenate([[0], np.cumsum(news)]).tolist())
    out = torch.full((T + 2, H, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    single = all(n == 1 for n in news)
    if single:
        Q, out = Q[:T], out[:T]
    r = ttq.ttq_cache_attention(Q, pages, _i32(lens), *cache.one, page_tokens=page, out=out,
                                offsets=None if single else off, window=window, **cache.kwargs(), **kw)
    torch.cuda.synchronize()
    assert r is out
    if not single:
        assert (out[T:] == 3).all()  # rows of no sequence as they were
    worst = 0.0
    for i in range(S):
        n = max(lens[i], 0)
        t = torch.arange(n, device="cuda")
        rows = pages[i].long()[t // page] * page + t % page
        a, b = int(off[i]), int(off[i + 1])
        ref, tol = reference(cache, Q[a:b], rows, n, n - news[i], kw.get("scale", hd ** -0.5), window,
                             tile=T * (H // KV) >= 64 * S)
        got = out[a:b].double().cpu()
        err = (got - ref).abs()
        assert torch.isfinite(got).all()
        assert (err <= tol).all(), (i, float((err - tol).max()), float(err.max()))
        worst = max(worst, float((err / tol.clamp(min=1e-30)).max()) if err.numel() else 0.0)
    print(f"  largest error {worst:.2f} of its bound", flush=True)
    return worst


CASES = [
    # H, KV, hd, bits, group, fmt, page, lens, rows, window, D, two caches
    (1, 1, 64, 4, 64, "asym", 16, [1], [1], 0, False, False),
    (8, 2, 128, 4, 128, "asym", 16, [1, 31, 32, 33, 100], [1] * 5, 0, False, False),
    (4, 4, 128, 4, 128, "asym", 16, [700, 1, 0, 257], [1] * 4, 0, False, False),
    (32, 8, 128, 4, 128, "asym", 16, [1000], [1], 0, False, True),
    (8, 8, 64, 4, 128, "sym", 8, [77, 500], [1, 1], 0, True, False),      # a group of two heads
    (6, 2, 256, 4, 256, "intzp", 32, [65, 300], [1, 1], 0, True, False),
    (6, 2, 256, 4, 32, "asym", 1, [65, 130], [1, 1], 0, False, False),    # a row a page
    (8, 1, 128, 4, 32, "asym", 2, [190], [1], 0, True, True),
    (20, 1, 64, 3, 32, "asym", 64, [129], [1], 0, False, False),          # 20 heads on one
    (4, 2, 128, 4, 64, "asym", 4096, [5000], [1], 0, False, False),
    (3, 3, 128, 8, 128, "asym", 16, [99, 64], [1, 1], 0, False, False),
    (4, 1, 64, 8, 32, "sym", 16, [333], [1], 0, True, False),
    (4, 2, 256, 6, 64, "intzp", 16, [140], [1], 0, False, False),
    (4, 2, 128, 8, 32, "fp8", 16, [222, 8], [1, 1], 0, False, False),
    (4, 2, 64, 8, 64, "fp8", 16, [500], [1], 0, True, True),
    (2, 1, 256, 8, 256, "fp8", 16, [97], [1], 0, False, False),
    # windows
    (4, 2, 128, 4, 128, "asym", 16, [300, 5, 33, 64], [1] * 4, 1, False, False),
    (4, 2, 128, 4, 128, "asym", 16, [300, 5, 33, 64], [1] * 4, 33, False, False),
    (4, 2, 64, 8, 64, "fp8", 16, [200, 77], [50, 77], 20, False, False),
    # several rows a sequence: prompts, chunks, a mixture, more rows than keys
    (4, 2, 128, 4, 128, "asym", 16, [37], [37], 0, False, False),
    (8, 2, 128, 4, 128, "asym", 16, [150, 64, 1, 33], [150, 64, 1, 33], 0, False, False),
    (6, 2, 64, 4, 32, "asym", 8, [300, 9, 70, 130], [7, 1, 0, 129], 0, True, False),
    (4, 4, 256, 4, 64, "asym", 16, [130, 200], [130, 17], 0, False, True),
    (2, 1, 128, 8, 32, "fp8", 64, [520], [260], 100, False, False),
    (5, 5, 128, 4, 128, "asym", 16, [4, 0, -3, 10], [6, 2, 1, 10], 0, False, False),
    (4, 2, 128, 8, 128, "asym", 16, [400, 260], [300, 260], 0, True, False),
    (8, 8, 64, 4, 64, "sym", 16, [777], [500], 0, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])) + f"-{sum(c[8])}of{sum(c[7])}w{c[9]}")
def test_against_float64(case):
    _run(case)


@pytest.mark.parametrize("lens,news", [([20000], [1]), ([9001, 3, 40, 4096], [1] * 4), ([6000], [40])])
def test_long_contexts(lens, news):
    _run((8, 2, 128, 4, 128, "asym", 64, lens, news, 0, False, False))
    _run((4, 2, 64, 8, 32, "fp8", 16, lens, news, 1000, True, False))


@pytest.mark.parametrize("fmt,bits", [("asym", 4), ("fp8", 8), ("sym", 8)])
def test_rows_of_very_different_size(fmt, bits):
    """Tokens whose rows differ by powers of two of normal spread 3 (factors of
    1000 among them), and scores of every size."""
    for q in (1e-3, 2.0, 30.0):
        _run((4, 2, 128, bits, 32, fmt, 16, [400, 70], [1, 40], 0, False, False), seed=3, spread=3.0, q_sigma=q)


def test_scale_and_bound_on_the_lengths():
    case = (4, 2, 128, 4, 128, "asym", 16, [500, 90], [1, 1], 0, False, False)
    _run(case, scale=0.5)
    _run(case, scale=-0.1)
    _run(case, max_len=500)
    _run(case, max_len=1 << 40)


def _small(n_slots=64, KV=2, hd=64, bits=4, group=32, fmt="asym", seed=0):
    import torch
    from attention_util import Cache
    g = torch.Generator(device="cuda").manual_seed(seed)
    return Cache(g, n_slots, KV, hd, bits, group, fmt), torch.randn(4, 4, hd, generator=g, device="cuda").bfloat16()


def _call(cache, Q, pages, lens, page=16, **kw):
    import online_activation_aware_ttq_amd as ttq
    return ttq.ttq_cache_attention(Q, pages, _i32(lens), *cache.one, page_tokens=page, **cache.kwargs(), **kw)


def test_pages_outside_the_cache_are_not_seen():
    """They count as keys that are not there; a row with no other is 0."""
    import torch
    from attention_util import reference
    cache, Q = _small()
    pages = _i32([[0, 99, 2], [4, -1, 1 << 30], [1, 2, 3], [3, 2, -5]])
    lens = [48, 40, 48, 35]
    out = _call(cache, Q, pages, lens)
    assert (out[1] == 0).all()
    for i, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        p = pages[i].long()[t // 16]
        rows = torch.where((p >= 0) & (p < 4), p * 16 + t % 16, -1)
        ref, tol = reference(cache, Q[i:i + 1], rows, n, n - 1, 0.125)
        assert ((out[i:i + 1].double().cpu() - ref).abs() <= tol).all()
    # lengths past the table are cut to it, as is a bound of the caller's
    same = Q[:1].repeat(4, 1, 1)
    far = _call(cache, same, pages[2:3].repeat(4, 1).contiguous(), [48, 1 << 30, 49, 2 ** 31 - 1])
    for k in (1, 2, 3):
        assert torch.equal(far[k], far[0])
    short = _call(cache, Q[:1], pages[2:3].contiguous(), [20], max_len=20)
    assert torch.equal(short, _call(cache, Q[:1], pages[2:3].contiguous(), [20]))


@pytest.mark.parametrize("fmt,bits", [("asym", 4), ("fp8", 8), ("intzp", 8)])
@pytest.mark.parametrize("rows", [1, 9, 40])
def test_nan_of_unseen_keys_stays_out(fmt, bits, rows):
    """NaN in the rows behind the length, of other sequences, before the window and
    of later tokens; and a seen one makes NaN of what it enters, and no more."""
    import torch
    cache, _ = _small(n_slots=128, bits=bits, fmt=fmt)
    g = torch.Generator(device="cuda").manual_seed(9)
    Q = torch.randn(rows, 4, 64, generator=g, device="cuda").bfloat16()
    pages, off, n = _i32([[5, 0, 3, 6]]), _i32([0, rows]), 50
    kw = dict(offsets=off, window=0)
    clean = _call(cache, Q, pages, [n], **kw)
    codes, s, m = cache.one
    keep = s.clone(), m.clone()
    nan = float("nan")
    at = [5 * 16 + t if t < 16 else t - 16 if t < 32 else 3 * 16 + t - 32 if t < 48 else 6 * 16 + t - 48
          for t in range(64)]
    used = torch.zeros(128, dtype=torch.bool, device="cuda")
    used[at[:n]] = True
    s[~used] = nan
    m[~used] = nan
    assert torch.equal(_call(cache, Q, pages, [n], **kw), clean)
    # the newest row's own V, the first group of head 1
    gv = cache.v_first // 32 + 2
    s[at[n - 1], gv] = m[at[n - 1], gv] = nan
    got = _call(cache, Q, pages, [n], **kw)
    bad = torch.isnan(got.float())
    assert not bad[:-1].any() and not bad[-1, :2].any()
    assert bad[-1, 2:, :32].all() and not bad[-1, 2:, 32:].any()
    assert torch.equal(got[~bad], clean[~bad])
    s[at[n - 1], gv], m[at[n - 1], gv] = keep[0][at[n - 1], gv], keep[1][at[n - 1], gv]
    # its K, head 0
    s[at[n - 1], 0] = nan
    got = _call(cache, Q, pages, [n], **kw)
    bad = torch.isnan(got.float())
    assert bad[-1, :2].all() and not bad[-1, 2:].any() and not bad[:-1].any()
    # behind a window
    s[at[n - 1], 0] = keep[0][at[n - 1], 0]
    s[at[:4]] = nan
    want = _call(cache, Q, pages, [n], offsets=off, window=5)
    assert torch.isfinite(want.float()).all() or n - rows - 4 < 4
    s.copy_(keep[0])
    m.copy_(keep[1])
    if n - rows - 4 >= 4:
        assert torch.equal(want, _call(cache, Q, pages, [n], offsets=off, window=5))


def test_queries_that_are_not_finite():
    import torch
    cache, Q = _small()
    pages = _i32([[0, 1, 2]]).repeat(4, 1).contiguous()
    clean = _call(cache, Q, pages, [40] * 4)
    Q[1, 2, 7] = float("nan")
    Q[2, 0, 3] = float("inf")
    got = _call(cache, Q, pages, [40] * 4)
    bad = torch.isnan(got.float()).all(-1).cpu()
    want = torch.zeros(4, 4, dtype=torch.bool)
    want[1, 2] = want[2, 0] = True
    assert torch.equal(bad, want)
    assert torch.equal(got[~bad], clean[~bad])


def test_zero_queries_and_constant_rows():
    """Equal scores give the mean; rows of one value (scale 0) read as themselves."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    cache, Q = _small()
    x = torch.full((64, cache.d), 0.75, device="cuda")
    ttq.ttq_cache_write(x, torch.arange(64, device="cuda"), *cache.one, **cache.how)
    pages = _i32([[0, 1, 2]]).repeat(4, 1).contiguous()
    out = _call(cache, Q.zero_(), pages, [40, 1, 33, 17])
    assert ((out.float() - 0.75).abs() <= 0.75 * 2 ** -7).all()
    for c in (x.zero_(), x + 3e4, x + 1e30, x + 1e-30):
        ttq.ttq_cache_write(c, torch.arange(64, device="cuda"), *cache.one, **cache.how)
        out = _call(cache, Q, pages, [40, 1, 33, 17])
        assert ((out.double() - c[0, 0].double()).abs() <= c[0, 0].double().abs() * 2 ** -7).all()


def test_rows_past_2_to_31_bytes():
    """Byte offsets of a long cache pass 32 bits."""
    import torch
    from attention_util import Cache, reference
    g = torch.Generator(device="cuda").manual_seed(4)
    KV, hd, n_slots = 32, 128, (1 << 19) + 64   # 4 GiB of 8-bit codes, K and V
    rows = torch.tensor([7, (1 << 18) + 3, n_slots - 1, 1 << 19, 12], device="cuda")
    cache = Cache(g, n_slots, KV, hd, 8, 128, "asym", rows=rows)
    assert cache.one[0].numel() > 1 << 32
    Q = torch.randn(1, KV, hd, generator=g, device="cuda").bfloat16()
    out = _call(cache, Q, rows.to(torch.int32)[None].contiguous(), [5], page=1)
    ref, tol = reference(cache, Q, rows, 5, 4, hd ** -0.5)
    assert ((out.double().cpu() - ref).abs() <= tol).all()


def test_captured_on_other_streams():
    """Two graphs of calls whose ranges are joined in a workspace, replayed at once,
    and calls on a stream given as argument: the eager call's bits."""
    import torch
    cache, _ = _small(n_slots=8192, KV=2, hd=128, group=128)
    g = torch.Generator(device="cuda").manual_seed(2)
    state = []
    for k in range(2):
        Q = torch.randn(3, 4, 128, generator=g, device="cuda").bfloat16()
        pages = torch.randperm(512, generator=g, device="cuda")[:510].view(3, 170).to(torch.int32).contiguous()
        state.append((Q, pages, _i32([2000, 5, 700]), torch.zeros_like(Q)))
    import online_activation_aware_ttq_amd as ttq

    def call(k, **kw):
        Q, pages, lens, out = state[k]
        return ttq.ttq_cache_attention(Q, pages, lens, *cache.one, page_tokens=16, **cache.kwargs(), **kw)

    call(0)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(k, out=state[k][3])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for step in range(4):
        for Q, pages, lens, out in state:
            Q.normal_()
            lens.copy_(_i32([100 * step, 2700 - step, 0 if step == 2 else 64]))
            out.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        got = [st[3].clone() for st in state]
        for k in range(2):
            a, b = call(k), call(k, stream=streams[k].cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(got[k], a) and torch.equal(a, b)


def test_repeated_calls_have_equal_bits():
    import torch
    cache, _ = _small(n_slots=4096, KV=2, hd=128, group=64)
    g = torch.Generator(device="cuda").manual_seed(2)
    Q = torch.randn(70, 4, 128, generator=g, device="cuda").bfloat16()
    pages = torch.arange(256, dtype=torch.int32, device="cuda")[None]
    for off in ([0, 70], [0, 1]):
        q = Q[:off[1]]
        first = _call(cache, q, pages, [4000], offsets=_i32(off))
        for _ in range(5):
            assert torch.equal(_call(cache, q, pages, [4000], offsets=_i32(off)), first)
