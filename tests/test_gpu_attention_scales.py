"""Keys whose scales are far apart: each row's result is right by a bound that goes key by
key (tests/attention_bounds.py), and no row depends on the size of a key it does not see."""
import pytest

pytestmark = pytest.mark.gpu

FORMS = [
    # H, KV, hd, bits, group, fmt, rows of len, D, two caches
    (4, 1, 64, 4, 64, "asym", 200, 400, False, False),
    (4, 1, 64, 3, 32, "asym", 150, 300, False, False),
    (8, 2, 128, 8, 32, "sym", 200, 333, False, False),
    (4, 1, 128, 8, 128, "fp8", 200, 250, True, False),
    (4, 1, 128, 4, 128, "asym", 200, 200, False, True),
    (2, 1, 256, 4, 64, "intzp", 150, 150, False, False),
    # ranges of keys: a group a head (a half of two heads' too), and several
    (4, 2, 128, 4, 128, "asym", 1, 300, False, False),
    (8, 4, 64, 4, 128, "intzp", 7, 200, False, True),
    (6, 3, 64, 3, 64, "asym", 9, 150, True, False),
    (2, 1, 256, 8, 256, "sym", 5, 100, False, False),
    (4, 1, 128, 8, 128, "fp8", 3, 250, True, False),
    (4, 2, 128, 4, 32, "asym", 9, 300, False, False),
    (4, 1, 64, 8, 32, "asym", 1, 200, False, True),
    (8, 2, 128, 8, 64, "fp8", 12, 333, True, False),
    (2, 1, 256, 4, 64, "sym", 20, 150, False, False),
]


def _id(c):
    return "-".join(map(str, c[:6])) + f"-{c[6]}of{c[7]}"


def _make(form, seed, k_spread, v_spread):
    import torch
    from attention_bounds import sized_cache
    from attention_util import Cache
    H, KV, hd, bits, group, fmt, n, length, dhalf, two = form
    print(f"[case] scales {form} spread {k_spread} {v_spread}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(seed)
    P = -(-length // 16)
    cache = Cache(g, (P + 1) * 16, KV, hd, bits, group, fmt, dhalf, two, first=group)
    sized_cache(cache, g, k_spread, v_spread)
    pages = torch.randperm(P + 1, generator=g, device="cuda")[:P].to(torch.int32)
    t = torch.arange(length, device="cuda")
    rows = pages.long()[t // 16] * 16 + t % 16
    Q = torch.randn(n, H, hd, generator=g, device="cuda").bfloat16()
    return cache, Q, pages[None].contiguous(), rows


def _call(cache, Q, pages, length, **kw):
    import online_activation_aware_ttq_amd as ttq
    from test_gpu_attention import _i32
    return ttq.ttq_cache_attention(Q, pages, _i32([length]), *cache.one, page_tokens=16,
                                   offsets=_i32([0, Q.shape[0]]), **cache.kwargs(), **kw)


def _compare(cache, Q, rows, length, got, scale, window=0, vacuous=0.1):
    import torch
    from attention_bounds import by_key
    n, H, _ = Q.shape
    ref, tol = by_key(cache, Q, rows, length - n, scale, window, tile=n * (H // cache.KV) >= 64)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    worst = float((err / tol.clamp(min=1e-300)).max())
    size = ref.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    share = float((tol / size).median())
    print(f"  largest error {worst:.2f} of its bound, whose median is {share:.4f} of a row's largest", flush=True)
    assert worst <= 1 and share <= vacuous


@pytest.mark.parametrize("form", FORMS, ids=_id)
@pytest.mark.parametrize("k_spread,v_spread,scale", [
    (3.0, 3.0, 2.0 ** -12),   # sizes 1000-fold apart
    (0.0, 8.0, 0.1),          # V's, 2^-24 to 2^24
    (8.0, 0.0, 2.0 ** -26),   # K's
    (8.0, 8.0, 2.0 ** -24),
])
def test_sizes_far_apart(form, k_spread, v_spread, scale):
    cache, Q, pages, rows = _make(form, 5, k_spread, v_spread)
    got = _call(cache, Q, pages, form[7], scale=scale)
    _compare(cache, Q, rows, form[7], got, scale)


@pytest.mark.parametrize("form", FORMS, ids=_id)
@pytest.mark.parametrize("size", [2.0 ** 9, 1e5, 1e30, 1e-30])
def test_a_large_key_is_its_own(form, size):
    """The newest key's scales and offsets times `size`, one group's or all: the rows that
    do not see it keep their bits, the one that does has what it should."""
    import torch
    cache, Q, pages, rows = _make(form, 6, 0.0, 0.0)
    length, hd = form[7], form[2]
    clean = _call(cache, Q, pages, length)
    newest = rows[-1]
    for which, c, at in ((1, cache.two or cache.one, cache.v_first), (0, cache.one, cache.first)):
        keep = [t[newest].clone() for t in c[1:]]
        a = at // cache.group
        for cut in (slice(a, a + 1), slice(a, a + max(1, cache.KV * hd // cache.group))):
            for t in c[1:]:
                t[newest, cut] *= size
            got = _call(cache, Q, pages, length)
            same = torch.equal(got[:-1], clean[:-1])
            assert same, (which, cut)
            # scores far from 0 are off by 2^-11 of themselves and more: no bound for them
            if which == 1 or size < 1:
                _compare(cache, Q[-1:], rows, length, got[-1:], hd ** -0.5)
            else:
                assert torch.isfinite(got).all()
            for t, k in zip(c[1:], keep):
                t[newest] = k


@pytest.mark.parametrize("form", FORMS, ids=_id)
@pytest.mark.parametrize("k_size,v_size", [(1.0, 2.0 ** 14), (2.0 ** -14, 2.0 ** -14), (1.0, 0.0), (0.0, 2.0 ** 60)])
def test_a_first_key_of_another_size(form, k_size, v_size):
    """The oldest key, from which the units of a prompt's first block are, and which all
    rows of a prompt see."""
    cache, Q, pages, rows = _make(form, 7, 0.0, 0.0)
    width = cache.KV * cache.hd
    for c, at, size in ((cache.one, cache.first, k_size), (cache.two or cache.one, cache.v_first, v_size)):
        for t in c[1:]:
            t[rows[0], at // cache.group:-(-(at + width) // cache.group)] *= size
    length = form[6]  # a prompt: no keys before it
    got = _call(cache, Q, pages, length)
    _compare(cache, Q, rows[:length], length, got, form[2] ** -0.5)


@pytest.mark.parametrize("form", FORMS, ids=_id)
def test_sizes_far_apart_in_a_window(form):
    cache, Q, pages, rows = _make(form, 8, 2.0, 8.0)
    got = _call(cache, Q, pages, form[7], scale=2.0 ** -8, window=40)
    _compare(cache, Q, rows, form[7], got, 2.0 ** -8, window=40)


@pytest.mark.parametrize("size", [1e-36, 1.0, 1e33, 3e37])
@pytest.mark.parametrize("length,n,H", [(20000, 1, 2), (20000, 70, 1), (900, 9, 2)])
def test_values_as_large_as_float32_goes(length, n, H, size):
    """Ranges of many keys joined: the mean of V is as large as V is."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    g = torch.Generator(device="cuda").manual_seed(2)
    cache = Cache(g, -(-length // 16) * 16, 1, 64, 8, 64, "asym")
    x = torch.randn(cache.one[0].shape[0], cache.d, generator=g, device="cuda")
    x[:, 64:] = x[:, 64:].clamp(-3, 3) * size
    ttq.ttq_cache_write(x, torch.arange(x.shape[0], device="cuda"), *cache.one, **cache.how)
    Q = torch.randn(n, H, 64, generator=g, device="cuda").bfloat16()
    pages = torch.arange(x.shape[0] // 16, dtype=torch.int32, device="cuda")[None]
    got = _call(cache, Q, pages, length)
    # (the mean of 20000 values of both signs is 141 times smaller than they are, to which
    # the bound, 0.0015 of them, goes: 0.21 of it)
    _compare(cache, Q, torch.arange(length, device="cuda"), length, got, 0.125, vacuous=0.3)


@pytest.mark.parametrize("rows", [9, 200])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 14, 2.0 ** -40])
def test_without_the_key_that_units_are_from(rows, size):
    """The newest pages are in no cache, so that no unit comes from them: any size is right."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache, reference
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(rows)
    cache = Cache(g, 512, 2, 64, 4, 64, "asym")
    for t in cache.one[1:]:
        t[:, cache.v_first // 64:] *= size
    length = 400
    pages = torch.randperm(32, generator=g, device="cuda")[:25].to(torch.int32)
    for p in range(25):  # every page that a block's first row is in
        if p % 2 or p > 20:
            pages[p] = -1
    Q = torch.randn(rows, 8, 64, generator=g, device="cuda").bfloat16()
    out = ttq.ttq_cache_attention(Q, pages[None], _i32([length]), *cache.one, page_tokens=16,
                                  offsets=_i32([0, rows]), **cache.kwargs())
    t = torch.arange(length, device="cuda")
    at = torch.where(pages[t // 16] >= 0, pages[t // 16].long() * 16 + t % 16, -1)
    ref, tol = reference(cache, Q, at, length, length - rows, 0.125, tile=rows * 4 >= 64)
    assert ((out.double().cpu() - ref).abs() <= tol).all()


def test_keys_of_another_size_in_a_long_context():
    """More tiles than there are marks for them, of a workgroup that has them all."""
    import torch
    from attention_bounds import by_key
    from attention_util import Cache
    g = torch.Generator(device="cuda").manual_seed(4)
    length, n = 140000, 33000
    cache = Cache(g, length + 16 - length % 16, 1, 64, 4, 64, "asym")
    far = torch.tensor([130, 131, 128 * 1024 + 5, 128 * 1025 + 2, 128 * 40, length - n], device="cuda")
    for t in cache.one[1:]:
        t[far] *= 2.0 ** 11
        t[far[:3], 0] *= 2.0 ** -22  # K of some small, their V large
    Q = torch.randn(n, 1, 64, generator=g, device="cuda").bfloat16()
    pages = torch.arange(cache.one[0].shape[0] // 16, dtype=torch.int32, device="cuda")[None]
    got = _call(cache, Q, pages, length, scale=2.0 ** -12)
    rows = torch.arange(length, device="cuda")
    for a, b in ((0, 2), (15000, 15002), (n - 2, n)):
        end = length - n + b
        ref, tol = by_key(cache, Q[a:b], rows[:end], end - (b - a), 2.0 ** -12, tile=True)
        err = (got[a:b].double() - ref).abs()
        worst = float((err / tol).max())
        print(f"  rows {a}..: largest error {worst:.2f} of its bound", flush=True)
        assert worst <= 1 and float((tol / ref.abs().amax(-1, keepdim=True)).median()) <= 0.3


@pytest.mark.parametrize("form", FORMS, ids=_id)
def test_sizes_2_to_100_apart(form):
    """All keys 2^-60, one of the oldest and one of the newest 2^40 of what they were."""
    cache, Q, pages, rows = _make(form, 9, 0.0, 0.0)
    width = cache.KV * cache.hd
    a = cache.v_first // cache.group
    cut = slice(a, a + max(1, width // cache.group))
    for t in (cache.two or cache.one)[1:]:
        t[:, cut] *= 2.0 ** -60
        t[rows[1], cut] *= 2.0 ** 100
        t[rows[-1], cut] *= 2.0 ** 100
    got = _call(cache, Q, pages, form[7])
    _compare(cache, Q, rows, form[7], got, form[2] ** -0.5)
