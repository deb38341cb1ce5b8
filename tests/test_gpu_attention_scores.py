"""Scores of any finite size: one far above the others takes its row, equal ones share it."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 9, 200])
@pytest.mark.parametrize("fmt,bits", [("asym", 4), ("fp8", 8)])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(rows, fmt, bits, sign):
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(rows)
    length, H, KV, hd = 300, 4, 1, 64
    cache = Cache(g, 320, KV, hd, bits, 64, fmt)
    pages = torch.randperm(20, generator=g, device="cuda").to(torch.int32)[None]
    t = torch.arange(length, device="cuda")
    at = pages[0].long()[t // 16] * 16 + t % 16
    k, v = (sum(cache.parts(at, w))[:, 0] for w in (0, 1))
    Q = torch.randn(rows, H, hd, generator=g, device="cuda").bfloat16()
    pos = length - rows + torch.arange(rows, device="cuda")
    for big in (1.0, 2.0 ** 18, 2.0 ** 22, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100, 2.0 ** 118):
        q = Q * big
        out = ttq.ttq_cache_attention(q, pages, _i32([length]), *cache.one, page_tokens=16,
                                      offsets=_i32([0, rows]), scale=0.125 * sign, **cache.kwargs())
        assert torch.isfinite(out).all(), big
        if big == 1:
            continue
        x = torch.where((t <= pos[:, None])[:, None], 0.125 * sign * Q.double() @ k.T, -torch.inf)
        two = x.topk(2, -1)
        # the largest score's value, where the next is 2^-8 of the largest |score| or more
        # below it: K in 11 bits moves a score by 3 x 2^-11 of sum |q k| at most
        room = 6 * 2.0 ** -11 * 0.125 * Q.double().abs() @ k.abs().T
        clear = two.values[..., 0] - two.values[..., 1] > room.amax(-1)
        assert clear.float().mean() > 0.3
        err = (out.double() - v[two.indices[..., 0]]).abs()[clear]
        assert (err <= 2.0 ** -7 * v.abs().amax(0)).all(), big


@pytest.mark.parametrize("rows", [1, 200])
def test_equal_scores_of_any_size(rows):
    """All keys alike: the mean of V, whatever the score."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = Cache(g, 320, 1, 64, 8, 64, "asym")
    x = torch.randn(320, cache.d, generator=g, device="cuda")
    x[:, :64] = 1.5
    ttq.ttq_cache_write(x, torch.arange(320, device="cuda"), *cache.one, **cache.how)
    pages = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    v = sum(cache.parts(torch.arange(300, device="cuda"), 1))[:, 0]
    pos = 300 - rows + torch.arange(rows, device="cuda")
    want = torch.stack([v[:p + 1].mean(0) for p in pos.tolist()])[:, None]
    for big in (1.0, 2.0 ** 20, 2.0 ** 27, -2.0 ** 31, 2.0 ** 90):
        Q = torch.full((rows, 4, 64), big, dtype=torch.bfloat16, device="cuda")
        out = ttq.ttq_cache_attention(Q, pages, _i32([300]), *cache.one, page_tokens=16,
                                      offsets=_i32([0, rows]), **cache.kwargs())
        # V in 11 bits three times and 2^-16 of the largest, the result in 8
        tol = 2.0 ** -8 * want.abs() + (3 * 2.0 ** -11 + 2.0 ** -16) * v.abs().amax()
        assert ((out.double() - want).abs() <= tol).all(), big


@pytest.mark.parametrize("rows", [1, 9, 200])
@pytest.mark.parametrize("fmt,bits", [("asym", 4), ("fp8", 8), ("sym", 8)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinite_queries_are_nan(rows, fmt, bits, value):
    """Also where every score would be -inf; a row without keys is 0 all the same."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = Cache(g, 320, 2, 64, bits, 64, fmt)
    x = torch.randn(320, cache.d, generator=g, device="cuda")
    x[:, :128] = -1 - x[:, :128].abs()
    ttq.ttq_cache_write(x, torch.arange(320, device="cuda"), *cache.one, **cache.how)
    pages = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    Q = torch.randn(rows, 8, 64, generator=g, device="cuda").bfloat16()
    call = lambda length: ttq.ttq_cache_attention(Q, pages, _i32([length]), *cache.one, page_tokens=16,
                                                  offsets=_i32([0, rows]), **cache.kwargs())
    Q[0, 5, 9] = 2.0 ** 127  # the largest finite ones are none
    clean = call(300)
    assert torch.isfinite(clean).all()
    at = rows // 2
    keep = Q[at, 3, 17].clone()
    Q[at, 3, 17] = value
    got = call(300)
    bad = torch.zeros(rows, 8, dtype=torch.bool, device="cuda")
    bad[at, 3] = True
    nan = torch.isnan(got.float())
    assert nan[bad].all() and not nan[~bad].any()
    same = torch.equal(got[~bad], clean[~bad])
    assert same
    if rows > 1:  # fewer keys than rows: the first rows see none
        Q[at, 3, 17] = keep
        Q[0, 3, 17] = value
        got = call(rows - 1)
        assert (got[0] == 0).all() and not torch.isnan(got.float()).any()


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("group", [32, 64])
def test_many_small_weights_add_up(rows, group):
    """One key far above thousands of equal ones, which together make the result: their p
    is 2^-25.6 of its."""
    import math
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(1)
    n, D = 16000, 25.6
    cache = Cache(g, n, 1, 64, 8, group, "asym")
    x = torch.zeros(n, cache.d, device="cuda")
    x[:, 64:128] = 1.0       # V of all keys but one, which is 0 and has the large score
    x[70, :64], x[70, 64:128] = 1.0, 0.0
    ttq.ttq_cache_write(x, torch.arange(n, device="cuda"), *cache.one, **cache.how)
    Q = torch.ones(rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = ttq.ttq_cache_attention(Q, torch.arange(n // 16, dtype=torch.int32, device="cuda")[None], _i32([n]),
                                  *cache.one, page_tokens=16, offsets=_i32([0, rows]),
                                  scale=D * math.log(2) / 64, **cache.kwargs())
    w = (n - rows + torch.arange(rows, device="cuda").double()) * 2.0 ** -D
    want = (w / (1 + w))[:, None, None]
    # p: 2^-25 of 2^7 times the largest, all the same way; the score's float32 roundings
    # (70 of 2^-24 D, as powers of two); the result's 8 bits
    tol = 2.0 ** (D - 32) + 70 * 2.0 ** -24 * D + 2.0 ** -8
    assert ((out.double() - want).abs() <= tol * want).all(), float((out.double() / want - 1).abs().max())


@pytest.mark.parametrize("rows", [9, 200])
@pytest.mark.parametrize("fmt,bits", [("asym", 4), ("fp8", 8)])
def test_large_scores_of_one_row_are_its_own(rows, fmt, bits):
    """Queries of one head of one row 2^30 times larger: the others keep their bits."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(rows)
    cache = Cache(g, 3008, 2, 128, bits, 128, fmt)
    pages = torch.randperm(188, generator=g, device="cuda").to(torch.int32)[None]
    Q = torch.randn(rows, 8, 128, generator=g, device="cuda").bfloat16()
    call = lambda: ttq.ttq_cache_attention(Q, pages, _i32([3000]), *cache.one, page_tokens=16,
                                           offsets=_i32([0, rows]), **cache.kwargs())
    clean = call()
    other = torch.ones(rows, 8, dtype=torch.bool, device="cuda")
    for at in range(0, rows, 5):
        Q[at, at % 8] *= 2.0 ** 30
        other[at, at % 8] = False
    got = call()
    same = torch.equal(got[other], clean[other])
    assert same and torch.isfinite(got).all()
