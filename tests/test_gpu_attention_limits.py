"""Calls with so many rows that one dimension of a launch does not hold their threads."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_seq,news,KV,hd", [(50000, 56, 6, 64)])
def test_more_rows_than_a_launch_has_along_x(n_seq, news, KV, hd):
    """2.8 million rows of 6 heads, joined by a workgroup each: 2^32 threads and more.  All
    sequences are alike, so are their results."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache, reference
    from test_gpu_attention import _i32
    T = n_seq * news
    assert T * KV > 2 ** 24
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = Cache(g, 64, KV, hd, 4, 64, "asym")
    one = torch.randn(news, KV, hd, generator=g, device="cuda").bfloat16()
    Q = one.repeat(n_seq, 1, 1)
    pages = _i32([[2, 0, 3, 1]]).repeat(n_seq, 1)
    off = torch.arange(n_seq + 1, dtype=torch.int32, device="cuda") * news
    lens = torch.full((n_seq,), news, dtype=torch.int32, device="cuda")
    out = torch.full((T, KV, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    ttq.ttq_cache_attention(Q, pages, lens, *cache.one, page_tokens=16, offsets=off, out=out, **cache.kwargs())
    torch.cuda.synchronize()
    rows = torch.tensor([2, 0, 3, 1], device="cuda").repeat_interleave(16) * 16 + torch.arange(16, device="cuda").repeat(4)
    ref, tol = reference(cache, one, rows, news, 0, hd ** -0.5)
    assert ((out[:news].double().cpu() - ref).abs() <= tol).all()
    for at in range(0, n_seq, 10000):
        same = bool((out.view(n_seq, news, KV, hd)[at:at + 10000] == out[:news]).all())
        assert same, at
    torch.cuda.empty_cache()


@pytest.mark.parametrize("case", [
    # one row a sequence of so many heads of a K/V head that tiles are decoded for them
    (64, 1, 64, 4, 64, "asym", 16, [500, 31, 0], [1, 1, 1], 0, False, False),
    (150, 1, 128, 8, 64, "fp8", 32, [900], [1], 100, True, False),
    (300, 1, 64, 4, 32, "sym", 16, [70, 257], [1, 1], 0, False, True),
], ids=lambda c: "-".join(map(str, c[:6])))
def test_many_heads_of_a_row(case):
    from test_gpu_attention import _run
    _run(case)
