"""Windows of any size: one that is as long as the context, or far longer, is none."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,news,H,KV,hd", [
    ([2000], [2000], 4, 1, 64),           # tiles of a prompt
    ([1500, 40], [300, 40], 8, 2, 128),
    ([20, 300], [200, 300], 2, 1, 64),    # more rows than keys
    ([700, 33], [1, 1], 4, 2, 128),       # ranges of keys
    ([500, 33], [9, 3], 4, 2, 64),
])
def test_windows_past_the_context_are_none(lens, news, H, KV, hd):
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(sum(lens))
    P = -(-max(lens) // 16)
    cache = Cache(g, len(lens) * P * 16, KV, hd, 4, 64, "asym")
    pages = torch.randperm(len(lens) * P, generator=g, device="cuda").view(-1, P).to(torch.int32)
    off = [0]
    for n in news:
        off.append(off[-1] + n)
    Q = torch.randn(off[-1], H, hd, generator=g, device="cuda").bfloat16()

    def call(window):
        return ttq.ttq_cache_attention(Q, pages, _i32(lens), *cache.one, page_tokens=16,
                                       offsets=_i32(off), window=window, **cache.kwargs())

    want = call(0)
    for window in (max(lens), 2 ** 20, 2 ** 31 - 2100, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, 2 ** 32, 2 ** 34 + 5,
                   2 ** 63 - 1):
        same = torch.equal(call(window), want)
        assert same, window


@pytest.mark.parametrize("window", [1, 63, 64, 65, 1999])
def test_windows_of_a_prompt(window):
    from test_gpu_attention import _run
    _run((4, 1, 64, 4, 64, "asym", 16, [2000], [600], window, False, False))
