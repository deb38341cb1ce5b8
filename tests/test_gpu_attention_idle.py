"""Attention of prompts beside requests that add nothing in the step but hold many keys
(ttq_cache_extend gives them no rows): first, in the middle and last of the batch."""
import pytest

pytestmark = pytest.mark.gpu

CASES = [
    # H, KV, hd, bits, group, fmt, page, lens, rows, window, D, two caches
    (4, 1, 64, 4, 64, "asym", 16, [200, 4096], [200, 0], 0, False, False),
    (4, 1, 64, 4, 64, "asym", 16, [4096, 200], [0, 200], 0, False, False),
    (4, 1, 128, 8, 64, "fp8", 32, [200, 4096, 700], [200, 0, 300], 0, True, False),
    (2, 1, 64, 4, 32, "sym", 16, [3000, 900, 300, 2000, 257], [0, 600, 0, 100, 0], 100, False, True),
    (1, 1, 64, 4, 64, "asym", 16, [900] + [300] * 5, [900] + [0] * 5, 0, False, False),
    # and where all are idle but one row of one request
    (64, 1, 64, 4, 64, "asym", 16, [700, 1000], [0, 2], 0, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])) + f"-{c[7]}of{c[8]}")
def test_against_float64(case):
    from test_gpu_attention import _run
    _run(case)


def test_a_block_is_done_once():
    """One request with a row, and thousands before or behind it that have none, take no
    longer than beside as many rows of empty requests: no workgroup does another's block."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(0)
    n, idle = 32768, 2100
    cache = Cache(g, n, 4, 64, 4, 64, "asym")
    pages = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None].repeat(idle + 1, 1)
    Q = torch.randn(1, 16, 64, generator=g, device="cuda").bfloat16()

    def timed(Q, lens, off):
        lens, times = _i32(lens), []
        off = None if off is None else _i32(off)
        for _ in range(6):
            ttq.timing_reset()
            ttq.timing_enable(True)
            out = ttq.ttq_cache_attention(Q, pages, lens, *cache.one, page_tokens=64, offsets=off, **cache.kwargs())
            torch.cuda.synchronize()
            ttq.timing_enable(False)
            times.append(ttq.timing_query()["attention_split"][0])
        return out, min(times)

    alone, t0 = timed(Q.repeat(idle + 1, 1, 1), [n] + [0] * idle, None)
    for at in (0, idle):
        lens = [64] * (idle + 1)
        lens[at] = n
        out, t = timed(Q, lens, [0] * (at + 1) + [1] * (idle + 1 - at))
        print(f"  {t:.3f} ms, {t0:.3f} beside empty rows", flush=True)
        same = torch.equal(out, alone[:1])
        assert same and t <= 2 * t0
