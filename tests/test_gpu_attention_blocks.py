"""Attention over a quantized cache where its rows and keys are divided in other ways:
many sequences, blocks of several, heads that are no multiple of a workgroup's, page
tables longer than a workgroup holds, and rows of the cache that are no keys."""
import random

import pytest

pytestmark = pytest.mark.gpu


def _lens(n, lo, hi, seed):
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(n)]


def _mixed(n, seed):
    """Lengths and new tokens: whole prompts, chunks of long ones, empty sequences."""
    rng = random.Random(seed)
    lens = [rng.choice((0, rng.randint(1, 90), rng.randint(200, 700))) for _ in range(n)]
    return lens, [rng.randint(0, n) if rng.random() < 0.5 else n for n in lens]


MANY = _lens(70, 30, 60, 1)
FEW, FEW_NEW = _mixed(64, 2)
ONES = _lens(1100, 1, 40, 3)
CASES = [
    # blocks of 256 rows: more sequences than lanes, as many, and a few of which one is long
    (8, 2, 64, 4, 64, "asym", 16, MANY, MANY, 0, False, False),
    (4, 2, 64, 4, 32, "sym", 16, FEW, FEW_NEW, 0, True, False),
    (4, 1, 128, 4, 128, "asym", 16, [700, 64, 1500, 0, 300, 33], [700, 40, 200, 0, 300, 1], 0, False, False),
    (4, 1, 128, 8, 64, "fp8", 32, [900, 300, 1200], [300, 300, 100], 200, True, True),
    (2, 1, 256, 4, 64, "intzp", 32, [200, 90], [100, 90], 0, False, False),
    (2, 1, 256, 8, 256, "asym", 8, [333], [333], 50, True, False),
    # a few rows of few keys on many workgroups: ranges of a tile
    (2, 1, 64, 8, 32, "asym", 16, [2600], [70], 0, False, False),
    # blocks of 16 rows: one a workgroup (more than 2048 of them), and divided evenly
    (16, 8, 64, 4, 64, "asym", 16, ONES, [1] * 1100, 0, False, False),
    (6, 3, 64, 4, 32, "sym", 16, [500, 3, 1200, 0, 77], [2, 3, 1, 0, 5], 0, True, False),
    (10, 5, 128, 8, 128, "asym", 64, [900, 64, 65], [1, 1, 1], 0, False, False),
    (24, 6, 128, 4, 128, "asym", 16, [1500, 10, 700], [3, 1, 2], 0, False, True),
    (40, 1, 64, 4, 64, "intzp", 16, [600, 31], [1, 1], 0, False, False),
    (2, 1, 256, 8, 32, "fp8", 16, [700, 100], [1, 1], 300, True, False),
    # page tables of more entries than a workgroup holds at a time
    (2, 1, 64, 8, 32, "fp8", 1, [3000, 1023, 1025], [1, 1, 1], 0, False, False),
    (8, 4, 128, 4, 128, "asym", 1, [2100], [1], 1500, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])) + f"-{len(c[7])}x{max(c[7])}")
def test_against_float64(case):
    from test_gpu_attention import _run
    _run(case)


@pytest.mark.parametrize("rows", [1, 9, 40])
def test_bytes_of_rows_that_are_no_keys(rows):
    """Every byte of the rows that belong to no key is E4M3's NaN, row 0 among them."""
    import torch
    from test_gpu_attention import _call, _i32, _small
    cache, _ = _small(n_slots=128, bits=8, fmt="fp8")
    g = torch.Generator(device="cuda").manual_seed(9)
    Q = torch.randn(rows, 4, 64, generator=g, device="cuda").bfloat16()
    pages, off, n = _i32([[5, 7, 3, -1]]), _i32([0, rows]), 44
    want = _call(cache, Q, pages, [n], offsets=off, window=0)
    assert torch.isfinite(want.float()).all()
    at = [p * 16 + i for p in (5, 7, 3) for i in range(16)][:n]
    free = torch.ones(128, dtype=torch.bool, device="cuda")
    free[at] = False
    for t in cache.one:
        t.view(torch.uint8)[free] = 255
    assert torch.equal(_call(cache, Q, pages, [n], offsets=off, window=0), want)


@pytest.mark.parametrize("fmt,bits", [("asym", 4), ("fp8", 8), ("sym", 8)])
@pytest.mark.parametrize("rows", [1, 9, 40])
def test_infinite_scales_stay_with_their_key(fmt, bits, rows):
    """The newest key's, which only the last row sees: NaN in what it enters, no more."""
    import torch
    from test_gpu_attention import _call, _i32, _small
    cache, _ = _small(n_slots=128, bits=bits, fmt=fmt)
    g = torch.Generator(device="cuda").manual_seed(9)
    Q = torch.randn(rows, 4, 64, generator=g, device="cuda").bfloat16()
    pages, off, n = _i32([[5, 0, 3, 6]]), _i32([0, rows]), 50
    clean = _call(cache, Q, pages, [n], offsets=off)
    s, at, gv = cache.one[1], 6 * 16 + 1, cache.v_first // 32 + 2
    keep = s[at].clone()
    s[at, gv] = float("inf")
    got = _call(cache, Q, pages, [n], offsets=off)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[-1, 2:, :32] = True  # the first group of head 1
    assert torch.equal(torch.isnan(got.float()), bad) and torch.equal(got[~bad], clean[~bad])
    s[at] = keep
    s[at, 0] = float("inf")  # K, head 0
    got = _call(cache, Q, pages, [n], offsets=off)
    bad[:] = False
    bad[-1, :2] = True
    assert torch.equal(torch.isnan(got.float()), bad) and torch.equal(got[~bad], clean[~bad])


def test_blocks_in_any_order_give_the_same_rows():
    """The rows of a sequence are the same alone and among others (few keys: one range)."""
    import torch
    from test_gpu_attention import _call, _i32, _small
    cache, _ = _small(n_slots=1024, bits=4, fmt="asym")
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = [200, 64, 130, 128, 255, 190]
    Q = torch.randn(sum(lens), 4, 64, generator=g, device="cuda").bfloat16()
    pages = torch.randperm(64, generator=g, device="cuda")[:16].to(torch.int32)[None].repeat(6, 1).contiguous()
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    every = _call(cache, Q, pages, lens, offsets=_i32(off))
    for i, n in enumerate(lens):
        one = _call(cache, Q[off[i]:off[i + 1]].contiguous(), pages[i:i + 1].contiguous(), [n], offsets=_i32([0, n]))
        assert torch.equal(one, every[off[i]:off[i + 1]])


@pytest.mark.parametrize("KV,hd,bits,group", [(8, 128, 4, 128), (8, 128, 4, 64), (4, 64, 8, 32), (2, 256, 8, 64)])
def test_scales_at_any_alignment(KV, hd, bits, group):
    """Scales read 16 bytes and 4 bytes at a time give the same bits, and the right ones."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache, reference
    from test_gpu_attention import _i32
    g = torch.Generator(device="cuda").manual_seed(hd + group)
    cache = Cache(g, 2048, KV, hd, bits, group, "asym")
    pages = torch.randperm(128, generator=g, device="cuda").view(2, 64).to(torch.int32)
    lens = [1000, 333]
    Q = torch.randn(2, 2 * KV, hd, generator=g, device="cuda").bfloat16()

    def call(c):
        return ttq.ttq_cache_attention(Q, pages, _i32(lens), *c, page_tokens=16, **cache.kwargs())

    want = call(cache.one)
    apart = [cache.one[0]]
    for t in cache.one[1:]:
        room = torch.empty(t.numel() + 1, device="cuda")
        room[1:] = t.flatten()
        apart.append(room[1:].view(t.shape))
        assert apart[-1].data_ptr() % 16 == 4
    assert torch.equal(call(apart), want)
    for i, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        ref, tol = reference(cache, Q[i:i + 1], pages[i].long()[t // 16] * 16 + t % 16, n, n - 1, hd ** -0.5)
        assert ((want[i:i + 1].double().cpu() - ref).abs() <= tol).all()


def test_captured_prompts():
    """Two graphs of prompts whose keys are divided, replayed at once: the eager call's bits."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    from test_gpu_attention import _i32, _small
    cache, _ = _small(n_slots=4096, KV=2, hd=128, group=128)
    g = torch.Generator(device="cuda").manual_seed(2)
    state = []
    for k in range(2):
        Q = torch.randn(260, 4, 128, generator=g, device="cuda").bfloat16()
        pages = torch.randperm(256, generator=g, device="cuda").view(2, 128).to(torch.int32).contiguous()
        state.append((Q, pages, _i32([2000, 700]), _i32([0, 130, 260]), torch.zeros_like(Q)))

    def call(k, **kw):
        Q, pages, lens, off, out = state[k]
        return ttq.ttq_cache_attention(Q, pages, lens, *cache.one, page_tokens=16, offsets=off,
                                       **cache.kwargs(), **kw)

    call(0)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(k, out=state[k][4])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for step in range(4):
        for Q, pages, lens, off, out in state:
            Q.normal_()
            lens.copy_(_i32([130 + 400 * step, 0 if step == 2 else 2048 - step]))
            off.copy_(_i32([0, 100 + 10 * step, 250]))
            out.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        got = [st[4].clone() for st in state]
        for k in range(2):
            a = call(k, out=torch.zeros_like(got[k]), stream=streams[k].cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(got[k], a) and (got[k][250:] == 0).all()
