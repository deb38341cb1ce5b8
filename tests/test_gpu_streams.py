"""Calls of several threads and on streams given as argument, on the GPU: every
result has the bits of the same call alone."""
import threading

import numpy as np
import pytest

from test_gpu_moe import _dev, _stored

pytestmark = pytest.mark.gpu


def _layer(seed, T=20, E=8, k=2, d=256, ff=256):
    """A call of ttq_moe, of ttq_adapters with a workspace and of ttq_qmatmul, on
    inputs of their own."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    rng = np.random.default_rng(seed)

    def bf16(*shape, sigma=1.0):
        return torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).cuda().bfloat16()

    gu, dn = (_dev(_stored(rng, E, r, c, 4, 128, "asym")) for r, c in ((2 * ff, d), (d, ff)))
    Wr, X = bf16(E, d, sigma=0.1), bf16(T, d)
    A, B = bf16(3, 32, 2048, sigma=0.05), bf16(3, 96, 32, sigma=0.05)
    X2, idx = bf16(150, 2048), torch.from_numpy(rng.integers(-1, 3, 150).astype(np.int32)).cuda()
    q = ttq.ttq_quantize(bf16(192, 256, sigma=0.05), bf16(16, 256), p=2.0, lam=1e-3, alpha=0.5, bits=4,
                         group=64)

    def run(**kw):
        return (ttq.ttq_moe(X, Wr, *gu, *dn, top_k=k, bits=4, group=128, **kw),
                ttq.ttq_adapters(X2, A, B, idx, **kw),
                ttq.ttq_qmatmul(*q, X, bits=4, group=64, **kw))

    return run


def _same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_threads_on_one_stream():
    import torch
    runs = [_layer(s) for s in (1, 2, 3)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(runs))

    def work(i):
        start.wait()
        for step in range(60):
            got = runs[i]()
            torch.cuda.current_stream().synchronize()
            if not _same(got, want[i]):
                wrong.append((i, step))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_captured_on_a_stream_given_as_argument():
    """Two graphs whose calls go to a side stream by argument, replayed at once,
    while larger eager calls of the same stream make its kept buffer grow."""
    import torch
    runs = [_layer(s) for s in (4, 5)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for r in runs:
        r(stream=side.cuda_stream)
    side.synchronize()
    graphs, got = [], []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            got.append(r(stream=side.cuda_stream))
            torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    big = _layer(6, T=128, ff=768)
    bigger = big()
    on = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        torch.cuda.synchronize()
        for ys in got:
            for y in ys:
                y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, on):
            with torch.cuda.stream(s):
                g.replay()
        eager = big(stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert _same(eager, bigger)
        for a, b in zip(got, want):
            assert _same(a, b)


def test_results_of_a_stream_given_as_argument():
    """While torch's current stream is busy: what the call makes, zeros behind the
    lengths among it, is in the order of the call's stream."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    d, n = 1024, 64
    codes = torch.zeros(n, d // 2, dtype=torch.uint8, device="cuda")
    s, m = torch.zeros(n, d // 128, device="cuda"), torch.zeros(n, d // 128, device="cuda")
    X = torch.randn(n, d, device="cuda")
    kw = dict(bits=4, group=128)
    ttq.ttq_cache_write(X, torch.arange(n, device="cuda"), codes, s, m, **kw)
    pages = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([50], dtype=torch.int32, device="cuda")
    read = lambda **k: ttq.ttq_cache_read(codes, s, m, pages, lens, page_tokens=16, **kw, **k)
    run = _layer(7)
    want, layer = read(), run()
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(8):
            a = a @ a * 1e-2                  # some milliseconds of the current stream
        got, rows = read(stream=side.cuda_stream), run(stream=side.cuda_stream)
        side.synchronize()
        with torch.cuda.stream(side):
            got, rows = got.clone(), [r.clone() for r in rows]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and _same(rows, layer)
        assert (got[0, 50:] == 0).all() and (got[0, :50] != 0).any(1).all()


def test_the_default_stream_given_as_argument():
    """From within another stream: handle 0, and a handle of torch's own streams."""
    import torch
    run = _layer(8)
    want = run()
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        for handle in (0, other.cuda_stream, side.cuda_stream):
            got = run(stream=handle)
            torch.cuda.synchronize()
            assert _same(got, want), handle
