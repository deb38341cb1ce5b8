"""The attention of a decoder layer served from stored codes, as its calls are used
together: the step's pages and slots, the projection of Q, K and V from codes, norms
and rotation with K and V quantized into their rows, attention over the cache and the
output projection; a ragged prompt step, then decode steps that a graph replays."""
import numpy as np
import pytest

import oracle
from parity_util import Y_MAX_REL, Y_MEAN_REL, y_errors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,bits,group,two", [("asym", 4, 64, False), ("fp8", 8, 128, True)])
def test_prompt_and_decode_steps(fmt, bits, group, two):
    import torch
    import online_activation_aware_ttq_amd as ttq
    from attention_util import Cache, reference
    g = torch.Generator(device="cuda").manual_seed(bits)
    S, dim, H, KV, hd, page, P, n_pages = 4, 512, 8, 2, 128, 16, 6, 20
    qw, kw = H * hd, KV * hd

    def weights(rows, cols):
        W = (torch.randn(rows, cols, generator=g, device="cuda") * 0.05).bfloat16()
        X = torch.randn(32, cols, generator=g, device="cuda").bfloat16()
        return ttq.ttq_quantize(W, X, p=2.0, lam=1e-3, alpha=0.5, bits=4, group=128)

    qkv, out_w = weights(qw + 2 * kw, dim), weights(dim, qw)
    wq, wk = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda") for _ in range(2))
    inv_freq = torch.from_numpy((10000.0 ** (-np.arange(0, hd, 2) / hd)).astype(np.float32)).cuda()
    cache = Cache(g, n_pages * page, KV, hd, bits, group, fmt, two=two)
    for c in (cache.one, cache.two):
        if c is not None:
            [t.zero_() for t in c]
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = torch.full((S, P), -1, **i32)
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    count, lens, added = (torch.tensor(v, **i32) for v in ([n_pages], [0] * S, [33, 1, 0, 17]))

    def step(x, T):
        """One pass; the rows and what the calls made of them."""
        off, pos = torch.empty(S + 1, **i32), torch.empty(T, **i32)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        ttq.ttq_cache_extend(lens, added, pages, free, count, page_tokens=page, lens_out=lens,
                             free_count_out=count, offsets=off, positions=pos, slots=slots)
        y = ttq.ttq_qmatmul(*qkv, x, bits=4, group=128)
        q = ttq.ttq_cache_rope(y[:, :qw], y[:, qw:qw + kw], y[:, qw + kw:], pos, slots, *cache.one,
                               head_dim=hd, inv_freq=inv_freq, q_weight=wq, k_weight=wk,
                               v_cache=cache.two, **cache.how)
        a = ttq.ttq_cache_attention(q, pages, lens, *cache.one, offsets=off, page_tokens=page,
                                    **cache.kwargs())
        o = ttq.ttq_qmatmul(*out_w, a.view(T, qw), bits=4, group=128)
        return dict(off=off, pos=pos, slots=slots, y=y, q=q, a=a, o=o)

    def check(r, T):
        """Every call against its definition on what the one before it gave."""
        y = r["y"].cpu().numpy()
        pos, slots = r["pos"].cpu().numpy(), r["slots"].cpu().numpy()
        fr, f64 = inv_freq.cpu().numpy(), lambda t: t.double().cpu().numpy()
        q = oracle.rope_heads(y[:, :qw].reshape(T, H, hd), wq.cpu().numpy(), 1e-6, fr, pos)
        k = oracle.rope_heads(y[:, qw:qw + kw].reshape(T, KV, hd), wk.cpu().numpy(), 1e-6, fr, pos)
        assert torch.equal(r["q"].cpu(), torch.from_numpy(q).bfloat16())
        live = slots >= 0
        for which, rows in ((0, k.reshape(T, kw)), (1, y[:, qw + kw:])):
            want = oracle.cache_rows(rows, np.ones(kw, np.float32), bits, group, fmt)["values"]
            parts = cache.parts(torch.from_numpy(slots[live]).cuda(), which)
            got = (parts[0] + parts[1]).cpu().numpy().reshape(-1, kw)
            np.testing.assert_array_equal(got, want[live])
        off, L, table = r["off"].tolist(), lens.tolist(), pages.long()
        for i in range(S):
            t = torch.arange(max(L[i], 0), device="cuda")
            rows = table[i][t // page] * page + t % page
            a, b = off[i], off[i + 1]
            ref, tol = reference(cache, r["q"][a:b], rows, max(L[i], 0), max(L[i], 0) - (b - a), hd ** -0.5)
            assert ((r["a"][a:b].double().cpu() - ref).abs() <= tol).all(), i
        assert (r["a"][off[-1]:] == 0).all()
        lv = oracle.unpack_codes(out_w[0].cpu().numpy(), 4, qw).astype(np.float64).reshape(dim, -1, 128)
        W = (f64(out_w[2])[:, :, None] + f64(out_w[1])[:, :, None] * lv).reshape(dim, qw) * f64(out_w[3])
        e, _ = y_errors(r["o"][:off[-1]].cpu().numpy(), f64(r["a"][:off[-1]].view(-1, qw)) @ W.T)
        assert e.max() <= Y_MAX_REL and e.mean() <= Y_MEAN_REL

    T = 64
    x = torch.randn(T, dim, generator=g, device="cuda").bfloat16()
    r = step(x, T)
    torch.cuda.synchronize()
    assert lens.tolist() == [33, 1, 0, 17] and r["off"].tolist() == [0, 33, 34, 34, 51]
    check(r, T)

    # decode: sequence 1 ends at step 2, sequence 2 begins there with a short prompt
    T = 8
    x = torch.zeros(T, dim, dtype=torch.bfloat16, device="cuda")
    keep = [t.clone() for t in (lens, pages, free, count)]
    added.copy_(torch.tensor([1, 1, 0, 1], **i32))
    step(x, T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(x, T)
    for t, v in zip((lens, pages, free, count), keep):
        t.copy_(v)
    want = [33, 1, 0, 17]
    for n, add in enumerate(([1, 1, 0, 1], [1, 1, 0, 1], [1, -1, 4, 1], [1, 0, 1, 1], [2, 0, 1, 1])):
        added.copy_(torch.tensor(add, **i32))
        x.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = [0 if a < 0 else w + a for w, a in zip(want, add)]
        assert lens.tolist() == want
        check(r, T)
