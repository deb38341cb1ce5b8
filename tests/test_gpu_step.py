"""One decode step of a layer served from stored codes, as its operators are
used together: projections from codes plus each request's adapters, K and V
rows quantized into the cache as they come and read back, attention by the
caller, and an expert layer, several steps long, against float64."""
import numpy as np
import pytest

import oracle
from parity_util import Y_MAX_REL, Y_MEAN_REL, y_errors
from test_gpu_moe import _reference as moe_reference
from test_gpu_moe import _stored
from test_gpu_moe import _dev as moe_dev

pytestmark = pytest.mark.gpu


def test_decode_steps_of_a_layer():
    import torch
    import online_activation_aware_ttq_amd as ttq
    rng = np.random.default_rng(3)
    R, d, heads, hd, ff, E, n_ad, rank = 3, 256, 4, 64, 128, 4, 2, 8
    bits, group, page, prompt, steps = 4, 64, 4, [5, 9, 2], 3

    def bf16(v):
        return torch.from_numpy(np.asarray(v, np.float32)).cuda().to(torch.bfloat16)

    def f64(t):
        return t.double().cpu().numpy()

    # weights, quantized once for a prompt's activations
    Xp = bf16(rng.standard_normal((16, d)))
    kw = dict(bits=bits, group=group)

    def quantize(d_out):
        W = bf16(rng.standard_normal((d_out, d)) * 0.05)
        return ttq.ttq_quantize(W, Xp, p=2.0, lam=1e-3, alpha=0.5, **kw)

    qkv, out = quantize(3 * d), quantize(d)
    index = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    ad = {n: (bf16(rng.standard_normal((n_ad, rank, d)) * 0.05),
              bf16(rng.standard_normal((n_ad, o, rank)) * 0.05)) for n, o in (("qkv", 3 * d), ("out", d))}
    gu, dn = (_stored(rng, E, r, c, bits, group, "asym") for r, c in ((2 * ff, d), (d, ff)))
    router = bf16(rng.standard_normal((E, d)) * 0.2)
    gud, dnd = moe_dev(gu), moe_dev(dn)

    # the cache: K and V of a token side by side, 8 bits, pages of 4 rows
    slots_n = 64
    cache = (torch.zeros(slots_n, 2 * d, dtype=torch.uint8, device="cuda"),
             torch.zeros(slots_n, 2 * d // group, device="cuda"),
             torch.zeros(slots_n, 2 * d // group, device="cuda"))
    pages = torch.from_numpy(rng.permutation(16)[:12].reshape(R, 4).astype(np.int32)).cuda()
    ckw = dict(bits=8, group=group)

    def slots(seq, pos):
        p = pages.cpu().numpy()
        return int(p[seq, pos // page]) * page + pos % page

    history = [np.zeros((0, 2 * d)) for _ in range(R)]  # what was written, float64
    for i, n in enumerate(prompt):
        kv = torch.from_numpy(rng.standard_normal((n, 2 * d)).astype(np.float32)).cuda()
        at = torch.tensor([slots(i, t) for t in range(n)], device="cuda")
        ttq.ttq_cache_write(kv, at, *cache, **ckw)
        history[i] = f64(kv)

    def stored64(q):
        lv = oracle.unpack_codes(q[0].cpu().numpy(), bits, d).astype(np.float64)
        G = d // group
        W = f64(q[2])[:, :, None] + f64(q[1])[:, :, None] * lv.reshape(len(lv), G, group)
        return W.reshape(len(lv), d) * f64(q[3])

    Wqkv, Wout = stored64(qkv), stored64(out)

    def project64(W, pair, x):
        A, B = f64(pair[0]), f64(pair[1])
        y = x @ W.T
        for t, e in enumerate(index.cpu().numpy()):
            if e >= 0:
                y[t] += B[e] @ (A[e] @ x[t])
        return y

    x = bf16(rng.standard_normal((R, d)))
    for step in range(steps):
        x64 = f64(x)
        y = ttq.ttq_qmatmul(*qkv, x, **kw)
        ttq.ttq_adapters(x, *ad["qkv"], index, base=y, Y=y)
        lens = [p + step + 1 for p in prompt]
        at = torch.tensor([slots(i, n - 1) for i, n in enumerate(lens)], device="cuda")
        ttq.ttq_cache_write(y[:, d:], at, *cache, **ckw)        # a column range of the projection
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kv = ttq.ttq_cache_read(*cache, pages, ld, page_tokens=page, T=16, d=2 * d,
                                dtype=torch.float32, **ckw)
        ref = project64(Wqkv, ad["qkv"], x64)
        e, _ = y_errors(y.cpu().numpy(), ref)
        assert e.max() <= Y_MAX_REL and e.mean() <= Y_MEAN_REL
        att, att_ref = [], []
        for i, n in enumerate(lens):
            # the cache holds the GPU's projection; its rows stay where they were
            history[i] = np.concatenate([history[i], f64(y[i:i + 1, d:])])
            got, want = f64(kv[i, :n]), history[i]
            grp = want.reshape(n, -1, group)
            half = (grp.max(-1) - grp.min(-1)) / 255 / 2
            assert (np.abs(got - want).reshape(grp.shape).max(-1) <= half * (1 + 1e-5) + 1e-6).all()
            assert (kv[i, n:] == 0).all()

            def attend(q, kv):
                k, v = kv[:, :d].reshape(n, heads, hd), kv[:, d:].reshape(n, heads, hd)
                s = np.einsum("hc,nhc->hn", q.reshape(heads, hd), k) / np.sqrt(hd)
                p = np.exp(s - s.max(1, keepdims=True))
                return np.einsum("hn,nhc->hc", p / p.sum(1, keepdims=True), v).reshape(d)

            att.append(attend(f64(y[i, :d]), got))
            att_ref.append(attend(f64(y[i, :d]), want))
        # half a step of 8 bits on keys and values moves the heads' means little
        assert np.abs(np.array(att) - np.array(att_ref)).max() <= 0.05 * np.abs(att_ref).max()
        a = bf16(np.array(att))
        o = ttq.ttq_adapters(a, *ad["out"], index, base=ttq.ttq_qmatmul(*out, a, **kw))
        e, _ = y_errors(o.cpu().numpy(), project64(Wout, ad["out"], f64(a)))
        assert e.max() <= Y_MAX_REL and e.mean() <= Y_MEAN_REL
        h = (x.float() + o).to(torch.bfloat16)
        mlp = ttq.ttq_moe(h, router, *gud, *dnd, top_k=2, **kw)
        want, tol, _, _ = moe_reference(f64(h), f64(router), gu, dn, 2, group)
        assert (np.abs(f64(mlp) - want) <= tol).all()
        x = (h.float() + mlp).to(torch.bfloat16)
    assert torch.isfinite(x).all()
