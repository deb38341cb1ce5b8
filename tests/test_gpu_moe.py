"""ttq_moe on the GPU against float64.

Routing must be equal (scores are summed in float64; the tests' scores differ
by far more than its rounding).  With whole numbers and gates so large that
silu(g) = g, every value is a whole number below 2^24 and the result must be
equal.  With ordinary values the error of each output is bounded by the
arithmetic: float32 sums of n terms are off by at most n 2^-24 of the sum of
their magnitudes (three planes of x', K terms each, then the groups' two
terms), silu has a slope of at most 1.1, expf and the divisions are good to
2^-21.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _bf16(v):
    import torch
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).double().numpy()


def _stored(rng, E, rows, cols, bits, group, fmt, sigma=0.05):
    """Random stored projections, quantized by the oracle: a dict of arrays."""
    out = dict(packed=[], s=[], m=[], dhi=[], levels=[])
    for _ in range(E):
        W = (rng.standard_normal((rows, cols)) * sigma).astype(np.float32)
        dh = (0.3 + rng.random(cols) * 2).astype(np.float32)
        q = oracle.quantize_format(W, dh, bits, group, fmt)
        out["packed"].append(oracle.pack_codes(q["codes"], bits))
        out["s"].append(q["s"])
        out["m"].append(oracle.format_offsets(q["s"], bits, fmt, q.get("m"), q.get("z")))
        out["dhi"].append((np.float32(1) / dh).astype(np.float32))
        out["levels"].append(oracle.e4m3_decode(q["codes"]) if fmt == "fp8"
                             else q["codes"].astype(np.float64))
    return {k: np.stack(v) for k, v in out.items()}


def _route(X, Wr, k, renorm):
    logits = X @ Wr.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(logits, ids, 1)
    p = np.exp(top - top[:, :1])
    return ids, p / (p.sum(1, keepdims=True) if renorm
                     else np.exp(logits - top[:, :1]).sum(1, keepdims=True))


def _product(w, e, x, dx, group):
    """(value, bound) of expert e's stored rows times x known to within dx."""
    x1 = x * w["dhi"][e].astype(np.float64)
    d1 = np.abs(dx) * w["dhi"][e] + 2 * U * np.abs(x1)
    G = w["s"].shape[2]
    lv = w["levels"][e].reshape(-1, G, group)
    s, m = w["s"][e].astype(np.float64), w["m"][e].astype(np.float64)
    W = (m[:, :, None] + s[:, :, None] * lv).reshape(lv.shape[0], -1)
    mag = (np.abs(m)[:, :, None] + np.abs(s[:, :, None] * lv)).reshape(W.shape)
    return W @ x1, np.abs(W) @ d1 + (3 * W.shape[1] + 3 * G + 16) * U * (mag @ np.abs(x1))


def _reference(X, Wr, gu, dn, k, group, renorm=True):
    T, d = X.shape
    ff = dn["dhi"].shape[1]
    ids, w = _route(X, Wr, k, renorm)
    Y, tol = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            a, da = _product(gu, ids[t, j], X[t], 0 * X[t], group)
            g, u, dg, du = a[:ff], a[ff:], da[:ff], da[ff:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 2.0 ** -20 * np.abs(h)
            y, dy = _product(dn, ids[t, j], h, dh, group)
            Y[t] += w[t, j] * y
            tol[t] += w[t, j] * (dy + 2.0 ** -19 * np.abs(y))
    return Y, tol + k * U * np.abs(Y), ids, w


def _dev(w):
    import torch
    return [torch.from_numpy(np.ascontiguousarray(w[n])).cuda() for n in ("packed", "s", "m", "dhi")]


def _run(X, Wr, gu, dn, k, bits, group, fmt, renorm=True, **kw):
    import torch
    import online_activation_aware_ttq_amd as ttq
    bf = lambda v: torch.from_numpy(np.asarray(v, np.float32)).cuda().to(torch.bfloat16)
    T = len(X)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), np.nan, device="cuda")
    Y = ttq.ttq_moe(bf(X), bf(Wr), *_dev(gu), *_dev(dn), top_k=k, bits=bits, group=group,
                    qformat=fmt, renormalize=renorm, ids_out=ids, weights_out=w, **kw)
    torch.cuda.synchronize()
    return Y.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy()


CASES = [
    # T, E, k, d, ff, bits, group, fmt, renorm
    (1, 8, 2, 256, 384, 4, 128, "asym", True),
    (1, 1, 1, 128, 32, 4, 32, "asym", True),
    (3, 5, 5, 96, 160, 8, 32, "asym", False),
    (16, 64, 8, 128, 128, 4, 64, "asym", True),
    (17, 4, 1, 192, 64, 3, 64, "sym", False),
    (40, 3, 2, 256, 320, 2, 32, "asym", True),
    (97, 16, 4, 128, 192, 4, 64, "intzp", True),
    (128, 2, 1, 512, 256, 4, 256, "asym", True),
    (5, 256, 16, 128, 128, 1, 128, "asym", True),
    (2, 7, 3, 256, 256, 8, 128, "fp8", True),
    (20, 9, 2, 96, 224, 8, 32, "fp8", False),
    (9, 6, 2, 512, 768, 8, 256, "intzp", True),
    (1, 100, 10, 256, 128, 2, 128, "sym", True),
    # many tokens an expert: their planes go through LDS
    (128, 1, 1, 384, 128, 4, 128, "asym", True),
    (33, 1, 1, 96, 160, 8, 32, "asym", True),
    (60, 2, 1, 96, 224, 8, 32, "fp8", True),
    (50, 2, 2, 256, 384, 8, 128, "fp8", False),
    (77, 3, 2, 128, 640, 1, 128, "asym", True),
    (45, 2, 1, 512, 768, 3, 256, "sym", True),
    (64, 2, 1, 768, 256, 8, 256, "intzp", True),
    (90, 4, 2, 320, 64, 2, 64, "asym", True),
    (128, 9, 8, 128, 288, 4, 32, "asym", True),
    # several passes over the codes
    (24, 2, 1, 256, 192, 4, 64, "asym", True),
    (13, 1, 1, 640, 96, 8, 32, "fp8", True),
    (26, 4, 2, 512, 768, 2, 256, "sym", True),
]


@pytest.mark.parametrize("T,E,k,d,ff,bits,group,fmt,renorm", CASES)
def test_values(T, E, k, d, ff, bits, group, fmt, renorm):
    print(f"[case] moe T={T} E={E} k={k} d={d} ff={ff} {fmt} b{bits} g{group}", flush=True)
    rng = np.random.default_rng(T * 100 + E)
    X = rng.standard_normal((T, d))
    X[:, rng.integers(0, d, 2)] *= 20
    X, Wr = _bf16(X), _bf16(rng.standard_normal((E, d)) * 0.1)
    gu = _stored(rng, E, 2 * ff, d, bits, group, fmt)
    dn = _stored(rng, E, d, ff, bits, group, fmt)
    ref, tol, ids, w = _reference(X, Wr, gu, dn, k, group, renorm)
    y, gi, gw = _run(X, Wr, gu, dn, k, bits, group, fmt, renorm)
    np.testing.assert_array_equal(gi, ids)
    assert np.abs(gw - w).max() <= 2.0 ** -20
    assert np.isfinite(y).all() and (np.abs(y - ref) <= tol).all()


@pytest.mark.parametrize("bits,group,T,E", [(4, 128, 1, 3), (4, 32, 20, 2), (2, 64, 5, 4), (1, 128, 2, 2),
                                            (8, 64, 18, 2), (3, 256, 1, 2), (4, 128, 70, 1),
                                            (2, 64, 70, 2), (8, 128, 64, 1), (1, 32, 48, 1)])
def test_whole_numbers_are_exact(bits, group, T, E):
    d, ff = 256, 256
    rng = np.random.default_rng(bits * 10 + T)
    X = np.zeros((T, d))
    live = 1 if bits == 8 else 8                    # few channels, all of them positive
    X[:, :live] = rng.integers(1, 4, (T, live))
    X[:, 100] = 1
    Wr = rng.integers(-3, 4, (E, d)).astype(float)
    Wr[:, 200] = 0

    def whole(rows, cols, lo):
        codes = rng.integers(0, 2 ** bits, (E, rows, cols)).astype(np.uint8)
        if bits == 8 and rows == 2 * ff:
            codes[:, ff:] &= 1                      # up rows small, the others of all 8 bits
        G = cols // group
        s = np.ones((E, rows, G), np.float32)
        m = np.full((E, rows, G), lo, np.float32)
        dhi = np.float32(2.0) ** rng.integers(0, 2, (E, cols)).astype(np.float32)
        return dict(packed=np.stack([oracle.pack_codes(c, bits) for c in codes]), s=s, m=m, dhi=dhi,
                    levels=codes.astype(np.float64))

    gu = whole(2 * ff, d, 1.0)
    gu["m"][:, :ff] = 54 // (live + 1)              # gates of at least 54: exp(-54) < 2^-25
    dn = whole(d, ff, -1.0)
    # keep the sums below 2^24: few hidden channels pass
    dn["dhi"][:, 12:] = 0
    gu["dhi"][:, :] = 1
    ref, _, ids, w = _reference(X, Wr, gu, dn, 1, group)
    assert np.abs(ref).max() < 2 ** 24 and (w == 1).all()
    y, gi, _ = _run(X, Wr, gu, dn, 1, bits, group, "asym")
    np.testing.assert_array_equal(gi, ids)
    np.testing.assert_array_equal(y, ref)


def test_ties_nan_and_infinite_scores():
    rng = np.random.default_rng(4)
    E, d, ff, k = 6, 128, 32, 3
    X = np.zeros((4, d))
    X[:, 0], X[:, 1] = 1, 1
    Wr = np.zeros((E, d))
    Wr[:, 0] = [2, 5, 5, 5, 1, 5]                   # equal scores go to the lower index
    gu, dn = (_stored(rng, E, r, c, 4, 32, "asym") for r, c in ((2 * ff, d), (d, ff)))
    y, ids, w = _run(X, Wr, gu, dn, k, 4, 32, "asym")
    assert (ids == [1, 2, 3]).all() and np.abs(w - 1 / 3).max() < 1e-6
    Wr[2, 1], Wr[4, 1] = np.nan, np.inf             # NaN last, infinity first
    y, ids, w = _run(X, Wr, gu, dn, k, 4, 32, "asym")
    assert (ids == [4, 1, 3]).all()
    Wr[:, 1] = np.nan                               # nothing but NaN: by index, no stray expert
    y, ids, w = _run(X, Wr, gu, dn, k, 4, 32, "asym")
    assert (ids == [0, 1, 2]).all() and np.isnan(y).all()
    # a row of NaN leaves the other rows alone
    Wr[:, 1] = 0
    ok, _, _ = _run(X, Wr, gu, dn, k, 4, 32, "asym")
    X[2, 7] = np.nan
    y, _, _ = _run(X, Wr, gu, dn, k, 4, 32, "asym")
    assert np.isnan(y[2]).all()
    np.testing.assert_array_equal(y[[0, 1, 3]], ok[[0, 1, 3]])


def test_repeats_bits_and_rows_stand_alone():
    rng = np.random.default_rng(8)
    T, E, k, d, ff = 40, 8, 2, 256, 384
    X, Wr = _bf16(rng.standard_normal((T, d))), _bf16(rng.standard_normal((E, d)) * 0.1)
    gu, dn = (_stored(rng, E, r, c, 4, 128, "asym") for r, c in ((2 * ff, d), (d, ff)))
    a = _run(X, Wr, gu, dn, k, 4, 128, "asym")
    b = _run(X, Wr, gu, dn, k, 4, 128, "asym")
    for u, v in zip(a, b):
        np.testing.assert_array_equal(u, v)
    _, tol, _, _ = _reference(X, Wr, gu, dn, k, 128)
    for t in (0, 39):
        one = _run(X[t:t + 1], Wr, gu, dn, k, 4, 128, "asym")
        assert (np.abs(one[0] - a[0][t]) <= 2 * tol[t]).all()
        np.testing.assert_array_equal(one[1][0], a[1][t])


def test_captured_on_streams_of_their_own():
    import torch
    import online_activation_aware_ttq_amd as ttq
    rng = np.random.default_rng(12)
    T, E, k, d, ff = 6, 8, 2, 256, 256
    gu, dn = (_dev(_stored(rng, E, r, c, 4, 128, "asym")) for r, c in ((2 * ff, d), (d, ff)))
    Wr = torch.from_numpy(rng.standard_normal((E, d)) * 0.1).cuda().to(torch.bfloat16)
    kw = dict(top_k=k, bits=4, group=128)
    X0 = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    ttq.ttq_moe(X0, Wr, *gu, *dn, **kw)
    sets = []
    for _ in range(2):
        x, y = X0.clone(), torch.empty(T, d, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ttq.ttq_moe(x, Wr, *gu, *dn, Y=y, **kw)
        sets.append((graph, x, y, torch.cuda.Stream()))
    for _ in range(4):
        for _, x, _, _ in sets:
            x.copy_(torch.randn(T, d, device="cuda"))
        torch.cuda.synchronize()
        for graph, _, _, s in sets:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, x, y, _ in sets:
            assert torch.equal(y, ttq.ttq_moe(x, Wr, *gu, *dn, **kw))
