"""ttq_adapters on the GPU against float64.

Two kinds of checks.  With small integers every product and partial sum is a
whole number below 2^24, so the result must be equal, whatever the order of
the sums: this is what holds the first product's 24 bits in the second.  With
ordinary values, the error of each output is bounded by the arithmetic: a sum
of n terms in float32, in any order, is off by at most n 2^-24 of the sum of
their magnitudes; the first product has d terms, the second 3 rank (three
planes) plus the partial sums' and the last fused multiply-add's roundings.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _reference(X, A, B, c, index, base):
    """float64 Y and the bound above."""
    T, d = X.shape
    n, r, _ = A.shape
    Y, tol = base.copy(), np.zeros_like(base)
    for t, e in enumerate(index):
        if not 0 <= e < n:
            continue
        S, mag = A[e] @ X[t], np.abs(A[e]) @ np.abs(X[t])
        Y[t] += c[e] * (B[e] @ S)
        tol[t] = U * abs(c[e]) * (np.abs(B[e]) @ ((d + 3 * r + 16) * mag))
    return Y, tol + 2 * U * (np.abs(Y) + np.abs(base))


def _run(X, A, B, c, index, base, **kw):
    import torch
    import online_activation_aware_ttq_amd as ttq
    bf = lambda v: torch.from_numpy(v.astype(np.float32)).cuda().to(torch.bfloat16)
    f32 = lambda v: None if v is None else torch.from_numpy(v.astype(np.float32)).cuda()
    Y = ttq.ttq_adapters(bf(X), bf(A), bf(B), torch.from_numpy(np.asarray(index, np.int32)).cuda(),
                         scale=f32(c), base=f32(base), **kw)
    torch.cuda.synchronize()
    return Y.double().cpu().numpy()


SHAPES = [
    # T, n, rank, d, d_out
    (1, 1, 8, 8, 1), (1, 5, 16, 512, 512), (2, 3, 24, 64, 3), (15, 4, 32, 520, 77),
    (16, 16, 8, 1032, 130), (17, 2, 64, 128, 1000), (33, 7, 128, 264, 36),
    (40, 1, 40, 4104, 260), (64, 100, 16, 256, 64), (300, 9, 48, 96, 129),
    (1100, 3, 16, 64, 40), (17000, 4, 8, 16, 8),
    (128, 60, 24, 2048, 5001), (129, 2, 64, 72, 516), (200, 5, 128, 136, 70), (700, 3, 88, 40, 2600),
    (96, 1, 72, 1000, 300),
]


@pytest.mark.parametrize("T,n,r,d,do", SHAPES)
def test_whole_numbers_are_exact(T, n, r, d, do):
    print(f"[case] adapters exact T={T} n={n} r={r} d={d} d_out={do}", flush=True)
    rng = np.random.default_rng(T * 7 + d)
    top = 120 if d <= 64 else 40  # |S| <= d * top^2 / density, see the assertion
    X = rng.integers(-top, top + 1, (T, d)).astype(np.float64)
    X[:, rng.random(d) > min(1.0, 64 / d)] = 0
    A = rng.integers(-top, top + 1, (n, r, d)).astype(np.float64)
    B = np.zeros((n, do, r))
    for e in range(n):  # three of the rank's columns in each output
        for k in range(3):
            B[e, np.arange(do), rng.integers(0, r, do)] = rng.choice([-1.0, 1.0, 2.0], do)
    c = rng.choice([1.0, -1.0, 0.5], n)
    index = rng.integers(-1, n + 1, T)
    base = rng.integers(-1000, 1000, (T, do)).astype(np.float64)
    mag = max((np.abs(B[e]) @ (np.abs(A[e]) @ np.abs(X).T)).max() for e in range(n))
    assert mag + 1000 < 2 ** 23
    ref, _ = _reference(X, A, B, c, index, base)
    np.testing.assert_array_equal(_run(X, A, B, c, index, base), ref)


def _data(T, n, r, d, do, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    bf = lambda v: torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).double().numpy()
    X = rng.standard_normal((T, d))
    X[:, rng.integers(0, d, max(1, d // 50))] *= 50
    return (bf(X), bf(rng.standard_normal((n, r, d)) * 0.02), bf(rng.standard_normal((n, do, r)) * 0.02),
            np.float32(0.5 + rng.random(n)).astype(np.float64), rng.integers(-1, n + 1, T),
            np.float32(rng.standard_normal((T, do))).astype(np.float64))


@pytest.mark.parametrize("T,n,r,d,do", SHAPES)
def test_values(T, n, r, d, do):
    print(f"[case] adapters T={T} n={n} r={r} d={d} d_out={do}", flush=True)
    X, A, B, c, index, base = _data(T, n, r, d, do, T + d)
    ref, tol = _reference(X, A, B, c, index, base)
    assert (np.abs(_run(X, A, B, c, index, base) - ref) <= tol).all()
    # without scales and base
    ref, tol = _reference(X, A, B, np.ones(n), index, np.zeros_like(base))
    got = _run(X, A, B, None, index, None)
    assert (np.abs(got - ref) <= tol).all()
    none = (index < 0) | (index >= n)
    assert (got[none] == 0).all()


@pytest.mark.parametrize("how", ["same", "none", "sorted", "one_each"])
def test_index_patterns(how):
    T, n = 50, 60
    X, A, B, c, index, base = _data(T, n, 16, 128, 96, 5)
    index = {"same": np.full(T, 37), "none": np.full(T, -1), "sorted": np.arange(T) // 7,
             "one_each": np.random.default_rng(1).permutation(n)[:T]}[how]
    ref, tol = _reference(X, A, B, c, index, base)
    got = _run(X, A, B, c, index, base)
    assert (np.abs(got - ref) <= tol).all()
    if how == "none":
        np.testing.assert_array_equal(got, base)


def test_rows_do_not_depend_on_their_batch():
    X, A, B, c, index, base = _data(70, 6, 32, 256, 200, 9)
    whole = _run(X, A, B, c, index, base)
    for t in (0, 17, 69):
        one = _run(X[t:t + 1], A, B, c, index[t:t + 1], base[t:t + 1])
        # other ranges of channels may be summed: within the bound of both
        _, tol = _reference(X[t:t + 1], A, B, c, index[t:t + 1], base[t:t + 1])
        assert (np.abs(one - whole[t:t + 1]) <= 2 * tol).all()
    np.testing.assert_array_equal(whole, _run(X, A, B, c, index, base))  # the same bits again


def test_what_is_not_finite_stays_in_its_row():
    X, A, B, c, index, base = _data(20, 4, 8, 64, 40, 11)
    index[:] = np.arange(20) % 3          # pair 3 is never used
    A[3] = np.nan
    B[3] = np.inf
    X[4, 10] = np.nan
    X[5, 11] = np.inf
    B[2, 7, :] = np.nan                   # an output of pair 2
    base[8, 1] = np.inf
    A[2][:, 11] = 0.5                     # row 5 names pair 2: all of S is +infinity,
    B[2][3], B[2][4] = 0.25, -0.25        # and where B has one sign, so is the output
    got = _run(X, A, B, c, index, base)
    clean = [x.copy() for x in (X, A, B, base)]
    for x in clean:
        x[~np.isfinite(x)] = 0
    ref, tol = _reference(clean[0], clean[1], clean[2], c, index, clean[3])
    bad = np.zeros(got.shape, bool)
    bad[4] = bad[5] = True
    bad[index == 2, 7] = True
    bad[8, 1] = True
    assert (np.abs(got - ref)[~bad] <= tol[~bad]).all()
    assert np.isnan(got[4]).all() and not np.isfinite(got[5]).any()
    assert got[5, 3] == np.inf and got[5, 4] == -np.inf
    assert np.isnan(got[index == 2, 7]).all() and got[8, 1] == np.inf


def test_in_place_no_pairs_and_caller_workspace():
    import torch
    import online_activation_aware_ttq_amd as ttq
    X, A, B, c, index, base = _data(9, 3, 8, 64, 33, 13)
    ref = _run(X, A, B, c, index, base)
    bf = lambda v: torch.from_numpy(v.astype(np.float32)).cuda().to(torch.bfloat16)
    Y = torch.from_numpy(base.astype(np.float32)).cuda()
    idx = torch.from_numpy(index.astype(np.int32)).cuda()
    prm = ttq.make_params(d=64, d_out=33, T=9, rank=8, bits=4, group=32, p=1, lam=0, alpha=0)
    ws = torch.empty(ttq.ttq_adapters_workspace_bytes(prm, 3), dtype=torch.uint8, device="cuda")
    r = ttq.ttq_adapters(bf(X), bf(A), bf(B), idx, scale=torch.from_numpy(c).float().cuda(), base=Y,
                         Y=Y, workspace=ws)
    assert r is Y
    np.testing.assert_array_equal(Y.double().cpu().numpy(), ref)
    z = ttq.ttq_adapters(bf(X), bf(A)[:0], bf(B)[:0], idx, base=Y)
    assert torch.equal(z, Y)
    assert ttq.ttq_adapters(bf(X)[:0], bf(A), bf(B), idx[:0]).shape == (0, 33)
    with pytest.raises(ValueError, match="workspace"):
        ttq.ttq_adapters(bf(X), bf(A), bf(B), idx, workspace=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(TypeError, match="workspace"):
        ttq.ttq_adapters(bf(X), bf(A), bf(B), idx, workspace=torch.empty(1 << 16, device="cuda"))
    big = torch.zeros(4, 8, 4096, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ttq.TTQError):  # too small for its partial sums
        ttq.ttq_adapters(torch.zeros(200, 4096, dtype=torch.bfloat16, device="cuda"), big,
                         big.transpose(1, 2).contiguous(), torch.zeros(200, dtype=torch.int32, device="cuda"),
                         workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_pairs_past_2_to_31_elements():
    import torch
    import online_activation_aware_ttq_amd as ttq
    n, r, d, do = 300, 128, 65536, 64    # A: 2.5e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.zeros(n, r, d, dtype=torch.bfloat16, device="cuda")
    for e in (0, 299):
        A[e] = torch.randint(-3, 4, (r, d), device="cuda", generator=g).to(torch.bfloat16)
    B = torch.zeros(n, do, r, dtype=torch.bfloat16, device="cuda")
    B[:, :, :64] = torch.eye(64, device="cuda").to(torch.bfloat16)
    X = torch.randint(-3, 4, (2, d), device="cuda", generator=g).to(torch.bfloat16)
    Y = ttq.ttq_adapters(X, A, B, torch.tensor([299, 0], dtype=torch.int32, device="cuda"))
    ref = torch.stack([(A[e, :64].double() @ X[i].double()) for i, e in enumerate((299, 0))])
    assert torch.equal(Y.double(), ref)


@pytest.mark.parametrize("T", [128, 200])
def test_tiles_of_2_to_31_bytes(T):
    """Whole numbers, so exact: the first and last of 2^22 outputs of every row."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    g = torch.Generator(device="cuda").manual_seed(T)
    do = 1 << 22
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(torch.bfloat16)
    X, A, B = ints(T, 64), ints(2, 8, 64), ints(2, do, 8)
    idx = (torch.arange(T, device="cuda") % 3 - 1).to(torch.int32)
    Y = ttq.ttq_adapters(X, A, B, idx)
    for cols in (slice(0, 300), slice(do - 300, do)):
        ref = torch.zeros(T, 300, dtype=torch.float64)
        for e in (0, 1):
            rows = (idx == e).cpu()
            ref[rows] = X.double().cpu()[rows] @ A[e].double().cpu().T @ B[e, cols].double().cpu().T
        assert torch.equal(Y[:, cols].double().cpu(), ref)


def test_captured_graphs_do_not_share_a_workspace():
    import torch
    import online_activation_aware_ttq_amd as ttq
    X, A, B, c, index, base = _data(24, 3, 16, 512, 256, 17)
    bf = lambda v: torch.from_numpy(v.astype(np.float32)).cuda().to(torch.bfloat16)
    A, B, idx = bf(A), bf(B), torch.from_numpy(index.astype(np.int32)).cuda()
    ttq.ttq_adapters(bf(X), A, B, idx)
    sets = []
    for k in range(2):
        x = bf(X) * (k + 1)
        graph = torch.cuda.CUDAGraph()
        y = torch.empty(24, 256, device="cuda")
        with torch.cuda.graph(graph):
            ttq.ttq_adapters(x, A, B, idx, Y=y)
        sets.append((graph, x, y))
    streams = [torch.cuda.Stream() for _ in sets]
    for step in range(4):
        for _, x, _ in sets:
            x.copy_(torch.randn(24, 512, device="cuda"))
        torch.cuda.synchronize()
        for (graph, _, _), s in zip(sets, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, x, y in sets:
            assert torch.equal(y, ttq.ttq_adapters(x, A, B, idx))
