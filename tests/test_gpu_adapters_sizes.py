"""ttq_adapters at the lengths of real layers, where the first product is split
over ranges of channels, with the bounds of test_gpu_adapters; and infinities."""
import numpy as np
import pytest

from test_gpu_adapters import _data, _reference, _run

pytestmark = pytest.mark.gpu

SHAPES = [
    # T, n, rank, d, d_out: prompts of two to four ranges, decode steps of two to eight
    (200, 3, 64, 1032, 129), (200, 5, 24, 4104, 260), (700, 4, 40, 1032, 77), (700, 2, 128, 4104, 68),
    (1500, 2, 8, 2056, 40), (131, 90, 16, 2056, 100), (129, 129, 72, 1544, 33),
    (127, 90, 48, 4104, 515), (24, 8, 64, 4104, 260), (128, 3, 128, 8200, 132), (8, 8, 104, 4096, 1000),
]


@pytest.mark.parametrize("T,n,r,d,do", SHAPES)
def test_values(T, n, r, d, do):
    print(f"[case] adapters T={T} n={n} r={r} d={d} d_out={do}", flush=True)
    X, A, B, c, index, base = _data(T, n, r, d, do, T + d)
    ref, tol = _reference(X, A, B, c, index, base)
    got = _run(X, A, B, c, index, base)
    assert (np.abs(got - ref) <= tol).all()
    np.testing.assert_array_equal(got, _run(X, A, B, c, index, base))


@pytest.mark.parametrize("T,n,r,d,do", SHAPES)
def test_whole_numbers_are_exact(T, n, r, d, do):
    """Products of small integers in every range of channels: sums below 2^23."""
    print(f"[case] adapters exact T={T} n={n} r={r} d={d} d_out={do}", flush=True)
    rng = np.random.default_rng(T + d)
    X = rng.integers(-7, 8, (T, d)).astype(np.float64)
    A = rng.integers(-7, 8, (n, r, d)).astype(np.float64)
    B = np.zeros((n, do, r))
    for e in range(n):
        for _ in range(3):
            B[e, np.arange(do), rng.integers(0, r, do)] = rng.choice([-1.0, 1.0, 2.0], do)
    c = rng.choice([1.0, -1.0, 0.5], n)
    index = rng.integers(-1, n + 1, T)
    base = rng.integers(-1000, 1000, (T, do)).astype(np.float64)
    assert 49 * d * 6 + 1000 < 2 ** 23
    ref, _ = _reference(X, A, B, c, index, base)
    np.testing.assert_array_equal(_run(X, A, B, c, index, base), ref)


@pytest.mark.parametrize("T", [3, 100, 300])
def test_infinite_second_factors_stay_in_their_output(T):
    X, A, B, c, index, base = _data(T, 3, 16, 1032 if T > 3 else 64, 40, 7)
    index[:] = np.arange(T) % 3
    ref, tol = _reference(X, A, B, c, index, base)
    B[1, 5, 2] = np.inf
    B[1, 6, :] = -np.inf
    got = _run(X, A, B, c, index, base)
    bad = np.zeros(got.shape, bool)
    bad[index == 1, 5] = bad[index == 1, 6] = True
    assert not np.isfinite(got[bad]).any()
    assert (np.abs(got - ref)[~bad] <= tol[~bad]).all()
