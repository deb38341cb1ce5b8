"""What is not finite, or overflows, in ttq_moe: where it may be seen."""
import numpy as np
import pytest

from test_gpu_moe import _bf16, _reference, _run, _stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(1, 2, 2), (1, 1, 1), (3, 2, 2), (40, 1, 1)])
def test_a_row_of_nan_codes_stays_in_its_output(T, E, k):
    """Rows of 96 channels end inside a slot of codes: the next row's codes lie
    behind theirs.  A down row of NaN (E4M3 codes 0x7F) is its own output's alone."""
    rng = np.random.default_rng(T)
    d = ff = 96
    X, Wr = _bf16(rng.standard_normal((T, d))), _bf16(rng.standard_normal((E, d)) * 0.1)
    gu, dn = (_stored(rng, E, r, c, 8, 32, "fp8") for r, c in ((2 * ff, d), (d, ff)))
    ref, tol, _, _ = _reference(X, Wr, gu, dn, k, 32)
    for row in (1, 16, 63, 95):
        codes = dn["packed"].copy()
        codes[:, row] = 0x7F
        y, _, _ = _run(X, Wr, gu, dict(dn, packed=codes), k, 8, 32, "fp8")
        rest = np.arange(d) != row
        assert np.isnan(y[:, row]).all()
        assert (np.abs(y - ref)[:, rest] <= tol[:, rest]).all(), row


@pytest.mark.parametrize("E,d", [(6, 128), (70, 1024)])
@pytest.mark.parametrize("exp", [70, -80])
def test_scores_whose_products_leave_float32(E, d, exp):
    """Scores are float64: two bfloat16 values of 2^70 have a product of 2^140,
    two of 2^-80 one of 2^-160.  (70 experts of 1024: the scores' own launch.)"""
    rng = np.random.default_rng(E + exp + 100)
    T, ff, k = 3, 64, 4
    X, Wr = np.zeros((T, d)), np.zeros((E, d))
    X[:, 5] = 2.0 ** exp
    Wr[:, 5] = rng.permutation(E) * 2.0 ** exp * np.where(np.arange(E) % 3 == 0, -1, 1)
    gu, dn = (_stored(rng, E, r, c, 4, 32, "asym") for r, c in ((2 * ff, d), (d, ff)))
    gu["dhi"][:, 5] = 0                       # the channel is the router's alone
    X[:, 7:] = rng.standard_normal((T, d - 7))
    X = _bf16(X)
    ref, tol, ids, w = _reference(X, Wr, gu, dn, k, 32)
    y, gi, gw = _run(X, Wr, gu, dn, k, 4, 32, "asym")
    np.testing.assert_array_equal(gi, ids)
    assert np.abs(gw - w).max() <= 2.0 ** -20
    assert np.isfinite(y).all() and (np.abs(y - ref) <= tol).all()


@pytest.mark.parametrize("T,E", [(1, 2), (4, 2), (40, 1)])
@pytest.mark.parametrize("how", ["x", "hidden"])
def test_what_overflows_makes_its_own_row_nan(T, E, how):
    """An infinite x D^{-1/2}, or a product of gate and up past float32, is a row
    of NaN; every other row has the bits that it has without it."""
    rng = np.random.default_rng(T)
    d, ff = 96, 160
    X, Wr = _bf16(rng.standard_normal((T, d))), _bf16(rng.standard_normal((E, d)) * 0.1)
    Wr[:, 9] = 0
    X[:, 9] = 1
    gu, dn = (_stored(rng, E, r, c, 8, 32, "asym") for r, c in ((2 * ff, d), (d, ff)))
    ok, ids, w = _run(X, Wr, gu, dn, 1, 8, 32, "asym")
    assert np.isfinite(ok).all()
    bad = X.copy()
    if how == "x":
        gu["dhi"][:, 9] = 8                   # 2^126 times 8 is infinite, 1 times 8 is 8
        ok, ids, w = _run(X, Wr, gu, dn, 1, 8, 32, "asym")
        bad[T // 2, 9] = 2.0 ** 126
    else:
        bad[T // 2, 9] = 2.0 ** 80            # gate and up of 2^75 and more
    y, gi, gw = _run(bad, Wr, gu, dn, 1, 8, 32, "asym")
    rest = np.arange(T) != T // 2
    np.testing.assert_array_equal(gi, ids)    # (the router does not see the channel)
    np.testing.assert_array_equal(gw, w)
    assert np.isnan(y[T // 2]).all()
    np.testing.assert_array_equal(y[rest], ok[rest])
