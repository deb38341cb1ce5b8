"""ttq_moe at the lengths of real layers, one dimension long at a time, against
float64 with the bounds of test_gpu_moe: more scale groups than are staged at a
time in every kernel that stages them, 8-bit codes whose slots and scales would
pass 64 KiB of LDS together, the scores' own launch, and routing by several
workgroups a token."""
import numpy as np
import pytest

from test_gpu_moe import _bf16, _reference, _run, _stored

pytestmark = pytest.mark.gpu

CASES = [
    # T, E, k, d, ff, bits, group, fmt
    # 8-bit containers with more than 48 scale groups, up and down
    (1, 3, 2, 4096, 64, 8, 32, "fp8"),
    (3, 4, 2, 4096, 64, 8, 32, "fp8"),
    (3, 4, 2, 64, 4096, 8, 32, "asym"),
    (2, 2, 1, 2048, 96, 8, 32, "intzp"),
    (4, 3, 2, 128, 8192, 8, 128, "fp8"),
    (3, 2, 2, 8192, 128, 5, 128, "sym"),
    (2, 2, 1, 256, 16384, 8, 256, "asym"),
    # more than 80 groups of narrower codes
    (4, 3, 2, 4096, 64, 4, 32, "asym"),
    (3, 3, 2, 64, 4096, 2, 32, "asym"),
    (5, 3, 1, 128, 8192, 1, 32, "asym"),
    (2, 2, 2, 8192, 64, 4, 32, "asym"),
    # one token's down products: 40 to 320 groups at a time
    (1, 8, 5, 128, 4096, 4, 32, "asym"),
    (1, 16, 16, 64, 2080, 4, 32, "asym"),
    (1, 2, 1, 32, 11008, 4, 32, "asym"),
    (1, 9, 8, 64, 4096, 8, 32, "fp8"),
    # scores by a launch of their own, several workgroups a token in the routing
    (3, 64, 8, 2048, 128, 4, 128, "asym"),
    (1, 16, 2, 8192, 128, 4, 128, "asym"),
    (40, 70, 4, 1024, 64, 2, 64, "sym"),
    # many tokens an expert, long rows
    (70, 3, 2, 2048, 128, 4, 128, "asym"),
    (64, 2, 1, 128, 4096, 2, 64, "asym"),
    (48, 2, 1, 1056, 96, 8, 32, "fp8"),
]


@pytest.mark.parametrize("T,E,k,d,ff,bits,group,fmt", CASES)
def test_values(T, E, k, d, ff, bits, group, fmt):
    print(f"[case] moe T={T} E={E} k={k} d={d} ff={ff} {fmt} b{bits} g{group}", flush=True)
    rng = np.random.default_rng(T * 1000 + d + ff)
    X = rng.standard_normal((T, d))
    X[:, rng.integers(0, d, 2)] *= 20
    X, Wr = _bf16(X), _bf16(rng.standard_normal((E, d)) * 0.1)
    gu = _stored(rng, E, 2 * ff, d, bits, group, fmt)
    dn = _stored(rng, E, d, ff, bits, group, fmt)
    ref, tol, ids, w = _reference(X, Wr, gu, dn, k, group)
    y, gi, gw = _run(X, Wr, gu, dn, k, bits, group, fmt)
    np.testing.assert_array_equal(gi, ids)
    assert np.abs(gw - w).max() <= 2.0 ** -20
    assert np.isfinite(y).all() and (np.abs(y - ref) <= tol).all()


@pytest.mark.parametrize("fmt,bits,group,T", [("asym", 4, 128, 1), ("asym", 4, 64, 9), ("sym", 3, 32, 50),
                                              ("intzp", 8, 64, 3), ("fp8", 8, 32, 2)])
def test_experts_stored_by_ttq_quantize(fmt, bits, group, T):
    """Each expert's projections quantized by the library for a prompt, stacked,
    and contracted as they are."""
    import torch
    import oracle
    import online_activation_aware_ttq_amd as ttq
    rng = np.random.default_rng(bits * 10 + T)
    E, k, d, ff = 4, 2, 256, 384

    def bf16(*shape, sigma=1.0):
        return torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).cuda().bfloat16()

    def stored(rows, cols):
        q = [ttq.ttq_quantize(bf16(rows, cols, sigma=0.05), bf16(16, cols), p=2.0, lam=1e-3, alpha=0.5,
                              bits=bits, group=group, qformat=fmt) for _ in range(E)]
        dev = [torch.stack([x[i] for x in q]) for i in range(4)]
        packed, s, m, dhi = (v.cpu().numpy() for v in dev)
        codes = np.stack([oracle.unpack_codes(p, bits, cols) for p in packed])
        return dev, dict(s=s, m=m, dhi=dhi, levels=oracle.e4m3_decode(codes) if fmt == "fp8"
                         else codes.astype(np.float64))

    (gud, gu), (dnd, dn) = stored(2 * ff, d), stored(d, ff)
    X, Wr = bf16(T, d), bf16(E, d, sigma=0.1)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    y = ttq.ttq_moe(X, Wr, *gud, *dnd, top_k=k, bits=bits, group=group, qformat=fmt, ids_out=ids)
    f64 = lambda t: t.double().cpu().numpy()
    ref, tol, want, _ = _reference(f64(X), f64(Wr), gu, dn, k, group)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    assert (np.abs(f64(y) - ref) <= tol).all()
