"""Refusals of the quantized cache (ttq_cache_write, ttq_cache_read): every
invalid call is answered on the host, before anything is enqueued (no GPU)."""
import ctypes

import pytest

import online_activation_aware_ttq_amd as ttq

FAKE = 0x7f0000000000  # 256-byte aligned, never dereferenced by validation


def prm(**kw):
    base = dict(d=256, d_out=0, T=4, bits=4, group=128, p=1.0, lam=0.0, alpha=0.0)
    base.update(kw)
    return ttq.make_params(**base)


def write(p, n_slots=64, x_type=0, X=FAKE, ldx=256, dhalf=None, slots=FAKE,
          codes=FAKE, scales=FAKE, mins=FAKE):
    return ttq.load_library().ttq_cache_write(
        ctypes.byref(p) if p is not None else None, n_slots, x_type, X, ldx,
        dhalf, slots, codes, scales, mins, None)


def read(p, n_slots=64, n_seq=2, max_pages=3, page=16, pages=FAKE, lens=FAKE,
         codes=FAKE, scales=FAKE, mins=FAKE, dhi=None, out_type=0, out=FAKE):
    return ttq.load_library().ttq_cache_read(
        ctypes.byref(p) if p is not None else None, n_slots, n_seq, max_pages,
        page, pages, lens, codes, scales, mins, dhi, out_type, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(bits=0), ttq.TTQ_EINVAL), (dict(bits=9), ttq.TTQ_EINVAL),
    (dict(d=0), ttq.TTQ_EINVAL), (dict(T=-1), ttq.TTQ_EINVAL),
    (dict(group=0), ttq.TTQ_EINVAL), (dict(group=96), ttq.TTQ_EINVAL),
    (dict(group=16), ttq.TTQ_EUNSUPPORTED), (dict(qformat=4), ttq.TTQ_EINVAL),
    (dict(qformat=1, bits=1), ttq.TTQ_EINVAL), (dict(qformat=3, bits=4), ttq.TTQ_EINVAL),
    (dict(flags=8), ttq.TTQ_EINVAL),
    (dict(d=32, group=32, bits=1), ttq.TTQ_EUNSUPPORTED),  # a row of 4 bytes
])
def test_parameters(kw, status):
    assert write(prm(**kw)) == status
    assert read(prm(**kw)) == status


def test_write_arguments():
    p = prm()
    assert write(None) == ttq.TTQ_ENULL
    for name in ("X", "slots", "codes", "scales", "mins"):
        assert write(p, **{name: None}) == ttq.TTQ_ENULL, name
    assert write(p, n_slots=-1) == ttq.TTQ_EINVAL
    assert write(p, x_type=2) == ttq.TTQ_EINVAL
    assert write(p, ldx=255) == ttq.TTQ_EINVAL
    assert write(p, ldx=260) == ttq.TTQ_EALIGN          # bf16 rows 520 bytes apart
    assert write(p, x_type=1, ldx=258) == ttq.TTQ_EALIGN
    assert write(p, X=FAKE + 8) == ttq.TTQ_EALIGN
    assert write(p, dhalf=FAKE + 4) == ttq.TTQ_EALIGN
    assert write(p, slots=FAKE + 4) == ttq.TTQ_EALIGN
    assert write(p, codes=FAKE + 8) == ttq.TTQ_EALIGN
    assert write(p, scales=FAKE + 2) == ttq.TTQ_EALIGN
    assert write(p, mins=FAKE + 1) == ttq.TTQ_EALIGN


def test_read_arguments():
    p = prm()
    assert read(None) == ttq.TTQ_ENULL
    for name in ("pages", "lens", "codes", "scales", "mins", "out"):
        assert read(p, **{name: None}) == ttq.TTQ_ENULL, name
    assert read(p, n_slots=-1) == ttq.TTQ_EINVAL
    assert read(p, n_seq=-1) == ttq.TTQ_EINVAL
    assert read(p, n_seq=65536) == ttq.TTQ_EINVAL
    assert read(p, max_pages=-1) == ttq.TTQ_EINVAL
    assert read(p, page=0) == ttq.TTQ_EINVAL
    assert read(p, page=24) == ttq.TTQ_EUNSUPPORTED
    assert read(p, page=8192) == ttq.TTQ_EUNSUPPORTED
    assert read(p, out_type=-1) == ttq.TTQ_EINVAL
    assert read(prm(d=1 << 19, T=1 << 15), n_seq=4096) == ttq.TTQ_EINVAL
    assert read(p, dhi=FAKE + 8) == ttq.TTQ_EALIGN
    assert read(p, out=FAKE + 8) == ttq.TTQ_EALIGN
    assert read(p, lens=FAKE + 2) == ttq.TTQ_EALIGN
    assert read(p, pages=FAKE + 2) == ttq.TTQ_EALIGN


def test_nothing_to_do():
    assert write(prm(T=0), X=None, slots=None, ldx=0) == ttq.TTQ_OK
    assert write(prm(), n_slots=0, codes=None, scales=None, mins=None) == ttq.TTQ_OK
    assert read(prm(T=0), out=None) == ttq.TTQ_OK
    assert read(prm(), n_seq=0, pages=None, lens=None) == ttq.TTQ_OK
    assert read(prm(), max_pages=0, pages=None) == ttq.TTQ_OK


def test_injected_hip_error_is_reported(monkeypatch):
    monkeypatch.setenv("TTQ_INJECT_HIP_ERROR", "1")
    assert write(prm()) == ttq.TTQ_EHIP
    assert read(prm()) == ttq.TTQ_EHIP


def test_binding_checks_tensors():
    import torch
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    z = torch.zeros(8, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        ttq.ttq_cache_write(X, torch.zeros(4, dtype=torch.int64),
                            torch.zeros(8, 128, dtype=torch.uint8), z, z, bits=4, group=128)


@pytest.mark.parametrize("fmt,bits", [("asym", 1), ("asym", 4), ("asym", 8), ("sym", 3), ("intzp", 4),
                                      ("fp8", 8)])
def test_oracle_rows_are_within_half_a_step(fmt, bits):
    """The cache's quantizer in the oracle: every value within half a step of
    what it stands for (E4M3: half a unit of its binade), codes in range, and a
    repeated call the same."""
    import numpy as np
    import oracle
    rng = np.random.default_rng(bits)
    x = (rng.standard_normal((7, 96)) * 10.0 ** rng.integers(-3, 3, (7, 1))).astype(np.float32)
    x[3] = 0
    dh = (0.5 + rng.random(96)).astype(np.float32)
    q = oracle.cache_rows(x, dh, bits, 32, fmt)
    u = (x * dh).astype(np.float64)
    s = np.repeat(q["s"].astype(np.float64), 32, axis=1)
    half = s / 2
    if fmt == "fp8":  # 3 fraction bits, and subnormals below 2^-6
        half = s * 2.0 ** (np.floor(np.log2(np.maximum(np.abs(u) / np.where(s > 0, s, 1), 2.0 ** -6))) - 4)
    assert (np.abs(q["values"] - u) <= half * (1 + 1e-5) + 1e-30).all()
    assert q["codes"].max() <= (0xFE if fmt == "fp8" else 2 ** bits - 1)
    assert (q["values"][3] == 0).all()
    assert (oracle.cache_rows(x, dh, bits, 32, fmt)["codes"] == q["codes"]).all()
