"""Refusals of ttq_adapters and ttq_moe: every invalid call is answered on the
host, before anything is enqueued (no GPU)."""
import ctypes

import pytest

import online_activation_aware_ttq_amd as ttq

FAKE = 0x7f0000000000  # 256-byte aligned, never dereferenced by validation


def lib():
    return ttq.load_library()


# ---------------------------------------------------------------- adapters
def aprm(**kw):
    base = dict(d=256, d_out=100, T=200, rank=16, bits=0, group=0, p=0.0, lam=0.0, alpha=0.0)
    base.update(kw)
    return ttq.make_params(**base)


def adapters(p, n=3, X=FAKE, A=FAKE, B=FAKE, scale=None, index=FAKE, base=None, Y=FAKE,
             ws=FAKE, ws_bytes=1 << 40):
    return lib().ttq_adapters(ctypes.byref(p) if p is not None else None, n, X, A, B, scale,
                              index, base, Y, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), ttq.TTQ_EINVAL), (dict(d=(1 << 20) + 8), ttq.TTQ_EINVAL),
    (dict(d_out=-1), ttq.TTQ_EINVAL), (dict(T=-1), ttq.TTQ_EINVAL),
    (dict(rank=0), ttq.TTQ_EINVAL), (dict(rank=-8), ttq.TTQ_EINVAL),
    (dict(T=1 << 22, d=1 << 13), ttq.TTQ_EINVAL),
    (dict(rank=12), ttq.TTQ_EUNSUPPORTED), (dict(rank=136), ttq.TTQ_EUNSUPPORTED),
    (dict(d=100), ttq.TTQ_EUNSUPPORTED),
])
def test_adapter_parameters(kw, status):
    out = ctypes.c_size_t(7)
    assert adapters(aprm(**kw)) == status
    assert lib().ttq_adapters_workspace_bytes(ctypes.byref(aprm(**kw)), 3, ctypes.byref(out)) == status
    assert out.value == 7


def test_adapter_arguments():
    p = aprm()
    need = ttq.ttq_adapters_workspace_bytes(p, 3)
    assert need > 0
    assert adapters(None) == ttq.TTQ_ENULL
    for name in ("X", "A", "B", "index", "Y", "ws"):
        assert adapters(p, **{name: None}) == ttq.TTQ_ENULL, name
    assert lib().ttq_adapters_workspace_bytes(ctypes.byref(p), 3, None) == ttq.TTQ_ENULL
    assert adapters(p, n=-1) == ttq.TTQ_EINVAL
    assert adapters(p, n=(1 << 20) + 1) == ttq.TTQ_EINVAL
    for name, off in (("X", 8), ("A", 2), ("B", 8), ("scale", 2), ("index", 1), ("base", 2),
                      ("Y", 2), ("ws", 128)):
        assert adapters(p, **{name: FAKE + off}) == ttq.TTQ_EALIGN, name
    assert adapters(p, ws_bytes=need - 1) == ttq.TTQ_EWORKSPACE


def test_adapters_workspace_of_every_size():
    for T in (0, 1, 127, 128, 129, 4096, 100000):
        for n in (0, 1, 1000):
            for d in (8, 512, 1 << 17):
                need = ttq.ttq_adapters_workspace_bytes(aprm(T=T, d=d), n)
                # none for nothing, nor for steps small enough for one launch
                assert need <= (8 if T <= 128 else 4) * T * 16 * 4  # partial sums
                assert (need > 0) == (T > 128 or (T > 0 and d == 1 << 17))


def test_adapters_nothing_to_do():
    nul = dict(X=None, A=None, B=None, index=None, Y=None, ws=None)
    assert adapters(aprm(T=0), **nul) == ttq.TTQ_OK
    assert adapters(aprm(d_out=0), **nul) == ttq.TTQ_OK


# --------------------------------------------------------------------- moe
def mprm(**kw):
    base = dict(T=3, d=256, ff=512, experts=8, top_k=2, bits=4, group=128)
    base.update(kw)
    return ttq.make_moe_params(**base)


NAMES = ("X", "router", "gu_codes", "gu_scales", "gu_mins", "gu_dhi", "dn_codes", "dn_scales",
         "dn_mins", "dn_dhi", "Y", "ids", "weights", "ws")


def moe(p, ws_bytes=1 << 40, **kw):
    v = dict.fromkeys(NAMES, FAKE)
    v["ids"] = v["weights"] = None
    v.update(kw)
    return lib().ttq_moe(ctypes.byref(p) if p is not None else None, *[v[n] for n in NAMES],
                         ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ttq.TTQ_EINVAL), (dict(d=0), ttq.TTQ_EINVAL), (dict(ff=0), ttq.TTQ_EINVAL),
    (dict(experts=0), ttq.TTQ_EINVAL), (dict(top_k=0), ttq.TTQ_EINVAL),
    (dict(top_k=9), ttq.TTQ_EINVAL), (dict(bits=0), ttq.TTQ_EINVAL), (dict(bits=9), ttq.TTQ_EINVAL),
    (dict(group=0), ttq.TTQ_EINVAL), (dict(group=96), ttq.TTQ_EINVAL),
    (dict(ff=192), ttq.TTQ_EINVAL),                      # group does not divide it
    (dict(qformat=4), ttq.TTQ_EINVAL), (dict(qformat="sym", bits=1), ttq.TTQ_EINVAL),
    (dict(qformat="fp8"), ttq.TTQ_EINVAL),
    (dict(d=1 << 18, ff=1 << 18), ttq.TTQ_EINVAL),
    (dict(group=16), ttq.TTQ_EUNSUPPORTED), (dict(T=129), ttq.TTQ_EUNSUPPORTED),
    (dict(experts=257), ttq.TTQ_EUNSUPPORTED), (dict(experts=64, top_k=17), ttq.TTQ_EUNSUPPORTED),
    (dict(d=96, ff=96, group=32, bits=1), ttq.TTQ_EUNSUPPORTED),  # rows of 12 bytes
])
def test_moe_parameters(kw, status):
    out = ctypes.c_size_t(7)
    assert moe(mprm(**kw)) == status
    assert lib().ttq_moe_workspace_bytes(ctypes.byref(mprm(**kw)), ctypes.byref(out)) == status
    assert out.value == 7


def test_moe_arguments():
    p = mprm()
    need = ttq.ttq_moe_workspace_bytes(p)
    assert need > 0
    assert moe(None) == ttq.TTQ_ENULL
    for name in NAMES:
        if name not in ("ids", "weights"):
            assert moe(p, **{name: None}) == ttq.TTQ_ENULL, name
    for name, off in (("X", 8), ("router", 8), ("gu_codes", 8), ("gu_scales", 2), ("gu_mins", 1),
                      ("gu_dhi", 4), ("dn_codes", 4), ("dn_scales", 2), ("dn_mins", 2),
                      ("dn_dhi", 8), ("Y", 4), ("ids", 2), ("weights", 1), ("ws", 16)):
        assert moe(p, **{name: FAKE + off}) == ttq.TTQ_EALIGN, name
    assert moe(p, ws_bytes=need - 1) == ttq.TTQ_EWORKSPACE
    q = mprm()
    q.flags = 2
    assert moe(q) == ttq.TTQ_EINVAL
    assert lib().ttq_moe_workspace_bytes(ctypes.byref(p), None) == ttq.TTQ_ENULL


def test_moe_nothing_to_do():
    assert moe(mprm(T=0), **{n: None for n in NAMES}) == ttq.TTQ_OK


def test_injected_hip_error_is_reported(monkeypatch):
    monkeypatch.setenv("TTQ_INJECT_HIP_ERROR", "1")
    assert adapters(aprm()) == ttq.TTQ_EHIP
    assert moe(mprm()) == ttq.TTQ_EHIP


def test_moe_struct_matches_header_layout():
    assert ctypes.sizeof(ttq.ttq_moe_params) == 3 * 8 + 6 * 4


def test_binding_checks_tensors():
    import torch
    X = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        ttq.ttq_adapters(X, X[None], X[None], torch.zeros(2, dtype=torch.int32))
    z = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        ttq.ttq_moe(X, X, X, z, z, z, X, z, z, z, top_k=1, bits=4, group=32)
