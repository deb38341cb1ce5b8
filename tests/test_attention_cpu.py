"""Refusals of ttq_cache_extend, ttq_cache_rope and ttq_cache_attention: every
invalid call is answered on the host, before anything is enqueued (no GPU); and
the oracle of the three against hand-worked values."""
import ctypes

import numpy as np
import pytest

import online_activation_aware_ttq_amd as ttq
import oracle

FAKE = 0x7f0000000000  # 256-byte aligned, never dereferenced by validation
OTHER = FAKE + (1 << 32)


def lib():
    return ttq.load_library()


def heads(**kw):
    base = dict(d=512, n_slots=64, k_first=0, v_first=256, heads=4, kv_heads=2, head_dim=128,
                bits=4, group=128, qformat=0)
    base.update(kw)
    return ttq.ttq_heads(*[base[n] for n, _ in ttq.ttq_heads._fields_])


def ref(h):
    return ctypes.byref(h) if h is not None else None


# ------------------------------------------------------------------ extend
EXTEND = ("lens", "added", "pages", "free_pages", "free_count", "lens_out", "free_count_out",
          "offsets", "positions", "slots")


def extend(n_seq=3, T=8, max_pages=4, n_pages=12, page=16, **kw):
    v = dict.fromkeys(EXTEND, FAKE)
    v.update(kw)
    return lib().ttq_cache_extend(n_seq, T, max_pages, n_pages, page, *[v[n] for n in EXTEND], None)


def test_extend_arguments():
    for kw in (dict(n_seq=-1), dict(n_seq=65536), dict(T=-1), dict(T=(1 << 22) + 1),
               dict(max_pages=-1), dict(n_pages=-1), dict(n_pages=1 << 31), dict(page=0)):
        assert extend(**kw) == ttq.TTQ_EINVAL, kw
    assert extend(page=24) == ttq.TTQ_EUNSUPPORTED
    assert extend(page=8192) == ttq.TTQ_EUNSUPPORTED
    for name in EXTEND:
        assert extend(**{name: None}) == ttq.TTQ_ENULL, name
        assert extend(**{name: FAKE + 2}) == ttq.TTQ_EALIGN, name
    assert extend(slots=FAKE + 4) == ttq.TTQ_EALIGN


# -------------------------------------------------------------------- rope
def rope(h, T=5, x_type=1, Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, wq=None, wk=None,
         eps=1e-6, freq=FAKE, rot=128, flags=0, positions=FAKE, out=FAKE, slots=FAKE, kdh=None,
         vdh=None, kc=FAKE, ks=FAKE, km=FAKE, vc=FAKE, vs=FAKE, vm=FAKE):
    return lib().ttq_cache_rope(ref(h), T, x_type, Q, ldq, K, ldk, V, ldv, wq, wk, eps, freq, rot,
                                flags, positions, out, slots, kdh, vdh, kc, ks, km, vc, vs, vm, None)


HEADS = [
    (dict(bits=0), ttq.TTQ_EINVAL), (dict(bits=9), ttq.TTQ_EINVAL), (dict(group=0), ttq.TTQ_EINVAL),
    (dict(qformat=4), ttq.TTQ_EINVAL), (dict(qformat=3), ttq.TTQ_EINVAL),
    (dict(group=16), ttq.TTQ_EUNSUPPORTED), (dict(n_slots=-1), ttq.TTQ_EINVAL),
    (dict(kv_heads=0), ttq.TTQ_EINVAL), (dict(heads=5), ttq.TTQ_EINVAL),
    (dict(heads=-2), ttq.TTQ_EINVAL), (dict(heads=70000, kv_heads=1), ttq.TTQ_EINVAL),
    (dict(head_dim=0), ttq.TTQ_EINVAL), (dict(head_dim=96), ttq.TTQ_EUNSUPPORTED),
    (dict(kv_heads=8, heads=8), ttq.TTQ_EINVAL),             # wider than a row
    (dict(k_first=-128), ttq.TTQ_EINVAL), (dict(k_first=384), ttq.TTQ_EINVAL),
    (dict(v_first=320), ttq.TTQ_EINVAL),                      # past the row's end
    (dict(k_first=64, v_first=256), ttq.TTQ_EINVAL),          # inside a group
    (dict(head_dim=64, kv_heads=1, heads=1, v_first=128), ttq.TTQ_EINVAL),  # half a group
]


@pytest.mark.parametrize("kw,status", HEADS)
def test_heads(kw, status):
    out = ctypes.c_size_t(7)
    assert rope(heads(**kw)) == status
    assert attention(heads(**kw)) == status
    assert lib().ttq_cache_attention_workspace_bytes(ref(heads(**kw)), 5, 2, 4, 16, 0,
                                                     ctypes.byref(out)) == status
    assert out.value == 7


def test_rope_arguments():
    h = heads()
    assert rope(None) == ttq.TTQ_ENULL
    for name in ("Q", "K", "V", "freq", "positions", "out", "slots", "kc", "ks", "km", "vc", "vs", "vm"):
        if name != "kc" and name != "vc":
            assert rope(h, **{name: None}) == ttq.TTQ_ENULL, name
        assert rope(h, **{name: FAKE + 2}) == ttq.TTQ_EALIGN, name
    assert rope(h, kc=None, vc=OTHER) == ttq.TTQ_ENULL
    assert rope(h, kc=OTHER, vc=None) == ttq.TTQ_ENULL
    for name in ("Q", "K", "V", "wq", "wk", "freq", "out", "kdh", "vdh", "kc", "vc"):
        assert rope(h, **{name: FAKE + 8}) == ttq.TTQ_EALIGN, name
    for kw in (dict(T=-1), dict(T=(1 << 22) + 1), dict(x_type=2), dict(flags=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(rot=-16), dict(rot=144),
               dict(rot=15), dict(ldq=511), dict(ldk=128), dict(ldv=0), dict(ldq=1 << 40)):
        assert rope(h, **kw) == ttq.TTQ_EINVAL, kw
    assert rope(h, rot=24) == ttq.TTQ_EUNSUPPORTED
    assert rope(h, ldk=258) == ttq.TTQ_EALIGN
    assert rope(h, x_type=0, ldv=260) == ttq.TTQ_EALIGN
    # K and V of one cache on the same channels; in two caches they may be
    assert rope(heads(v_first=128)) == ttq.TTQ_EINVAL
    assert rope(heads(v_first=0)) == ttq.TTQ_EINVAL


def test_rope_nothing_to_do():
    nul = dict(Q=None, K=None, V=None, freq=None, positions=None, out=None, slots=None, kc=None,
               ks=None, km=None, vc=None, vs=None, vm=None)
    assert rope(heads(), T=0, ldq=0, ldk=0, ldv=0, **nul) == ttq.TTQ_OK


# --------------------------------------------------------------- attention
def attention(h, T=5, n_seq=2, max_pages=4, page=16, max_len=0, window=0, scale=0.1, Q=FAKE,
              ldq=512, offsets=FAKE, pages=FAKE, lens=FAKE, kc=FAKE, ks=FAKE, km=FAKE, vc=FAKE,
              vs=FAKE, vm=FAKE, kdhi=None, vdhi=None, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib().ttq_cache_attention(ref(h), T, n_seq, max_pages, page, max_len, window, scale, Q,
                                     ldq, offsets, pages, lens, kc, ks, km, vc, vs, vm, kdhi, vdhi,
                                     out, ws, ws_bytes, None)


def need(h, T, n_seq, max_pages=4, page=16, max_len=0):
    return ttq.ttq_cache_attention_workspace_bytes(h, T, n_seq, max_pages, page, max_len)


def test_attention_arguments():
    h = heads()
    assert attention(None) == ttq.TTQ_ENULL
    for name in ("Q", "pages", "lens", "kc", "ks", "km", "vc", "vs", "vm", "out"):
        assert attention(h, **{name: None}) == ttq.TTQ_ENULL, name
        assert attention(h, **{name: FAKE + 2}) == ttq.TTQ_EALIGN, name
    for name in ("Q", "kc", "vc", "kdhi", "vdhi", "out", "ws"):
        assert attention(h, **{name: FAKE + 8}) == ttq.TTQ_EALIGN, name
    assert attention(h, offsets=FAKE + 2) == ttq.TTQ_EALIGN
    for kw in (dict(T=-1), dict(T=1 << 23), dict(n_seq=-1), dict(n_seq=65536), dict(max_pages=-1),
               dict(page=0), dict(max_len=-1), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(ldq=511), dict(ldq=1 << 40), dict(offsets=None)):
        assert attention(h, **kw) == ttq.TTQ_EINVAL, kw
    assert attention(h, page=24) == ttq.TTQ_EUNSUPPORTED
    assert attention(h, ldq=516) == ttq.TTQ_EALIGN
    assert attention(heads(heads=0)) == ttq.TTQ_EINVAL
    assert attention(heads(bits=2)) == ttq.TTQ_EUNSUPPORTED
    assert attention(heads(bits=1)) == ttq.TTQ_EUNSUPPORTED
    assert attention(heads(n_slots=1 << 31)) == ttq.TTQ_EUNSUPPORTED
    assert attention(heads(heads=32768, kv_heads=2), T=1 << 16, ldq=1 << 23) == ttq.TTQ_EINVAL


def test_attention_workspace():
    h = heads()
    few = need(h, 2, 2, max_pages=64)  # few rows, long contexts: ranges of keys
    assert few > 0
    assert attention(h, T=2, max_pages=64, ws_bytes=few - 1) == ttq.TTQ_EWORKSPACE
    assert attention(h, T=2, max_pages=64, ws=None) == ttq.TTQ_ENULL
    # a shorter bound on the lengths needs less; one key of four heads, a wave's each, nothing
    assert need(h, 2, 2, max_pages=64, max_len=256) < few
    assert need(heads(d=1024, v_first=512, kv_heads=4), 2, 2, max_pages=64, max_len=1) == 0
    # many rows fill the chip by themselves
    assert need(h, 1 << 20, 2, max_pages=64) == 0
    for T, n in ((0, 0), (1, 1), (65535, 65535), (1 << 20, 1), (7, 0)):
        need(h, T, n, max_pages=1 << 22, page=4096)
    assert lib().ttq_cache_attention_workspace_bytes(ref(h), 2, 2, 4, 16, 0, None) == ttq.TTQ_ENULL


def test_attention_nothing_to_do():
    nul = dict(Q=None, pages=None, lens=None, out=None, kc=None, ws=None, ldq=0)
    assert attention(heads(), T=0, **nul) == ttq.TTQ_OK
    nul["ldq"] = 512
    assert attention(heads(), n_seq=0, **nul) == ttq.TTQ_OK


def test_injected_hip_error_is_reported(monkeypatch):
    monkeypatch.setenv("TTQ_INJECT_HIP_ERROR", "1")
    assert extend() == ttq.TTQ_EHIP
    assert rope(heads()) == ttq.TTQ_EHIP
    assert attention(heads()) == ttq.TTQ_EHIP


def test_struct_matches_header_layout():
    assert ctypes.sizeof(ttq.ttq_heads) == 4 * 8 + 6 * 4


def test_binding_checks_tensors():
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    z = torch.zeros(8, 2)
    c = torch.zeros(8, 128, dtype=torch.uint8)
    X = torch.zeros(2, 128)
    with pytest.raises(ValueError, match="GPU tensor"):
        ttq.ttq_cache_extend(i, i, i[None], i, i[:1], page_tokens=16, T=2)
    with pytest.raises(ValueError, match="GPU tensor"):
        ttq.ttq_cache_rope(X, X, X, i, i.long(), c, z, z, head_dim=128, bits=4, group=128)
    with pytest.raises(ValueError, match="GPU tensor"):
        ttq.ttq_cache_attention(X.view(2, 1, 128).bfloat16(), i[None], i[:1], c, z, z, kv_heads=1,
                                bits=4, group=128, page_tokens=16)


# ------------------------------------------------------------------ oracle
def test_oracle_extend_by_hand():
    """Pages of 4 rows; the stack (top last) is 9 8 7; sequence 1 ends and gives
    back 5, which is taken first; sequence 3 finds too few pages, so sequence 4,
    which needs one, gets none; sequence 5 needs none."""
    pages = np.array([[1, -1, -1], [5, 6, -1], [-1, -1, -1], [2, -1, -1], [3, -1, -1], [4, -1, -1]])
    r = oracle.cache_extend([3, 3, 0, 4, 4, 1], [2, -1, 5, 5, 1, 3], pages,
                            np.array([9, 8, 7, 0, 0, 0]), 3, 4, 20)
    assert r["lens_out"].tolist() == [5, 0, 5, -5, -5, 4]
    assert r["free_count_out"] == 1
    assert r["offsets"].tolist() == [0, 2, 2, 7, 12, 13, 16]
    assert r["pages"][0].tolist() == [1, 5, -1] and r["pages"][2].tolist() == [7, 8, -1]
    assert r["slots"][:7].tolist() == [7, 20, 28, 29, 30, 31, 32]
    assert (r["slots"][7:13] == -1).all() and r["slots"][13:16].tolist() == [17, 18, 19]
    assert (r["slots"][16:] == -1).all()
    assert r["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, 4, 5, 6, 7, 8, 4, 1, 2, 3, 0, 0, 0, 0]


def test_oracle_rope_keeps_lengths_and_angles():
    """A rotation keeps each pair's length, and a product of a query and a key
    depends on the distance of their positions alone."""
    rng = np.random.default_rng(0)
    f = (10.0 ** -np.arange(4)).astype(np.float32)
    x = rng.standard_normal((2, 1, 8)).astype(np.float32)
    for inter in (False, True):
        a = oracle.rope_heads(x, None, 0.0, f, [5, 9], inter).astype(np.float64)
        b = oracle.rope_heads(x, None, 0.0, f, [105, 109], inter).astype(np.float64)
        assert np.abs((a[0] * a[1]).sum() - (b[0] * b[1]).sum()) < 1e-5
        assert np.abs(np.linalg.norm(a) - np.linalg.norm(x)) < 1e-5
    n = oracle.rope_heads(x, np.ones(8), 0.0, None, None)
    assert np.abs((n.astype(np.float64) ** 2).mean(-1) - 1).max() < 1e-6


def test_oracle_attention_by_hand():
    K = np.zeros((3, 1, 2))
    V = np.arange(6.0).reshape(3, 1, 2)
    Q = np.ones((2, 2, 2))
    out = oracle.cache_attention(Q, K, V, [1, 2], 1.0)
    np.testing.assert_allclose(out[0, 1], V[:2, 0].mean(0))
    np.testing.assert_allclose(out[1, 0], V[:, 0].mean(0))
    np.testing.assert_allclose(oracle.cache_attention(Q, K, V, [1, 2], 1.0, 1)[1, 1], V[2, 0])
    assert (oracle.cache_attention(Q, K, V, [-1, -5], 1.0) == 0).all()
