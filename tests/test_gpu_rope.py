"""ttq_cache_rope on the GPU.  The definition fixes every float32 rounding of the
heads, so the codes, scales and offsets that it stores are the oracle's bit for bit,
and the queries are the oracle's float32 values rounded once to bfloat16."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


def _inv_freq(rot):
    return (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32) if rot else None


def _bf16_bits(x32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x32)).to(torch.bfloat16).view(torch.int16).numpy()


def _dev(v):
    import torch
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()


CASES = [
    # T, H, KV, hd, rot, inter, norm, x, bits, group, fmt, dhalf, two caches
    (1, 32, 8, 128, 128, False, True, "f32", 4, 128, "asym", False, False),
    (3, 4, 4, 64, 64, True, False, "bf16", 4, 64, "asym", True, False),
    (5, 3, 1, 256, 256, False, True, "f32", 8, 32, "fp8", False, True),
    (7, 10, 5, 64, 48, False, True, "bf16", 3, 32, "sym", True, False),
    (2, 8, 2, 128, 16, True, True, "f32", 4, 256, "intzp", False, False),
    (4, 8, 4, 64, 32, False, False, "f32", 2, 128, "asym", True, True),
    (6, 9, 9, 128, 0, False, True, "bf16", 1, 128, "asym", False, False),
    (130, 12, 4, 128, 128, False, True, "bf16", 4, 128, "asym", False, False),
    (2500, 2, 1, 64, 64, False, True, "f32", 4, 32, "asym", False, False),
    (9000, 1, 1, 128, 128, True, False, "bf16", 8, 64, "asym", False, False),
]


@pytest.mark.parametrize("T,H,KV,hd,rot,inter,norm,xt,bits,group,fmt,with_d,two", CASES)
def test_rope(T, H, KV, hd, rot, inter, norm, xt, bits, group, fmt, with_d, two):
    import torch
    import online_activation_aware_ttq_amd as ttq
    print(f"[case] rope T={T} H={H}/{KV} hd={hd} rot={rot} {xt} b{bits} g{group} {fmt}", flush=True)
    rng = np.random.default_rng(T * 7 + hd + H)
    qw, kw = H * hd, KV * hd
    x = rng.standard_normal((T, qw + 2 * kw)).astype(np.float32)
    x[:, rng.integers(0, qw + 2 * kw, 5)] *= 20
    if xt == "bf16":
        x = (np.ascontiguousarray(_bf16_bits(x)).view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    # a wider projection, whose columns Q, K and V are
    wide = torch.zeros(T, qw + 2 * kw + 64, dtype=torch.float32 if xt == "f32" else torch.bfloat16,
                       device="cuda")
    X = wide[:, 32:32 + qw + 2 * kw]
    X.copy_(torch.from_numpy(x))
    wq, wk = ((1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) for _ in range(2))
    if not norm:
        wq = wk = None
    positions = (rng.integers(0, 1 << 20) + np.arange(T)).astype(np.int32)
    positions[:2] = [0, 2 ** 31 - 1][:min(2, T)]
    first = group                                    # the row holds other channels too
    d = first + (kw if two else 2 * kw) + group
    d += -d % (128 * 8 // (group * 8) * group) if bits < 3 else 0
    dh, vdh = ((0.5 + rng.random(d)).astype(np.float32) if with_d else None for _ in range(2))
    n_slots = T + 5
    slots = rng.permutation(n_slots)[:T].astype(np.int64)
    if T > 2:
        slots[1] = -1
        slots[2] = n_slots
    rb = d * oracle.code_container_bits(bits) // 8

    def cache():
        return (torch.full((n_slots, rb), 0xAB, dtype=torch.uint8, device="cuda"),
                torch.full((n_slots, d // group), 7.0, device="cuda"),
                torch.full((n_slots, d // group), -7.0, device="cuda"))

    kc = cache()
    vc = cache() if two else kc
    out = ttq.ttq_cache_rope(
        X[:, :qw], X[:, qw:qw + kw], X[:, qw + kw:], _dev(positions), _dev(slots), *kc, head_dim=hd,
        bits=bits, group=group, inv_freq=_dev(_inv_freq(rot)), interleaved=inter, q_weight=_dev(wq),
        k_weight=_dev(wk), eps=1e-5, k_first=first, v_first=first if two else None,
        v_cache=vc if two else None, dhalf=_dev(dh), v_dhalf=_dev(vdh) if two else None, qformat=fmt)
    torch.cuda.synchronize()
    args = (1e-5, _inv_freq(rot), positions, inter)
    q = oracle.rope_heads(x[:, :qw].reshape(T, H, hd), wq, *args)
    k = oracle.rope_heads(x[:, qw:qw + kw].reshape(T, KV, hd), wk, *args).reshape(T, kw)
    v = x[:, qw + kw:]
    np.testing.assert_array_equal(out.cpu().view(torch.int16).numpy(), _bf16_bits(q))
    live = np.ones(T, bool)
    if T > 2:
        live[1:3] = False
    ones = np.ones(kw, np.float32)
    parts = [(kc, first, k, dh), (vc, first + (0 if two else kw), v, vdh if two else dh)]
    rest = {id(c): np.ones((n_slots, d), bool) for c in (kc, vc)}
    for c, at, rows, scale in parts:
        ref = oracle.cache_rows(rows, ones if scale is None else scale[at:at + kw], bits, group, fmt)
        b0, b1 = at * rb // d, (at + kw) * rb // d
        got = c[0].cpu().numpy()[slots[live], b0:b1]
        np.testing.assert_array_equal(got, oracle.pack_codes(ref["codes"], bits)[live])
        g = slice(at // group, (at + kw) // group)
        np.testing.assert_array_equal(c[1].cpu().numpy()[slots[live], g].view(np.uint32),
                                      ref["s"][live].view(np.uint32))
        np.testing.assert_array_equal(c[2].cpu().numpy()[slots[live], g], ref["off"][live])
        rest[id(c)][slots[live], at:at + kw] = False
    for c in (kc, vc):  # everything else as it was
        m = rest[id(c)]
        assert (c[0].cpu().numpy()[m[:, ::d // rb] if rb <= d else m] == 0xAB).all()
        assert (c[1].cpu().numpy()[m[:, ::group]] == 7).all()
        assert (c[2].cpu().numpy()[m[:, ::group]] == -7).all()


def test_equals_cache_write_of_the_rows():
    """Without norms and rotation: the bits of ttq_cache_write; Q None: no queries."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    g = torch.Generator(device="cuda").manual_seed(1)
    T, kw = 33, 512
    kv = torch.randn(T, 2 * kw, generator=g, device="cuda")
    slots = torch.randperm(40, generator=g, device="cuda")[:T].contiguous()
    make = lambda: (torch.zeros(40, kw, dtype=torch.uint8, device="cuda"),
                    torch.zeros(40, 2 * kw // 64, device="cuda"), torch.zeros(40, 2 * kw // 64, device="cuda"))
    a, b = make(), make()
    kws = dict(bits=4, group=64, qformat="intzp")
    ttq.ttq_cache_write(kv, slots, *a, **kws)
    r = ttq.ttq_cache_rope(None, kv[:, :kw], kv[:, kw:], None, slots, *b, head_dim=128, **kws)
    assert r is None
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_values_that_are_not_finite_stay_in_their_head():
    import torch
    import online_activation_aware_ttq_amd as ttq
    T, hd, KV = 4, 64, 2
    x = torch.randn(T, 4 * KV * hd // 2, device="cuda")
    x[1, 5] = float("nan")
    x[2, KV * hd + 70] = float("inf")
    w = torch.ones(hd, device="cuda")
    kw = KV * hd
    c = (torch.zeros(T, kw, dtype=torch.uint8, device="cuda"), torch.zeros(T, kw // 32, device="cuda"),
         torch.zeros(T, kw // 32, device="cuda"))
    xs = torch.cat((x[:, :kw], x), 1)
    q = ttq.ttq_cache_rope(xs[:, :kw], x[:, :kw], x[:, kw:], torch.arange(T, dtype=torch.int32, device="cuda"),
                           torch.arange(T, device="cuda"), *c, head_dim=hd, bits=4, group=64,
                           inv_freq=_dev(_inv_freq(hd)), q_weight=w, k_weight=w)
    bad = torch.isnan(q.float()).any(-1).cpu()
    assert bad.tolist() == [[False, False], [True, False], [False, False], [False, False]]
    s = torch.isnan(c[1]).cpu()
    want = torch.zeros_like(s)
    want[1, 0] = want[2, 3] = True
    assert torch.equal(s, want)


def test_captured_on_another_stream():
    import torch
    import online_activation_aware_ttq_amd as ttq
    T, H, KV, hd = 6, 4, 2, 128
    X = torch.zeros(T, (H + 2 * KV) * hd, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    c = (torch.zeros(16, KV * hd, dtype=torch.uint8, device="cuda"), torch.zeros(16, 4, device="cuda"),
         torch.zeros(16, 4, device="cuda"))
    out = torch.zeros(T, H, hd, dtype=torch.bfloat16, device="cuda")
    fr = _dev(_inv_freq(hd))

    def step(**kw):
        return ttq.ttq_cache_rope(X[:, :H * hd], X[:, H * hd:(H + KV) * hd], X[:, (H + KV) * hd:], pos,
                                  slots, *c, head_dim=hd, bits=4, group=128, inv_freq=fr, **kw)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(stream=side.cuda_stream, out=out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out=out)
    for k in range(4):
        X.normal_()
        pos.fill_(1000 * k)
        slots.copy_(torch.arange(T, device="cuda") + k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, *c)]
        eager = step(stream=side.cuda_stream)
        side.synchronize()
        for a, b in zip(got, (eager, *c)):
            assert torch.equal(a, b)
