"""The quantized cache on the GPU against the oracle's quantizer.

Stored codes, scales and offsets must equal the oracle's float32 decision bit
for bit.  What is read back is held to the float64 value of the stored terms,
(m + s q) D^{-1/2}: the kernel rounds it twice in float32 (one fused
multiply-add, one product), at most 2 * 2^-24 of the result (and 2^-149 for
each where it is subnormal); a bfloat16 result is rounded once more, 2^-8.
"""
import numpy as np
import pytest

import oracle
from parity_util import to_dev
from workloads.configs import draw_x

pytestmark = pytest.mark.gpu

REL = {"f32": 2 * 2.0 ** -24 * (1 + 2.0 ** -20), "bf16": 2.0 ** -8 + 2 * 2.0 ** -24 * (1 + 2.0 ** -6)}


def _rows(seed, T, d, f32):
    bits = draw_x(seed, 0, 1, T, d, "logu10_100", max(1, d // 100))[0]
    x = oracle.bf16_to_f32(bits)
    if f32:  # values with all 24 bits
        x = (x * np.float32(1.2345678)).astype(np.float32)
    return bits, x


def _cache(n_slots, d, bits, group, fill=0xAB):
    import torch
    rb = d * oracle.code_container_bits(bits) // 8
    return (torch.full((n_slots, rb), fill, dtype=torch.uint8, device="cuda"),
            torch.full((n_slots, d // group), 7.0, device="cuda"),
            torch.full((n_slots, d // group), -7.0, device="cuda"))


CASES = [
    # fmt, bits, group, d, T, page, x, out, with D
    ("asym", 4, 128, 1024, 33, 16, "bf16", "bf16", False),
    ("asym", 4, 128, 128, 1, 1, "bf16", "f32", True),
    ("asym", 2, 64, 192, 70, 64, "f32", "f32", True),
    ("asym", 3, 32, 544, 5, 2, "f32", "bf16", False),
    ("asym", 1, 256, 1280, 9, 8, "bf16", "f32", False),
    ("asym", 8, 32, 96, 17, 4, "bf16", "f32", True),
    ("sym", 4, 64, 576, 31, 16, "f32", "f32", False),
    ("sym", 2, 128, 640, 6, 4, "bf16", "bf16", True),
    ("intzp", 4, 128, 1152, 12, 16, "bf16", "f32", True),
    ("intzp", 7, 256, 768, 4, 1, "f32", "bf16", False),
    ("fp8", 8, 32, 160, 40, 32, "bf16", "bf16", False),
    ("fp8", 8, 256, 4352, 3, 4096, "f32", "f32", True),
]


@pytest.mark.parametrize("fmt,bits,group,d,T,page,xt,ot,with_d", CASES)
def test_write_and_read(fmt, bits, group, d, T, page, xt, ot, with_d):
    import torch
    import online_activation_aware_ttq_amd as ttq
    print(f"[case] cache {fmt} b{bits} g{group} d={d} T={T} page={page} {xt}->{ot}", flush=True)
    rng = np.random.default_rng(d * 31 + T)
    xb, x = _rows(60 + d, T, d, xt == "f32")
    dh = (0.3 + rng.random(d) * 3).astype(np.float32) if with_d else np.ones(d, np.float32)
    dhi = (np.float32(1) / dh).astype(np.float32)
    # three sequences; the first T rows go to sequence 1, whose pages are shuffled
    P = -(-T // page) + 1
    n_slots = 3 * P * page
    pages = rng.permutation(3 * P).reshape(3, P).astype(np.int32)
    pos = np.arange(T)
    slots = pages[1][pos // page].astype(np.int64) * page + pos % page
    skip = T // 2  # one row of padding in the middle
    slots_w = slots.copy()
    if T > 2:
        slots_w[skip] = -1
    codes, s, m = _cache(n_slots, d, bits, group)
    # X as a column range of a wider matrix
    wide = torch.zeros(T, d + 64, dtype=torch.float32 if xt == "f32" else torch.bfloat16, device="cuda")
    X = wide[:, 32:32 + d]
    X.copy_(torch.from_numpy(x).cuda() if xt == "f32" else to_dev(xb))
    ddev = torch.from_numpy(dh).cuda() if with_d else None
    kw = dict(bits=bits, group=group, qformat=fmt)
    ttq.ttq_cache_write(X, torch.from_numpy(slots_w).cuda(), codes, s, m, dhalf=ddev, **kw)
    torch.cuda.synchronize()
    ref = oracle.cache_rows(x, dh, bits, group, fmt)
    qc, qs, off, v = ref["codes"], ref["s"], ref["off"], ref["values"]
    live = np.ones(T, bool)
    if T > 2:
        live[skip] = False
    got = codes.cpu().numpy()
    np.testing.assert_array_equal(got[slots[live]], oracle.pack_codes(qc, bits)[live])
    np.testing.assert_array_equal(s.cpu().numpy()[slots[live]].view(np.uint32), qs[live].view(np.uint32))
    np.testing.assert_array_equal(m.cpu().numpy()[slots[live]], off[live])
    rest = np.ones(n_slots, bool)  # every other row as it was
    rest[slots[live]] = False
    assert (got[rest] == 0xAB).all()
    assert (s.cpu().numpy()[rest] == 7).all() and (m.cpu().numpy()[rest] == -7).all()
    if T > 2:  # the skipped row is written by a call of its own
        ttq.ttq_cache_write(X[skip:skip + 1], torch.from_numpy(slots[skip:skip + 1]).cuda(),
                            codes, s, m, dhalf=ddev, **kw)
    # read: sequence 0 empty, 1 all rows, 2 a negative length; room for more
    out = torch.full((3, T + 3, d), 5.0, dtype=torch.float32 if ot == "f32" else torch.bfloat16,
                     device="cuda")
    lens = torch.tensor([0, T, -4], dtype=torch.int32, device="cuda")
    r = ttq.ttq_cache_read(codes, s, m, torch.from_numpy(pages).cuda(), lens, page_tokens=page,
                           dhalf_inv=torch.from_numpy(dhi).cuda() if with_d else None, out=out, **kw)
    torch.cuda.synchronize()
    assert r is out
    o = out.double().cpu().numpy()
    assert (o[0] == 5).all() and (o[2] == 5).all() and (o[1, T:] == 5).all()
    ref = v * dhi.astype(np.float64)
    # the fused multiply-add is off by 2^-24 of m + s q, which is what is read
    assert (np.abs(o[1, :T] - ref) <= REL[ot] * np.abs(ref) + 2.0 ** -140).all()


def _small(T=4, d=64, bits=4, group=32, fmt="asym"):
    rng = np.random.default_rng(T + d)
    return rng.standard_normal((T, d)).astype(np.float32), _cache(8, d, bits, group)


def test_values_that_are_not_finite_stay_in_their_group():
    import torch
    import online_activation_aware_ttq_amd as ttq
    for fmt, bits in (("asym", 4), ("sym", 4), ("intzp", 3), ("fp8", 8)):
        x, (codes, s, m) = _small(T=5, bits=bits)
        x[0, 3] = np.nan
        x[1, 40] = np.inf
        x[2, 5] = -np.inf
        x[3, 32:34] = [3e38, -3e38]  # finite, but the range is not (asym, intzp)
        X = torch.from_numpy(x).cuda()
        ttq.ttq_cache_write(X, torch.arange(5, device="cuda"), codes, s, m, bits=bits, group=32,
                            qformat=fmt)
        out = ttq.ttq_cache_read(codes, s, m, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                 torch.tensor([5], dtype=torch.int32, device="cuda"), bits=bits,
                                 group=32, page_tokens=8, qformat=fmt, dtype=torch.float32)
        bad = torch.isnan(out[0, :5]).cpu().numpy().reshape(5, 2, 32)
        want = np.zeros((5, 2), bool)
        want[0, 0] = want[1, 1] = want[2, 0] = True
        want[3, 1] = fmt in ("asym", "intzp")
        assert (bad == want[:, :, None]).all(), fmt
        assert (out[0, 5:] == 0).all()


def test_constant_tiny_and_zero_groups():
    import torch
    import online_activation_aware_ttq_amd as ttq
    for fmt, bits in (("asym", 4), ("sym", 4), ("intzp", 4), ("fp8", 8)):
        x = np.zeros((4, 64), np.float32)
        x[1] = 0.75                                   # constant
        x[2, ::2] = 1e-38                             # a scale below 2^-126
        x[3] = np.linspace(-1, 1, 64, dtype=np.float32) * np.float32(1e-30)
        codes, s, m = _cache(8, 64, bits, 32)
        ttq.ttq_cache_write(torch.from_numpy(x).cuda(), torch.arange(4, device="cuda"), codes, s, m,
                            bits=bits, group=32, qformat=fmt)
        out = ttq.ttq_cache_read(codes, s, m, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                 torch.tensor([4], dtype=torch.int32, device="cuda"), bits=bits,
                                 group=32, page_tokens=8, qformat=fmt, dtype=torch.float32)
        o = out[0].double().cpu().numpy()
        assert (o[0] == 0).all()
        # half a step of the format: asym has none on a constant group
        step = {"asym": 0.0, "sym": 0.75 / 7, "intzp": 0.75 / 15, "fp8": 0.75 / 8}[fmt]
        assert np.abs(o[1] - 0.75).max() <= step / 2 + 2.0 ** -23
        assert np.abs(o[2] - x[2]).max() <= 1.1e-38
        assert np.abs(o[3] - x[3]).max() <= {"fp8": 1e-30 / 16}.get(fmt, 1e-30 / 7 / 2 * 1.001)


def test_pages_and_slots_outside_the_cache_touch_nothing():
    import torch
    import online_activation_aware_ttq_amd as ttq
    x, (codes, s, m) = _small(T=4)
    X = torch.from_numpy(x).cuda()
    before = [t.clone() for t in (codes, s, m)]
    slots = torch.tensor([-1, 8, 1 << 40, -(1 << 62)], device="cuda")
    ttq.ttq_cache_write(X, slots, codes, s, m, bits=4, group=32)
    for a, b in zip(before, (codes, s, m)):
        assert torch.equal(a, b)
    ttq.ttq_cache_write(X, torch.arange(4, device="cuda"), codes, s, m, bits=4, group=32)
    # pages of 4 rows, a cache of 8: pages 0 and 1 exist
    pages = torch.tensor([[2, -1, 1 << 30, 0], [0, 1, 0, 1]], dtype=torch.int32, device="cuda")
    out = torch.full((2, 20, 64), 5.0, device="cuda")
    ttq.ttq_cache_read(codes, s, m, pages, torch.tensor([99, 3], dtype=torch.int32, device="cuda"),
                       bits=4, group=32, page_tokens=4, out=out)
    o = out.cpu()
    assert (o[0, :12] == 5).all() and (o[0, 16:] == 5).all() and (o[1, 3:] == 5).all()
    assert torch.equal(o[0, 12:15], o[1, :3]) and not (o[1, :3] == 5).any()


def test_rows_past_2_to_31_bytes():
    """Byte offsets of a long cache pass 32 bits."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    d, group, n_slots = 8192, 256, (1 << 19) + 64  # 4 GiB of 8-bit codes
    codes = torch.zeros(n_slots, d, dtype=torch.uint8, device="cuda")
    s = torch.zeros(n_slots, d // group, device="cuda")
    m = torch.zeros_like(s)
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(3, d, device="cuda", generator=g)
    slots = torch.tensor([5, (1 << 18) + 3, n_slots - 1], device="cuda")
    ttq.ttq_cache_write(X, slots, codes, s, m, bits=8, group=group)
    pages = slots.to(torch.int32)[None].contiguous()
    out = ttq.ttq_cache_read(codes, s, m, pages, torch.tensor([3], dtype=torch.int32, device="cuda"),
                             bits=8, group=group, page_tokens=1, dtype=torch.float32)
    small = [t[:3].clone() for t in (codes, s, m)]
    ttq.ttq_cache_write(X, torch.arange(3, device="cuda"), *small, bits=8, group=group)
    assert torch.equal(codes[slots], small[0]) and torch.equal(s[slots], small[1])
    assert int((codes != 0).any(1).sum()) == 3
    step = (X.view(3, -1, group).amax(-1) - X.view(3, -1, group).amin(-1)) / 255
    err = (out[0] - X).abs().view(3, -1, group).amax(-1)
    assert (err <= step * 0.5001 + 1e-6).all()


@pytest.mark.parametrize("ot", ["bf16", "f32"])
def test_results_larger_than_the_last_level_cache(ot):
    """They are written past it by another kernel, which has to give the same."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    d, group, page, T = 4096, 128, 64, 18000
    dt = torch.bfloat16 if ot == "bf16" else torch.float32
    codes, s, m = _cache(640, d, 4, group)
    g = torch.Generator(device="cuda").manual_seed(7)
    X = torch.randn(640, d, device="cuda", generator=g)
    ttq.ttq_cache_write(X, torch.arange(640, device="cuda"), codes, s, m, bits=4, group=group)
    pages = torch.randint(0, 10, (2, 282), device="cuda", generator=g).to(torch.int32)
    lens = torch.tensor([301, 17998], dtype=torch.int32, device="cuda")
    kw = dict(bits=4, group=group, page_tokens=page)
    big = ttq.ttq_cache_read(codes, s, m, pages, lens,
                             out=torch.full((2, T, d), 3.0, dtype=dt, device="cuda"), **kw)
    assert big.numel() * big.element_size() > 256 << 20
    small = ttq.ttq_cache_read(codes, s, m, torch.arange(10, dtype=torch.int32, device="cuda")[None],
                               torch.tensor([640], dtype=torch.int32, device="cuda"), T=640, dtype=dt, **kw)
    for i, n in enumerate((301, 17998)):
        rows = (pages[i].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        assert torch.equal(big[i, :n], small[0][rows])
        assert (big[i, n:] == 3).all()


def test_captured_and_on_another_stream():
    import torch
    import online_activation_aware_ttq_amd as ttq
    d, T = 512, 6
    codes, s, m = _cache(32, d, 4, 128)
    X = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(T, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    pages = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    out = torch.zeros(1, 8, d, device="cuda")
    kw = dict(bits=4, group=128)

    def step():
        ttq.ttq_cache_write(X, slots, codes, s, m, **kw)
        ttq.ttq_cache_read(codes, s, m, pages, lens, page_tokens=16, out=out, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        X.copy_(torch.randn(T, d, device="cuda"))
        slots.copy_(torch.arange(T, device="cuda") + (k % 3))
        lens.fill_(T + k % 3)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        c2, s2, m2 = codes.clone(), s.clone(), m.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(codes, c2) and torch.equal(s, s2)
