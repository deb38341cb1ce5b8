"""How far the cache's quantizer is from the weights': a scale is the range times
the float32 nearest to 1/N there and the range divided by N here, so codes can
differ where a value lies next to the border of two levels, and nowhere else."""
import numpy as np
import pytest

import oracle

CASES = [("asym", 4, 128), ("asym", 2, 64), ("asym", 8, 32), ("sym", 4, 64), ("intzp", 4, 128),
         ("intzp", 8, 32), ("fp8", 8, 32)]


@pytest.mark.parametrize("with_d", [False, True])
@pytest.mark.parametrize("fmt,bits,group", CASES)
def test_codes_differ_next_to_a_border_alone(fmt, bits, group, with_d):
    rng = np.random.default_rng(bits * 100 + group)
    rows, d = 500, 1024
    x = rng.standard_normal((rows, d)).astype(np.float32)
    x = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)  # bfloat16 values
    dh = (0.5 + rng.random(d)).astype(np.float32) if with_d else np.ones(d, np.float32)
    a = oracle.cache_rows(x, dh, bits, group, fmt)
    b = oracle.quantize_format(x, dh, bits, group, fmt)
    wide = lambda v: np.repeat(v.astype(np.float64), group, axis=1)
    sa, sb = wide(a["s"]), wide(b["s"])
    # the reciprocal and the product are each off by half a unit, the quotient by one
    assert (np.abs(sa / sb - 1) <= 3 * 2.0 ** -24 * 1.001).all()
    if fmt == "fp8":
        la, lb = oracle.e4m3_decode(a["codes"]), oracle.e4m3_decode(b["codes"])
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.maximum(np.abs(la), np.abs(lb)), 2.0 ** -6))) - 3)
    else:
        # levels u / s: the codes with the integer part of the offset (Z or the zero point)
        z = 0.0 if fmt == "asym" else 1.0
        off = oracle.format_offsets(b["s"], bits, fmt, b.get("m"), b.get("z"))
        la = a["codes"] + z * np.rint(wide(a["off"]) / sa)
        lb = b["codes"] + z * np.rint(wide(off) / sb)
        step = 1.0
    differ = la != lb
    assert (np.abs(la - lb) <= step).all()
    # where they do, both are half a step from the value, but for the roundings: three
    # of half a unit to a level (difference, reciprocal, product) and three between the scales
    off = wide(a["off"]) if fmt == "asym" else 0.0
    t = ((x * dh).astype(np.float64) - off) / sa
    half = np.maximum(np.abs(t - la), np.abs(t - lb)) - step / 2
    assert (half[differ] <= 6.01 * 2.0 ** -24 * np.maximum(np.abs(t), 1.0)[differ]).all()
    share, rows_hit = differ.mean(), differ.any(axis=1).mean()
    moved = (a["codes"] != b["codes"]).mean()
    print(f"{fmt} {bits} bits, groups of {group}, D {with_d}: {moved:.2e} of codes, {share:.2e} of levels, "
          f"{rows_hit:.2f} of rows, {(a['s'] != b['s']).mean():.2f} of scales")
    assert share <= 0.01 and moved <= 0.02
