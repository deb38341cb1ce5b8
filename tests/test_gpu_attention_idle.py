"""Attention of prompts beside requests that add nothing in the step but hold many keys
(ttq_cache_extend gives them no rows): first, in the middle and last of the batch."""
import pytest

pytestmark = pytest.mark.gpu

CASES = [
    # H, KV, hd, bits, group, fmt, page, lens, rows, window, D, two caches
    (4, 1, 64, 4, 64, "asym", 16, [200, 4096], [200, 0], 0, False, False),
    (4, 1, 64, 4, 64, "asym", 16, [4096, 200], [0, 200], 0, False, False),
    (4, 1, 128, 8, 64, "fp8", 32, [200, 4096, 700], [200, 0, 300], 0, True, False),
    (2, 1, 64, 4, 32, "sym", 16, [3000, 900, 300, 2000, 257], [0, 600, 0, 100, 0], 100, False, True),
    (1, 1, 64, 4, 64, "asym", 16, [900] + [300] * 5, [900] + [0] * 5, 0, False, False),
    # and where all are idle but one row of one request
    (64, 1, 64, 4, 64, "asym", 16, [700, 1000], [0, 2], 0, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])) + f"-{c[7]}of{c[8]}")
def test_against_float64(case):
    from test_gpu_attention import _run
    _run(case)
