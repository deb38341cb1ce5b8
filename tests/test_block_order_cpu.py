"""The order in which the kernel of prompts takes its blocks of 256 query rows, built
for the host: every block exactly once, none that is not there, the most keys first."""
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    import ctypes
    so = str(tmp_path_factory.mktemp("order") / "block_order.so")
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "online_activation_aware_ttq_amd", "csrc"),
                    os.path.join(ROOT, "tests", "block_order_host.cpp"), "-o", so], check=True)
    fn = ctypes.CDLL(so).block_order
    fn.restype = None
    p64 = np.ctypeslib.ndpointer(np.int64)
    fn.argtypes = [ctypes.c_int, p64, p64, p64, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                   np.ctypeslib.ndpointer(np.int32), p64]

    def call(tokens, lens, G, max_len):
        tokens, lens = np.array(tokens, np.int64), np.maximum(np.array(lens, np.int64), 0)
        rows, shift = tokens * G, lens - tokens
        tiles = int(tokens.sum()) * G // 256 + len(tokens)  # what a call launches
        lane, r0 = np.empty(tiles, np.int32), np.zeros(tiles, np.int64)
        fn(len(tokens), rows, shift, lens, G, max_len, tiles, lane, r0)
        return [(int(i), int(r)) for i, r in zip(lane, r0)], rows, shift, lens

    return call


def check(order, tokens, lens, G, max_len):
    got, rows, shift, held = order(tokens, lens, G, max_len)
    want = {(i, r) for i in range(len(rows)) for r in range(0, int(rows[i]), 256)}
    n = len(want)
    assert len(got) >= n
    assert len(set(got[:n])) == n and set(got[:n]) == want, (tokens, lens, G, max_len)
    assert all(i == -1 for i, _ in got[n:])
    # those of the most keys first: 256 x < keys <= 256 (x + 1) are alike, 0 among the
    # first of them, and what a bound hides
    cap = 256 << max(0, int(max_len) >> 8).bit_length()
    keys = [min(min(int(held[i]), int(shift[i]) + min(r + 255, int(rows[i]) - 1) // G + 1), cap) for i, r in got[:n]]
    most = [max(0, k) for k in keys]
    assert all(a + 256 >= b for a, b in zip(np.minimum.accumulate(most), most)), (tokens, lens, G, max_len)


@pytest.mark.parametrize("tokens,lens,G", [
    ([200, 0], [200, 4096], 4),            # a prompt beside a request that adds nothing
    ([0, 200], [4096, 200], 4),
    ([200, 0, 300], [200, 4096, 700], 4),
    ([0] * 63 + [900], [100000] * 63 + [900], 1),
    ([0, 0], [5, 300], 2),                 # no rows at all
    ([64], [64], 4), ([65], [65], 4), ([2047, 900, 1, 0], [2047, 5000, 1, 257], 4),
    ([300], [10], 3),                      # more rows than keys
    ([70, 70], [0, -5], 8),
])
def test_by_hand(order, tokens, lens, G):
    for max_len in (1, 255, 4096, 1 << 20, 2 ** 31 - 4097):
        check(order, tokens, lens, G, max_len)


def test_random_batches(order):
    rng = random.Random(0)
    for _ in range(3000):
        n = rng.choice((1, 2, 3, 8, 63, 64, rng.randint(1, 64)))
        G, big = rng.choice((1, 2, 3, 4, 8, 20)), rng.choice((40, 400, 3000))
        tokens = [rng.choice((0, 0, 1, rng.randint(0, big))) for _ in range(n)]
        lens = [rng.choice((0, t, rng.randint(0, 2 * big), t + rng.randint(0, 100000))) for t in tokens]
        check(order, tokens, lens, G, rng.choice((1, 64, 1000, 5000, 200000, 2 ** 31 - 4097)))
