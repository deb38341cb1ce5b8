"""ttq_cache_extend on the GPU against the oracle, which takes one sequence and one
page after another: whole numbers, all equal."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

NAMES = ("lens_out", "free_count_out", "offsets", "positions", "slots")


def _dev(v):
    import torch
    return torch.from_numpy(np.asarray(v, np.int32)).cuda()


def _run(lens, added, pages, free, count, page, T, **kw):
    import torch
    import online_activation_aware_ttq_amd as ttq
    pd, fd = _dev(pages), _dev(free)
    out = ttq.ttq_cache_extend(_dev(lens), _dev(added), pd, fd, _dev([count]), page_tokens=page,
                               T=T, **kw)
    torch.cuda.synchronize()
    got = {n: t.cpu().numpy() for n, t in zip(NAMES, out)}
    return got, pd.cpu().numpy(), fd.cpu().numpy()


def _check(lens, added, pages, free, count, page, T):
    got, p, f = _run(lens, added, pages, free, count, page, T)
    ref = oracle.cache_extend(lens, added, pages, free, count, page, T)
    for n in NAMES:
        np.testing.assert_array_equal(got[n].reshape(-1), np.atleast_1d(ref[n]), err_msg=n)
    np.testing.assert_array_equal(p, ref["pages"])
    np.testing.assert_array_equal(f, ref["free_pages"])
    return ref


def _state(rng, S, P, page, most, spare):
    """Sequences of 0 .. most rows with pages of their own, and a stack of the rest."""
    lens = rng.integers(0, most + 1, S)
    held = np.minimum(-(-lens // page), P)
    n = int(held.sum()) + spare
    order = rng.permutation(n).astype(np.int32)
    pages = np.full((S, P), -7, np.int32)
    at = 0
    for i in range(S):
        pages[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    free = np.full(n, -9, np.int32)
    free[:spare] = order[at:]
    return lens, pages, free


@pytest.mark.parametrize("S,page,most,new,spare,T", [
    (1, 16, 0, 1, 1, 1),            # the first row of one request
    (1, 1, 5, 3, 3, 4),             # a row a page
    (8, 16, 200, 1, 8, 8),          # a decode step
    (64, 8, 40, 9, 30, 400),        # too few pages for all
    (65, 8, 40, 9, 200, 200),       # too few rows for all
    (300, 4, 30, 3, 100, 700),
    (1000, 32, 100, 2, 700, 2000),
    (1024, 16, 100, 40, 3000, 4096),
    (1025, 16, 20, 1, 100, 1100),   # a second chunk of sequences
    (3000, 2, 9, 4, 5000, 4097),    # rows dealt to many workgroups
    (70, 64, 3000, 900, 900, 65536),
])
def test_steps(S, page, most, new, spare, T):
    print(f"[case] extend S={S} page={page} T={T}", flush=True)
    rng = np.random.default_rng(S + T)
    P = -(-(most + new) // page)
    for step in range(3):
        lens, pages, free = _state(rng, S, P, page, most, spare)
        added = rng.integers(0, new + 1, S)
        if step:
            added[rng.random(S) < 0.2] = -1
        if step == 2:  # some were refused before, some ask for more than a table holds
            again = rng.random(S) < 0.3
            lens = np.where(again, -1 - lens, lens)
            added = np.where(rng.random(S) < 0.1, added + P * page, added)
        _check(lens, added, pages, free, spare, page, T)


def test_pages_of_ended_sequences_come_back():
    """One gives, another takes in the same call; a stack that is full keeps its own."""
    pages = np.array([[3, 1, -1], [0, -1, -1]], np.int32)
    free = np.array([2, 4, -1, -1, -1], np.int32)
    ref = _check([20, 16], [-1, 17], pages, free, 2, 16, 20)
    assert ref["pages"][1].tolist() == [0, 1, 3] and ref["free_count_out"] == 2
    full = np.array([7, 8], np.int32)
    ref = _check([20, 16], [-1, 1], pages, full, 2, 16, 20)
    assert ref["free_count_out"] == 1 and ref["pages"][1].tolist() == [0, 8, -1]
    # counts outside the stack are taken to its ends
    assert _check([0, 0], [1, 1], pages, free, -5, 16, 2)["lens_out"].tolist() == [-1, -1]
    _check([0, 0], [1, 1], pages, full, 99, 16, 2)


def test_nothing():
    import torch
    import online_activation_aware_ttq_amd as ttq
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    lens, count, off, pos, slots = ttq.ttq_cache_extend(z(0), z(0), z(0, 4), z(3), z(1) + 2,
                                                        page_tokens=16, T=5)
    assert int(count) == 2 and off.tolist() == [0] and pos.tolist() == [0] * 5
    assert slots.tolist() == [-1] * 5
    ref = _check([5, 0], [0, 0], np.full((2, 1), 3, np.int32), np.zeros(0, np.int32), 0, 16, 0)
    assert ref["lens_out"].tolist() == [5, 0]


def test_in_place_over_steps_and_captured():
    """A decode loop that updates its lengths and stack in place, as a graph."""
    import torch
    import online_activation_aware_ttq_amd as ttq
    rng = np.random.default_rng(5)
    S, page, P, T = 9, 4, 6, 12
    lens_h, pages_h, free_h = _state(rng, S, P, page, 6, 20)
    lens, pages, free, count = _dev(lens_h), _dev(pages_h), _dev(free_h), _dev([20])
    added = torch.ones(S, dtype=torch.int32, device="cuda")
    off, pos = _dev(np.zeros(S + 1)), _dev(np.zeros(T))
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")

    def step():
        ttq.ttq_cache_extend(lens, added, pages, free, count, page_tokens=page, lens_out=lens,
                             free_count_out=count, offsets=off, positions=pos, slots=slots)

    keep = [t.clone() for t in (lens, pages, free, count)]
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t, k in zip((lens, pages, free, count), keep):
        t.copy_(k)
    c = 20
    for k in range(9):
        a = rng.integers(-1, 3, S)
        added.copy_(_dev(a))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle.cache_extend(lens_h, a, pages_h, free_h, c, page, T)
        for n, t in zip(NAMES, (lens, count, off, pos, slots)):
            np.testing.assert_array_equal(t.cpu().numpy().reshape(-1), np.atleast_1d(ref[n]), err_msg=n)
        lens_h, pages_h, free_h, c = (ref[n] for n in ("lens_out", "pages", "free_pages", "free_count_out"))
        np.testing.assert_array_equal(pages.cpu().numpy(), pages_h)
        assert (np.sort(np.concatenate([free_h[:c]] + [pages_h[i, :-(-(n if n >= 0 else -1 - n) // page)]
                                                       for i, n in enumerate(lens_h)]))
                == np.sort(np.unique(np.concatenate([keep[2][:20].cpu().numpy()] + [
                    keep[1][i, :-(-int(n) // page)].cpu().numpy() for i, n in enumerate(keep[0])])))).all()
