"""Page tables built and released on the GPU (rpa_build_tables,
rpa_release_tables) against their definition in Python: every output equal."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def cuda(a, dt=np.int32):
    return torch.from_numpy(np.asarray(a, dtype=dt)).cuda()


def build_ref(new, prev, table, free, count, p, room):
    table, slots, cu = table.copy(), [], [0]
    for s in range(len(new)):
        for j in range(-(-prev[s] // p), -(-(prev[s] + new[s]) // p)):
            count -= 1
            table[s, j] = free[count]
        slots += [int(table[s, pos // p]) * p + pos % p for pos in range(prev[s], prev[s] + new[s])]
        cu.append(cu[-1] + new[s])
    return table, cu, [a + b for a, b in zip(new, prev)], slots + [-1] * (room - len(slots)), count


def state(new, prev, p, spare, seed):
    """A page table that holds the previous lengths, the stack and its height."""
    rng = np.random.default_rng(seed)
    held = [-(-x // p) for x in prev]
    need = [-(-(a + b) // p) for a, b in zip(prev, new)]
    pool = sum(held) + spare
    perm = rng.permutation(max(pool, 1))
    table = np.full((len(new), max([1] + need)), -1)
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = perm[at:at + n]
        at += n
    free = np.full(max(pool, 1), -7)
    free[:spare] = perm[at:at + spare]
    return table, free, spare


def need_of(new, prev, p):
    return sum(-(-(a + b) // p) - -(-b // p) for a, b in zip(new, prev))


BUILD = [
    # (new, prev, page_size, padding)
    ([1], [0], 16, 0), ([1], [15], 16, 0), ([1], [16], 16, 3), ([0], [0], 16, 2), ([0, 0, 5], [3, 0, 0], 1, 0),
    ([3, 0, 700, 1, 16], [0, 77, 5, 127, 128], 128, 40), ([1] * 513, [i % 300 for i in range(513)], 16, 0),
    ([i % 37 for i in range(2048)], [i % 50 for i in range(2048)], 32, 100),
    ([(i * 7) % 5 for i in range(5000)], [(i * 11) % 90 for i in range(5000)], 16, 1),
    ([40000], [70000], 64, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(BUILD)))
def test_build(case, in_place):
    new, prev, p, pad = BUILD[case]
    spare = need_of(new, prev, p) + case % 3
    table, free, count = state(new, prev, p, spare, case)
    room = sum(new) + pad
    want = build_ref(new, prev, table, free, count, p, room)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    t, f, c0, kv0 = cuda(table), cuda(free), cuda([count]), cuda(prev)
    kv, c1 = (kv0, c0) if in_place else (cuda([9] * len(new)), cuda([9]))
    cu, slots = cuda([9] * (len(new) + 1)), cuda([9] * room, np.int64)
    binding.rpa_build_tables(cuda(new), kv0, t, f, c0, cu, kv, slots, c1, p, ws)
    assert binding.rpa_get_device_error(ws) == 0
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert cu.cpu().tolist() == want[1] and kv.cpu().tolist() == want[2]
    assert slots.cpu().tolist() == want[3] and c1.item() == want[4]
    assert np.array_equal(f.cpu().numpy(), free)
    assert bool((ws == 0).all())            # the counter is back at zero
    if not in_place:
        assert kv0.cpu().tolist() == prev and c0.item() == count


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,p", [(1, 16), (3, 128), (700, 16), (3000, 32)])
def test_release(seqs, p, in_place):
    rng = np.random.default_rng(seqs)
    prev = rng.integers(0, 200, seqs).tolist()
    done = (rng.random(seqs) < 0.3).astype(int).tolist()
    done[0] = 3                               # any value but zero
    table, free, count = state([0] * seqs, prev, p, 5, seqs)
    want, h = free.copy(), count
    for s in range(seqs):
        if done[s]:
            n = -(-prev[s] // p)
            want[h:h + n] = table[s, :n]
            h += n
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    t, f, c0, kv0 = cuda(table), cuda(free), cuda([count]), cuda(prev)
    kv, c1 = (kv0, c0) if in_place else (cuda([9] * seqs), cuda([9]))
    binding.rpa_release_tables(cuda(done), kv0, t, f, c0, kv, c1, p, ws)
    assert binding.rpa_get_device_error(ws) == 0
    assert np.array_equal(f.cpu().numpy(), want) and c1.item() == h
    assert kv.cpu().tolist() == [0 if d else x for d, x in zip(done, prev)]
    assert np.array_equal(t.cpu().numpy(), table) and bool((ws == 0).all())


def test_no_requests():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    table = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    cu, slots, c1 = cuda([9]), cuda([9] * 3, np.int64), cuda([9])
    e = cuda([])
    binding.rpa_build_tables(e, e, table, cuda([1, 2]), cuda([2]), cu, e, slots, c1, 16, ws)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and c1.item() == 2
    binding.rpa_release_tables(e, e, table, cuda([1, 2]), cuda([2]), e, c1, 16, ws)
    assert c1.item() == 2 and binding.rpa_get_device_error(ws) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["stack", "room", "negative", "width", "height"])
def test_a_step_that_does_not_fit_changes_nothing(what, in_place):
    new, prev, p = [20, 3, 40], [10, 16, 0], 16
    table, free, count = state(new, prev, p, need_of(new, prev, p) - (what == "stack"), 1)
    room = sum(new) - (what == "room")
    if what == "negative":
        new = [20, -1, 40]
    if what == "height":
        count = len(free) + 1
    if what == "width":
        table = table[:, :2].copy()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    t, c0, kv0 = cuda(table), cuda([count]), cuda(prev)
    kv, c1 = (kv0, c0) if in_place else (cuda([9] * 3), cuda([9]))
    cu, slots = cuda([9] * 4), cuda([9] * room, np.int64)
    binding.rpa_build_tables(cuda(new), kv0, t, cuda(free), c0, cu, kv, slots, c1, p, ws)
    want = binding.RPA_DEVERR_PAGES if what in ("stack", "height") else binding.RPA_DEVERR_LENGTHS
    assert binding.rpa_get_device_error(ws) == want
    assert np.array_equal(t.cpu().numpy(), table) and c1.item() == count
    assert kv.tolist() == prev and cu.tolist() == [0] * 4 and slots.tolist() == [-1] * room


def test_a_release_that_does_not_fit_changes_nothing():
    prev, p = [40, 20], 16
    table, free, _ = state([0, 0], prev, p, 2, 3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for count, lens, want in ((4, prev, binding.RPA_DEVERR_PAGES), (-1, prev, binding.RPA_DEVERR_PAGES),
                              (0, [-5, 20], binding.RPA_DEVERR_LENGTHS), (0, [60, 20], binding.RPA_DEVERR_LENGTHS)):
        f, kv, c1 = cuda(free), cuda([9, 9]), cuda([9])
        binding.rpa_release_tables(cuda([1, 1]), cuda(lens), cuda(table), f, cuda([count]), kv, c1, p, ws)
        assert binding.rpa_get_device_error(ws) == want
        assert np.array_equal(f.cpu().numpy(), free) and kv.tolist() == lens and c1.item() == count


def test_bad_page_ids():
    """An id outside the pool, in a row or in the stack, is never followed."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    table, free = cuda([[99, -1], [1, -1]]), cuda([0, 2, -3, 3])
    cu, kv, slots, c1 = cuda([9] * 3), cuda([9] * 2), cuda([9] * 4, np.int64), cuda([9])
    binding.rpa_build_tables(cuda([1, 3]), cuda([5, 15]), table, free, cuda([3]), cu, kv, slots, c1, 16, ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
    assert slots.tolist() == [-1, 31, -1, -1] and table.tolist() == [[99, -1], [1, -1]]
    f, kv = cuda([0, 9, 9, 9]), cuda([9] * 2)
    binding.rpa_release_tables(cuda([1, 1]), cuda([5, 5]), table, f, cuda([1]), kv, c1, 16, ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
    assert f.tolist() == [0, -1, 1, 9] and c1.item() == 3


def test_a_captured_decode_step_advances_in_place():
    """One captured build with in-place lengths and stack, replayed: each
    replay is the next step; then the stack runs dry and the steps stop."""
    p, seqs, pool = 16, 600, 700
    rng = np.random.default_rng(4)
    prev = rng.integers(1, 16, seqs).tolist()
    table, free, count = state([40] * seqs, prev, p, pool - seqs, 4)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    new, kv, c, t, f = cuda([1] * seqs), cuda(prev), cuda([count]), cuda(table), cuda(free)
    cu, slots = cuda([0] * (seqs + 1)), cuda([0] * 1100, np.int64)   # three CTAs
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.rpa_build_tables(new, kv, t, f, c, cu, kv, slots, c, p, ws)
    assert kv.tolist() == prev                                        # captured, not run
    for step in range(20):
        fits = need_of([1] * seqs, prev, p) <= count
        if fits:
            table, want_cu, prev, want_slots, count = build_ref([1] * seqs, prev, table, free, count, p, 1100)
        g.replay()
        assert binding.rpa_get_device_error(ws) == (0 if fits else binding.RPA_DEVERR_PAGES)
        assert kv.tolist() == prev and c.item() == count
        assert np.array_equal(t.cpu().numpy(), table)
        assert slots.tolist() == (want_slots if fits else [-1] * 1100)
    assert not fits
