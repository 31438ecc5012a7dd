"""Attention of drafted trees (rpa_forward_tree) against its definition in 64 bits:
head layouts, page sizes, trees and masks of every size, windows, empty rows, NaN in
places that a row does not see, lengths that differ from the plan's, streams and
graphs.  The bound adds up what is rounded (tree_reference.attention_bound)."""

from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build

from . import tree_reference as ref

pytestmark = pytest.mark.gpu

PATHS = [binding.RPA_PATH_AUTO, binding.RPA_PATH_SIMT]


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def cuda(a):
    a = a.view(np.int64) if isinstance(a, np.ndarray) and a.dtype == np.uint64 else a
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()


class Tree:
    """A batch on the GPU."""

    def __init__(self, b):
        self.b = b
        for n in ("q", "k_pages", "v_pages", "table", "cu", "kv", "mask", "pos"):
            setattr(self, n, cuda(getattr(b, n)))
        self.win = None if b.win is None else cuda(b.win)
        self.out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda")

    def plan(self, **kw):
        b = self.b
        dt = binding.RPA_DTYPE_BF16 if b.dtype == "bf16" else binding.RPA_DTYPE_F32
        return binding.rpa_plan(b.cu, b.kv, b.win, b.hq, b.hkv, b.d, b.page, b.table.shape[1], b.pool, dtype=dt,
                                tree_words=b.words, **kw)

    def args(self, plan, ws, out=None):
        return (self.q, self.k_pages, self.v_pages, self.table, self.cu, self.kv, self.mask,
                None if self.win is None else self.pos, self.win, self.b.scale, self.out if out is None else out, plan, ws)

    def run(self, error=0, **kw):
        plan = self.plan(**kw)
        ws = binding.alloc_workspace(plan)
        self.out.fill_(float("nan"))
        binding.rpa_forward_tree(*self.args(plan, ws))
        assert binding.rpa_get_device_error(ws) == error
        return self.out


def check(b, out, want=None):
    want = ref.attention(b) if want is None else want
    got = out.double().cpu()
    nan = torch.isnan(want[0])
    assert torch.equal(torch.isnan(got), nan), "%d NaN missing, %d too many" % (
        (nan & ~torch.isnan(got)).sum(), (torch.isnan(got) & ~nan).sum())
    inf = torch.isinf(want[0])
    assert torch.equal(got[inf], want[0][inf])
    off = torch.where(nan | inf, 0.0, (got - want[0]).abs())
    bound = torch.where(nan | inf, 0.0, torch.nan_to_num(ref.attention_bound(b, want), 0.0, 0.0, 0.0))
    assert (off <= bound).all(), "off by %.3g of the bound" % float((off / bound.clamp(min=1e-30)).max())


# (nodes, context, Hq, Hkv, D, page size, windows)
CASES = [
    ([1], [0], 4, 1, 64, 16, None),                                  # a single key
    ([6], [700], 4, 1, 64, 16, None),
    ([1, 2, 3], [127, 128, 129], 8, 1, 256, 128, None),
    ([8] * 5, [0, 1, 119, 120, 1000], 8, 1, 256, 128, None),
    ([5, 0, 7, 0], [300, 50, 0, 0], 6, 2, 128, 32, None),             # requests without nodes
    ([64, 63, 65], [64, 190, 1], 4, 4, 64, 64, None),                 # words of the mask
    ([128, 1, 129], [256, 4000, 77], 2, 1, 128, 16, None),
    ([300], [1000], 3, 1, 64, 256, None),                             # five words, three row tiles
    ([40, 33], [500, 2000], 7, 1, 128, 64, None),                     # 18 nodes of 7 heads a tile
    ([17, 20], [333, 901], 10, 2, 256, 16, None),                     # 25 nodes of 5 heads
    ([9, 2], [450, 3], 128, 1, 64, 32, None),                         # a node a tile
    ([3], [200], 130, 1, 64, 32, None),                               # more heads than a tile has rows
    ([4, 12], [100, 31], 16, 4, 128, 8, None),                        # small pages
    ([4, 12], [100, 31], 4, 2, 64, 1, None),
    ([12] * 6, [900, 64, 63, 500, 128, 2], 8, 2, 128, 16, [64, 64, 1, 0, 130, 3]),
    ([24] * 4, [256, 700, 1100, 2000], 8, 1, 256, 128, [1024, 0, 1, 200]),
    ([100, 30], [3000, 150], 8, 2, 64, 128, [7, 129]),
    ([1024], [513], 2, 1, 64, 128, None),                             # the largest mask
    ([16, 48, 30], [20000, 7777, 129], 32, 8, 128, 64, None),
    ([8] * 60, list(range(100, 2500, 40)), 8, 1, 256, 128, None),
]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_trees(case, path):
    nodes, ctx, hq, hkv, d, page, windows = CASES[case]
    b = ref.tree_batch(nodes, ctx, hq, hkv, d, page, windows, seed=case)
    check(b, Tree(b).run(path=path))


@pytest.mark.parametrize("sms", [1, 2, 5, 40])
@pytest.mark.parametrize("case", [3, 8, 14, 15])
def test_segments_cut_anywhere(case, sms):
    nodes, ctx, hq, hkv, d, page, windows = CASES[case]
    b = ref.tree_batch(nodes, ctx, hq, hkv, d, page, windows, seed=50 + case)
    check(b, Tree(b).run(num_sms=sms))


@pytest.mark.parametrize("case", [1, 4, 5, 11, 14])
def test_f32(case):
    nodes, ctx, hq, hkv, d, page, windows = CASES[case]
    b = ref.tree_batch(nodes, ctx, hq, hkv, d, page, windows, seed=100 + case, dtype="f32")
    check(b, Tree(b).run())


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_any_mask(d, path):
    """Masks that are no trees: later nodes seen, nodes that do not see themselves, rows that see nothing."""
    rng = np.random.default_rng(d)
    nodes, ctx = [70, 9, 1, 130], [0, 0, 0, 40]
    sees = [rng.random((t, t)) < 0.3 for t in nodes]
    sees[0][5] = sees[0][69] = sees[1][0] = False
    sees[2][:] = False
    b = ref.tree_batch(nodes, ctx, 6, 2, d, 16, None, seed=d, sees=sees)
    out = Tree(b).run(path=path)
    assert (out[[5, 69, 70, 79]] == 0).all()
    check(b, out)


@pytest.mark.parametrize("path", PATHS)
def test_a_window_can_leave_a_row_empty(path):
    sees = [np.eye(3, dtype=bool) & np.array([True, False, True])]
    b = ref.tree_batch([3], [200], 4, 2, 128, 16, [2], seed=1, sees=sees)
    b.pos[:] = [200, 202, 201]   # node 1 sees no context (202 - 199 > 1) and nothing of the tree
    out = Tree(b).run(path=path)
    assert (out[1] == 0).all() and (out[0] != 0).any()
    check(b, out)


@pytest.mark.parametrize("path", PATHS)
def test_bits_behind_the_nodes_mean_nothing(path):
    b = ref.tree_batch([5, 66], [130, 250], 4, 2, 128, 16, None, seed=2, words=3)
    t = Tree(b)
    t.mask[:5] |= ~31
    t.mask[5:, 1] |= ~3
    t.mask[5:, 2] = -1
    check(b, t.run(path=path))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale", [-0.125, 0.0, 0.5, 1e-30])
def test_scales(scale, path):
    b = ref.tree_batch([9, 20], [300, 0], 8, 2, 64, 16, [0, 40], seed=3, scale=scale)
    check(b, Tree(b).run(path=path))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_scores(d):
    """Scores far apart: the running maximum grows by steps of hundreds, and most weights underflow."""
    b = ref.tree_batch([20, 3], [1500, 700], 4, 1, d, 32, None, seed=4, scale=1.0)
    check(b, Tree(b).run())


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d,windows", [(64, None), (128, [50, 300]), (256, [0, 129])])
def test_slots_that_nobody_sees_may_hold_anything(d, windows, path):
    """NaN in every slot but those of keys that some node sees."""
    b = ref.tree_batch([10, 37], [260, 1000], 8, 2, d, 64, windows, seed=5)
    want = ref.attention(b)
    used = torch.zeros(b.k_pages.shape[:2], dtype=torch.bool)
    for s in range(2):
        for key in np.flatnonzero(ref.visible(b, s).any(0)):
            used[ref.slot(b, s, int(key))] = True
    for pages in (b.k_pages, b.v_pages):
        pages[~used] = float("nan")
    check(b, Tree(b).run(path=path), want)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_and_infinity_reach_the_rows_that_see_them(d, bad, path):
    """In V: of a context key, of nodes, of keys at a window's edge; single elements."""
    b = ref.tree_batch([30, 90, 12], [140, 300, 500], 4, 2, d, 16, [0, 100, 0], seed=6)
    for s, key, g, dim in [(0, 141, 0, 3), (0, 160, 1, d - 1), (1, 300 - 60, 0, 0), (1, 310, 1, 17), (1, 389, 0, 40)]:
        page, i = ref.slot(b, s, key)
        b.v_pages[page, i, g, dim] = bad
    page, i = ref.slot(b, 2, 3)
    b.v_pages[page, i, 1] = bad   # a context key that every node of request 2 sees
    check(b, Tree(b).run(path=path))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_keys(d, path):
    b = ref.tree_batch([30, 90], [140, 300], 4, 2, d, 16, [0, 100], seed=7)
    for s, key, g in [(0, 150, 0), (1, 300 - 60, 1), (1, 388, 0)]:
        page, i = ref.slot(b, s, key)
        b.k_pages[page, i, g, 5] = float("nan")
    check(b, Tree(b).run(path=path))


@pytest.mark.parametrize("path", PATHS)
def test_many_requests(path):
    """More than one launch's worth, some without nodes."""
    rng = np.random.default_rng(8)
    nodes = rng.integers(0, 4, size=1100).tolist()
    b = ref.tree_batch(nodes, rng.integers(0, 60, size=1100).tolist(), 2, 1, 64, 16, None, seed=8)
    check(b, Tree(b).run(path=path))


@pytest.mark.parametrize("path", PATHS)
def test_rows_behind_the_last_request_stay(path):
    b = ref.tree_batch([5, 9], [100, 300], 8, 2, 128, 16, None, seed=9)
    t = Tree(b)
    plan = t.plan(path=path)
    ws = binding.alloc_workspace(plan)
    q = torch.cat([t.q, torch.full((40, 8, 128), float("nan"), dtype=t.q.dtype, device="cuda")])
    out = torch.full_like(q, 7.0)
    mask = torch.cat([t.mask, torch.full((40, b.words), -1, dtype=torch.int64, device="cuda")])
    binding.rpa_forward_tree(q, t.k_pages, t.v_pages, t.table, t.cu, t.kv, mask, None, None, b.scale, out, plan, ws)
    assert binding.rpa_get_device_error(ws) == 0
    assert (out[14:] == 7).all()
    check(b, out[:14])


@pytest.mark.parametrize("path", PATHS)
def test_bad_pages_and_lengths_are_reported(path):
    b = ref.tree_batch([5, 9], [100, 300], 8, 2, 128, 16, [0, 50], seed=10)
    want = ref.attention(b)
    t = Tree(b)
    plan = t.plan(path=path)
    for name, at, value, code in [("table", (0, 2), b.pool, binding.RPA_DEVERR_PAGE_ID),
                                  ("table", (1, 18), -5, binding.RPA_DEVERR_PAGE_ID),
                                  ("kv", 0, 4, binding.RPA_DEVERR_LENGTHS), ("kv", 1, 1 << 30, binding.RPA_DEVERR_LENGTHS),
                                  ("cu", 1, -3, binding.RPA_DEVERR_LENGTHS), ("cu", 2, 1 << 30, binding.RPA_DEVERR_LENGTHS),
                                  ("pos", 6, -(1 << 31), binding.RPA_DEVERR_LENGTHS),
                                  ("pos", 7, (1 << 31) - 1, binding.RPA_DEVERR_LENGTHS)]:
        keep = getattr(t, name).clone()
        getattr(t, name)[at] = value
        ws = binding.alloc_workspace(plan)
        binding.rpa_forward_tree(*t.args(plan, ws))
        assert binding.rpa_get_device_error(ws) == code, name
        getattr(t, name).copy_(keep)
    t.out.fill_(float("nan"))
    binding.rpa_forward_tree(*t.args(plan, ws))
    assert binding.rpa_get_device_error(ws) == 0
    check(b, t.out, want)


def test_the_same_bits_every_time_and_from_a_graph():
    b = ref.tree_batch([8] * 20, list(range(50, 2050, 100)), 8, 1, 256, 128, None, seed=11)
    t = Tree(b)
    first = t.run().clone()
    plan = t.plan()
    ws = binding.alloc_workspace(plan)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    t.out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        binding.ForwardTreeCall(*t.args(plan, ws))()
        binding.rpa_forward_tree(*t.args(plan, ws))
    for _ in range(3):
        t.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.out.view(torch.int16), first.view(torch.int16))
    assert binding.rpa_get_device_error(ws) == 0
    check(b, first)


def test_calls_from_several_threads():
    bs = [ref.tree_batch([8 + i] * 12, [int(x) for x in np.random.default_rng(i).integers(0, 3000, 12)], 8, 2, 128, 64,
                         None, seed=20 + i) for i in range(3)]
    ts = [Tree(b) for b in bs]
    plans = [t.plan() for t in ts]
    wss = [binding.alloc_workspace(p) for p in plans]
    alone = [t.run().clone() for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    for t in ts:
        t.out.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(20):
                binding.rpa_forward_tree(*ts[i].args(plans[i], wss[i]), stream=streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not errors
    for t, a, ws in zip(ts, alone, wss):
        assert binding.rpa_get_device_error(ws) == 0
        assert torch.equal(t.out.view(torch.int16), a.view(torch.int16))


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    d, page = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128, 256]))
    hkv, group = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 33]))
    s = int(rng.integers(1, 9))
    most = int(2 ** rng.uniform(0, 8))
    nodes = rng.integers(0, most + 1, size=s).tolist()
    nodes[0] = max(1, nodes[0])
    ctx = (2 ** rng.uniform(0, 12, size=s)).astype(int).tolist()
    ctx[-1] = 0
    windows = [int(w) for w in rng.integers(0, 300, size=s)] if rng.random() < 0.5 else None
    b = ref.tree_batch(nodes, ctx, hkv * group, hkv, d, page, windows, seed=seed)
    t = Tree(b)
    sms = int(rng.choice([0, 0, 3, 17]))
    first = t.run(num_sms=sms).clone()
    check(b, first)
    assert torch.equal(first.view(torch.int16), t.run(num_sms=sms).view(torch.int16))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinite_keys(d, path):
    """A score of -infinity weighs nothing, one of +infinity makes its rows NaN; a row that sees nothing else is zeros."""
    b = ref.tree_batch([30, 90, 1], [140, 300, 0], 4, 2, d, 16, [0, 100, 0], seed=12)
    for s, key, g, bad in [(0, 150, 0, float("inf")), (1, 300 - 60, 1, -float("inf")), (1, 388, 0, float("inf"))]:
        page, i = ref.slot(b, s, key)
        b.k_pages[page, i, g, 5] = bad
    page, i = ref.slot(b, 2, 0)
    b.k_pages[page, i, :, 7] = float("inf")
    b.q[-1, :, 7] = -b.q[-1, :, 7].abs() - 1
    want = ref.attention(b)
    assert (want[0][-1] == 0).all() and torch.isnan(want[0]).any()
    check(b, Tree(b).run(path=path), want)


def test_two_graphs_share_a_workspace():
    bs = [ref.tree_batch([8] * 10, list(range(50, 2050, 200)), 8, 1, 256, 128, None, seed=13),
          ref.tree_batch([70, 5], [4000, 900], 8, 2, 128, 32, [0, 500], seed=14)]
    ts = [Tree(b) for b in bs]
    plans = [t.plan() for t in ts]
    ws = max((binding.alloc_workspace(p) for p in plans), key=lambda w: w.nbytes)
    graphs = []
    for t, p in zip(ts, plans):
        binding.rpa_forward_tree(*t.args(p, ws))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                binding.rpa_forward_tree(*t.args(p, ws))
        graphs.append(g)
    for _ in range(4):
        for t, g in zip(ts, graphs):
            t.out.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    assert binding.rpa_get_device_error(ws) == 0
    for b, t in zip(bs, ts):
        check(b, t.out)


@pytest.mark.parametrize("path", PATHS)
def test_a_pool_beyond_32_bits(path):
    """Pages past 2^32 elements: read, written by an append and moved by a commit."""
    b = ref.tree_batch([20, 9], [700, 130], 8, 2, 128, 256, None, seed=15)
    t = Tree(b)
    pages = (1 << 32) // (256 * 2 * 128) + 10
    shift = pages - b.pool
    small = t.k_pages, t.v_pages
    t.k_pages, t.v_pages = (torch.empty((pages, 256, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b.pool = pages
    t.table = torch.where(t.table >= 0, t.table + shift, -1).int()
    for big, s in zip((t.k_pages, t.v_pages), small):
        big[shift:] = s
    # The nodes' rows once more, by the append: no rotation.
    where = torch.tensor([(shift + p) * 256 + i for s in range(2) for p, i in
                          (ref.slot(b, s, b.ctx[s] + n) for n in range(b.nodes[s]))], device="cuda")
    assert int(where.min()) * 256 > 1 << 32
    flat = [x.view(-1, 2, 128) for x in (t.k_pages, t.v_pages)]
    rows = [f[where].clone() for f in flat]
    for f in flat:
        f[where] = float("nan")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.rpa_append_rope(None, *rows, None, where, None, None, t.k_pages, t.v_pages, workspace=ws)
    assert binding.rpa_get_device_error(ws) == 0
    assert all(torch.equal(f[where], r) for f, r in zip(flat, rows))
    check(b, t.run(path=path))
    moved = torch.tensor([[2, 5, 19], [0, 8, -1]], dtype=torch.int32, device="cuda")
    binding.rpa_commit_tree(t.k_pages, t.v_pages, where, t.cu, moved, ws)
    assert binding.rpa_get_device_error(ws) == 0
    for f, r in zip(flat, rows):
        assert torch.equal(f[where[:3]], r[[2, 5, 19]]) and torch.equal(f[where[20:22]], r[[20, 28]])
        assert torch.equal(f[where[3:20]], r[3:20])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_values(d, path):
    """Values of 2^90 under scores that grow by dozens from one tile of keys to the next."""
    b = ref.tree_batch([20, 3], [1500, 700], 4, 1, d, 32, None, seed=16, scale=0.5)
    for s in range(2):
        for key in range(b.kv[s]):
            page, i = ref.slot(b, s, key)
            b.k_pages[page, i] *= 0.25 + key / 500
    b.v_pages *= 2.0 ** 90
    check(b, Tree(b).run(path=path))
