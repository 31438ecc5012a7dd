"""The operators around the attention of drafted trees, each against its definition:
rpa_build_tree, rpa_append_rope, rpa_commit_tree, rpa_trim_tables, and a step of all of
them over a cache."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build

from . import tree_reference as ref
from .test_gpu_tree import check, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int64).astype(np.int32)).cuda()


# ---------------------------------------------------------------- masks and positions

@pytest.mark.parametrize("nodes,words,windows", [
    ([1], 1, None), ([8] * 3, 1, None), ([0, 5, 0], 2, None), ([64, 65, 1], 2, [3, 0, 1]), ([256, 17], 4, [0, 5]),
    ([1024, 1000], 16, None), ([1024], 16, [40]), ([3] * 700, 1, None), ([130, 200], 5, [1, 2]),
])
def test_build_tree(nodes, words, windows):
    rng = np.random.default_rng(sum(nodes))
    parents = [ref.random_parents(t, rng) if t else [] for t in nodes]
    ctx = rng.integers(0, 5000, size=len(nodes)).tolist()
    cu = np.concatenate([[0], np.cumsum(nodes)])
    total = int(cu[-1])
    pad = 7
    mask = torch.full((total + pad, words), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((total + pad,), 99, dtype=torch.int32, device="cuda")
    ws = workspace()
    binding.rpa_build_tree(i32(sum(parents, []) + [0] * pad), i32(cu), i32(np.array(ctx) + nodes),
                           None if windows is None else i32(windows), mask, pos, ws)
    assert binding.rpa_get_device_error(ws) == 0
    for s, t in enumerate(nodes):
        sees, depth = ref.tree_of(parents[s], windows[s] if windows else 0)
        got = mask[cu[s]:cu[s + 1]].cpu().numpy().view(np.uint64)
        assert np.array_equal(got, ref.mask_words(sees, words))
        assert np.array_equal(pos[cu[s]:cu[s + 1]].cpu().numpy(), ctx[s] + depth)
    assert (mask[total:] == 99).all() and (pos[total:] == 99).all()


def test_build_tree_chain_of_the_largest_size():
    mask = torch.zeros((1024, 16), dtype=torch.int64, device="cuda")
    pos = torch.zeros(1024, dtype=torch.int32, device="cuda")
    binding.rpa_build_tree(i32(range(-1, 1023)), i32([0, 1024]), i32([1024]), None, mask, pos)
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), ref.mask_words(np.tri(1024, dtype=bool), 16))
    assert np.array_equal(pos.cpu().numpy(), np.arange(1024))


def test_build_tree_reports():
    """Bad parents count as -1, requests of unusable lengths are left out."""
    ws = workspace()
    mask = torch.full((9, 1), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((9,), 99, dtype=torch.int32, device="cuda")
    binding.rpa_build_tree(i32([-1, 1, -7, 0, 1, 5, 100, -1, 0]), i32([0, 3, 9]), i32([13, 6]), None, mask, pos, ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_LENGTHS
    assert mask.flatten().tolist()[:3] == [1, 2, 4] and pos.tolist()[:3] == [10, 10, 10]
    for cu, kv in [([0, 70, 70], [70, 0]), ([0, -3, 9], [5, 12]), ([0, 3, 2], [5, 5]), ([0, 3, 100], [5, 100]),
                   ([0, 3, 9], [2, 5]), ([-1, 3, 9], [5, 5]), ([0, 3, 9], [-1, -1 << 31]), ([3, 1 << 30, -1 << 31], [5, 5])]:
        mask.fill_(99)
        pos.fill_(99)
        binding.rpa_build_tree(i32([-1] * 9), i32(cu), i32(kv), None, mask, pos, ws)
        assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_LENGTHS, (cu, kv)
        for s in range(2):  # rows of a usable request are written, no others
            ok = 0 <= cu[s] <= cu[s + 1] <= 9 and cu[s + 1] - cu[s] <= min(64, kv[s])
            if not ok and 0 <= cu[s] < cu[s + 1] <= 9 and not (s == 0 and cu[1] > cu[2] >= 0):
                assert (mask[cu[s]:cu[s + 1]] == 99).all() and (pos[cu[s]:cu[s + 1]] == 99).all()


# ---------------------------------------------------------------- rotation and cache write

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f32": (torch.float32, 2.0 ** -24)}


def e4m3(x):
    """Values of e4m3 bytes."""
    x = x.cpu().numpy().astype(np.int64)
    e, m = (x >> 3) & 15, x & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((x & 127) == 127, np.nan, v)
    return torch.from_numpy(np.where(x & 128, -v, v))


def near_turned(got, x, pos, freq, pairs, half, scale=None):
    want = ref.turned(x, pos, freq, pairs)
    size = ref.turned(x.abs(), 0 * np.asarray(pos), freq, pairs)  # |x|, then |x| + |y| of a pair
    n = len(freq)
    i = torch.arange(n)
    first, second = (2 * i, 2 * i + 1) if pairs else (i, i + n)
    both = size[..., first] + size[..., second]
    size[..., first] = both
    size[..., second] = both
    most = float(np.max(np.abs(np.asarray(pos, np.float64)))) * float(np.max(freq)) if n and len(pos) else 0.0
    bound = half * want.abs() + size * (2.0 ** -47 * most + 2.0 ** -21)
    if scale is not None:
        # (two roundings more: the quotient's)
        want, bound = want / scale, 2.0 ** -4 * (want / scale).abs() + 2.0 ** -10 + bound / scale
        want = want.clamp(-448, 448)
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-300)).max())


APPEND = [
    # (tokens, Hq, Hkv, D, page, rotary, pairs, fused, reach)
    (1, 4, 1, 64, 16, 64, False, False, 100), (7, 8, 1, 256, 128, 256, False, True, 131072),
    (33, 6, 3, 128, 1, 128, True, True, 5000), (200, 7, 7, 64, 32, 32, False, False, 1 << 24),
    (65, 0, 2, 128, 64, 128, False, True, 4096), (513, 32, 16, 256, 128, 64, True, False, 1 << 20),
    (3000, 16, 2, 128, 16, 128, False, True, 40000), (5, 2, 1, 64, 256, 16, True, False, 10),
    (90, 3, 1, 256, 16, 0, False, False, 10), (20, 1, 5, 64, 64, 48, False, True, 2000),
]


@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, dtype, kv):
    t, hq, hkv, d, page, rotary, pairs, fused, reach = APPEND[case]
    dt, half = TYPES[dtype]
    gen = torch.Generator().manual_seed(case)
    rows = torch.randn((t, hq + 2 * hkv, d), generator=gen).to(dt)
    dev = rows.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pool = ref.ceil_div(t, page) + 2
    slots = torch.randperm(pool * page, generator=gen)[:t]
    slots[::5] = -1
    pos = torch.randint(0, reach, (t,), generator=gen, dtype=torch.int32)
    pos[0] = reach - 1
    freq = (10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))).float()
    fp8 = kv == "fp8"
    fill = 0x31 if fp8 else 3.0
    kp = torch.full((pool, page, hkv, d), fill, dtype=torch.uint8 if fp8 else dt, device="cuda")
    vp = kp.clone()
    ks, vs = (torch.rand(hkv, generator=gen) * 0.02 + 0.005 for _ in range(2))
    q_out = torch.empty((t, hq, d), dtype=dt, device="cuda") if hq else None
    ws = workspace()
    binding.rpa_append_rope(q if hq else None, k, v, pos.cuda(), slots.cuda(), freq.cuda() if rotary else None, q_out,
                            kp, vp, k_scale=ks.cuda() if fp8 else None, v_scale=vs.cuda() if fp8 else None,
                            interleaved=pairs, workspace=ws)
    assert binding.rpa_get_device_error(ws) == 0
    x = rows.double()
    if hq:
        near_turned(q_out, x[:, :hq], pos, freq.numpy(), pairs, half)
    use = slots >= 0
    at = slots[use]
    for pages, part, p, f, s in ((kp, x[:, hq:hq + hkv], pos, freq.numpy(), ks), (vp, x[:, hq + hkv:], pos, freq[:0].numpy(), vs)):
        flat = pages.flatten(0, 1).cpu()
        got = e4m3(flat[at]) if fp8 else flat[at]
        near_turned(got, part[use], p[use], f, pairs, half, s.double()[None, :, None] if fp8 else None)
        rest = torch.ones(pool * page, dtype=torch.bool)
        rest[at] = False
        assert (flat[rest] == fill).all()   # nothing else changes
    if not fp8:  # v goes over bit by bit
        assert torch.equal(vp.flatten(0, 1).cpu()[at], rows[:, hq + hkv:][use])


def test_append_in_place_and_on_another_stream():
    t, hq, hkv, d = 40, 8, 2, 128
    q, k, v = (torch.randn((t, h, d), device="cuda", dtype=torch.bfloat16) for h in (hq, hkv, hkv))
    pos, slots = torch.arange(t, dtype=torch.int32, device="cuda"), torch.arange(t, device="cuda")
    freq = 10000.0 ** (-torch.arange(64, device="cuda") / 64.0)
    pools = [torch.zeros((3, 16, hkv, d), device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    binding.rpa_append_rope(q, k, v, pos, slots, freq, out, pools[0], pools[1], stream=side)
    torch.cuda.synchronize()
    binding.rpa_append_rope(q, k, v, pos, slots, freq, q, pools[2], pools[3])
    assert torch.equal(q, out) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.parametrize("pos", [0, 1, (1 << 31) - 1, -(1 << 31), -5])
def test_append_any_position(pos):
    x = torch.randn((1, 1, 64), dtype=torch.float32)
    freq = torch.tensor([1.0, 0.5, 3.0, -0.3, 1e-3, 7.5, 100.0, 0.0])
    out = torch.empty((1, 1, 64), device="cuda")
    pages = torch.zeros((1, 1, 1, 64), device="cuda")
    binding.rpa_append_rope(x.cuda(), x.cuda(), x.cuda(), i32([pos]), torch.zeros(1, dtype=torch.int64, device="cuda"),
                            freq.cuda(), out, pages, pages.clone())
    p = torch.tensor([pos])
    near_turned(out, x.double(), p, freq.numpy(), False, 2.0 ** -24)


def test_append_keeps_nan_and_saturates():
    """e4m3: the middle of two codes to the even one, 448 at most, NaN as NaN; zero, and values below the smallest."""
    v = torch.zeros((1, 1, 64))
    v[0, 0, :12] = torch.tensor([float("nan"), float("inf"), -float("inf"), 500.0, -1e9, 448.0, 2.0 ** -10, 1.5 * 2.0 ** -9,
                                 17.0, 19.0, -0.0, 464.0])
    k = torch.zeros((1, 1, 64))
    kp = torch.zeros((1, 1, 1, 64), dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    one = torch.ones(1, device="cuda")
    binding.rpa_append_rope(None, k.cuda(), v.cuda(), None, torch.zeros(1, dtype=torch.int64, device="cuda"), None, None,
                            kp, vp, k_scale=one, v_scale=one)
    got = e4m3(vp.flatten())
    assert torch.isnan(got[0])
    assert got[1:12].tolist() == [448.0, -448.0, 448.0, -448.0, 448.0, 0.0, 2.0 ** -8, 16.0, 20.0, 0.0, 448.0]
    assert (got[12:] == 0).all()


def test_append_reports_slots_outside_the_pool():
    t = 6
    k = torch.randn((t, 2, 64), device="cuda", dtype=torch.bfloat16)
    pool = torch.zeros((2, 16, 2, 64), device="cuda", dtype=torch.bfloat16)
    other, q_out = pool.clone(), torch.empty_like(k)
    ws = workspace()
    slots = torch.tensor([0, 32, -1, 1 << 40, 31, -(1 << 62)], device="cuda")
    binding.rpa_append_rope(k, k, k, i32([0] * t), slots, torch.ones(32, device="cuda"), q_out, pool, other, workspace=ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
    flat = other.flatten(0, 1)
    assert torch.equal(flat[0], k[0]) and torch.equal(flat[31], k[4]) and not flat[1:31].any()
    assert torch.equal(q_out, k)


# ---------------------------------------------------------------- the path

def commit_ref(pages, slots, cu, path):
    flat = pages.flatten(0, 1).clone()
    for s, row in enumerate(path):
        old = flat.clone()
        for k, j in enumerate(row):
            if j >= 0:
                flat[slots[cu[s] + k]] = old[slots[cu[s] + j]]
    return flat.view_as(pages)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("nodes,width,hkv,d,page", [
    ([1], 1, 1, 64, 16), ([8, 3, 0, 20], 6, 2, 128, 16), ([64] * 5, 30, 1, 256, 128), ([300, 40], 200, 3, 64, 1),
    ([1024], 1024, 1, 64, 32), ([6] * 400, 5, 1, 64, 16), ([30, 12], 11, 16, 256, 128),
])
def test_commit(nodes, width, hkv, d, page, dt):
    rng = np.random.default_rng(len(nodes) + width)
    cu = np.concatenate([[0], np.cumsum(nodes)])
    path = np.full((len(nodes), width), -1, np.int32)
    for s, t in enumerate(nodes):
        n = int(rng.integers(0, min(t, width) + 1))
        path[s, :n] = np.sort(rng.choice(t, n, replace=False))
    pool = ref.ceil_div(int(cu[-1]), page) + 2
    slots = torch.from_numpy(rng.permutation(pool * page)[:int(cu[-1])])
    pages = [torch.from_numpy(rng.integers(0, 120, (pool, page, hkv, d))).to(dt) for _ in range(2)]
    dev = [p.cuda() for p in pages]
    ws = workspace()
    binding.rpa_commit_tree(*dev, slots.cuda(), i32(cu), torch.from_numpy(path).cuda(), ws)
    assert binding.rpa_get_device_error(ws) == 0
    for got, p in zip(dev, pages):
        assert torch.equal(got.cpu(), commit_ref(p, slots, cu, path))


def test_commit_reports_and_leaves():
    pages = torch.arange(4 * 8 * 64, dtype=torch.float32).view(4, 8, 1, 64).cuda()
    slots = torch.arange(12, device="cuda")
    cu = i32([0, 6, 12])
    good = [1, 3, -1]
    for row, code in [([3, 1, -1], binding.RPA_DEVERR_LENGTHS), ([2, 2, -1], binding.RPA_DEVERR_LENGTHS),
                      ([1, 6, -1], binding.RPA_DEVERR_LENGTHS), ([-1, 2, -1], binding.RPA_DEVERR_LENGTHS),
                      ([0, -1, 5], binding.RPA_DEVERR_LENGTHS), ([1 << 30, -1, -1], binding.RPA_DEVERR_LENGTHS)]:
        k, v, ws = pages.clone(), -pages, workspace()
        binding.rpa_commit_tree(k, v, slots, cu, torch.tensor([row, good], dtype=torch.int32, device="cuda"), ws)
        assert binding.rpa_get_device_error(ws) == code, row
        want = commit_ref(pages.cpu(), slots.cpu(), [0, 6, 12], [[-1], good])
        assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), -want), row
    for bad in (32, -1, 1 << 40):
        k, v, ws = pages.clone(), -pages, workspace()
        s = slots.clone()
        s[3] = bad
        binding.rpa_commit_tree(k, v, s, cu, torch.tensor([[0, 3, 4], good], dtype=torch.int32, device="cuda"), ws)
        assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
        assert torch.equal(k.cpu(), commit_ref(pages.cpu(), slots.cpu(), [0, 6, 12], [[-1], good]))
    for bad_cu in ([0, -6, 12], [0, 6, 13], [6, 0, 12], [0, 1 << 30, 12]):
        k, v, ws = pages.clone(), -pages, workspace()
        binding.rpa_commit_tree(k, v, slots, i32(bad_cu), torch.tensor([[1, 2, 3], [1, 2, 3]], dtype=torch.int32, device="cuda"), ws)
        assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_LENGTHS, bad_cu


# ---------------------------------------------------------------- requests cut short

TRIM = [([1], [0], 16), ([5, 0, 40], [2, 0, 40], 16), ([100, 17, 16, 15], [1, 1, 1, 15], 1), ([300] * 600, None, 16),
        ([(i * 37) % 900 for i in range(5000)], None, 32), ([70000], [69999], 64), ([128, 129, 127], [0, 1, 127], 128)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(TRIM)))
def test_trim(case, in_place):
    kv, drop, p = TRIM[case]
    rng = np.random.default_rng(case)
    drop = [int(rng.integers(0, k + 1)) for k in kv] if drop is None else drop
    held = [ref.ceil_div(k, p) for k in kv]
    spare, pool = 3, sum(held) + 3
    perm = rng.permutation(pool)
    table, free = np.full((len(kv), max(held) + 1), -1), np.full(pool, -7)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = perm[at:at + h]
        at += h
    free[:spare] = perm[at:]
    want, count, left = free.copy(), spare, [k - d for k, d in zip(kv, drop)]
    for s, h in enumerate(held):
        for j in range(ref.ceil_div(left[s], p), h):
            want[count] = table[s, j]
            count += 1
    t, f, kv0, c0, ws = i32(table), i32(free), i32(kv), i32([spare]), workspace()
    kv1, c1 = (kv0, c0) if in_place else (i32([9] * len(kv)), i32([9]))
    binding.rpa_trim_tables(i32(drop), kv0, t, f, c0, kv1, c1, p, ws)
    assert binding.rpa_get_device_error(ws) == 0
    assert f.tolist() == want.tolist() and int(c1) == count and kv1.tolist() == left
    assert np.array_equal(t.cpu().numpy(), table)


@pytest.mark.parametrize("kv,drop,count,code", [
    ([40, 20], [41, 0], 1, binding.RPA_DEVERR_LENGTHS), ([40, 20], [0, -1], 1, binding.RPA_DEVERR_LENGTHS),
    ([-1, 20], [0, 3], 1, binding.RPA_DEVERR_LENGTHS), ([100, 20], [1, 3], 1, binding.RPA_DEVERR_LENGTHS),
    ([40, 20], [40, 20], 8, binding.RPA_DEVERR_PAGES), ([40, 20], [0, 0], -1, binding.RPA_DEVERR_PAGES),
])
def test_trim_all_or_nothing(kv, drop, count, code):
    table, free = i32([[0, 1, 2], [3, 4, -1]]), i32([9] * 10)
    kv0, c0, ws = i32(kv), i32([count]), workspace()
    kv1, c1 = i32([7, 7]), i32([7])
    binding.rpa_trim_tables(i32(drop), kv0, table, free, c0, kv1, c1, 16, ws)
    assert binding.rpa_get_device_error(ws) == code
    assert kv1.tolist() == kv and int(c1) == count and free.tolist() == [9] * 10


def test_trim_reports_bad_pages():
    free, ws = i32([9] * 10), workspace()
    kv, c = i32([40]), i32([0])
    binding.rpa_trim_tables(i32([39]), kv, i32([[0, 77, 2]]), free, c, kv, c, 16, ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
    assert free.tolist()[:2] == [-1, 2] and int(c) == 2 and kv.tolist() == [1]


# ---------------------------------------------------------------- the step

@pytest.mark.parametrize("captured", [False, True])
def test_a_step_of_all_operators(captured):
    """Two speculative steps: pages taken, nodes appended, attended and committed, pages given back.  The cache then
    holds the accepted tokens' rows in order, and no page is lost."""
    rng = np.random.default_rng(5)
    hq, hkv, d, page, seqs, most = 8, 2, 128, 16, 3, 12
    kv_host = [130, 15, 40]
    pool, width = 60, 20
    perm = rng.permutation(pool)
    table_host, at = np.full((seqs, width), -1), 0
    for s, k in enumerate(kv_host):
        table_host[s, :ref.ceil_div(k, page)] = perm[at:at + ref.ceil_div(k, page)]
        at += ref.ceil_div(k, page)
    free_host = np.full(pool, -1)
    free_host[:pool - at] = perm[at:]
    table, free, count, kv = i32(table_host), i32(free_host), i32([pool - at]), i32(kv_host)
    k_pages, v_pages = (torch.randn((pool, page, hkv, d), device="cuda").bfloat16() for _ in range(2))
    cached = [[p[table_host[s, np.arange(n) // page], np.arange(n) % page].cpu() for p in (k_pages, v_pages)]
              for s, n in enumerate(kv_host)]
    freq = 10000.0 ** (-torch.arange(d // 2, device="cuda") / (d / 2))
    nodes, words = [most, 7, 1], 1
    total = sum(nodes)
    cu_host = np.concatenate([[0], np.cumsum(nodes)])
    new, cu = i32(nodes), i32([0] * (seqs + 1))
    slots = torch.zeros(total, dtype=torch.int64, device="cuda")
    parents, mask, pos = i32([0] * total), torch.zeros((total, words), dtype=torch.int64, device="cuda"), i32([0] * total)
    rows = torch.zeros((total, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    q, out = torch.zeros((total, hq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((total, hq, d), dtype=torch.bfloat16, device="cuda")
    path, drop = i32([[-1] * most] * seqs), i32([0] * seqs)

    for step in range(2):
        plan = binding.rpa_plan(cu_host, np.array(kv_host) + nodes, None, hq, hkv, d, page, width, pool, tree_words=words)
        ws = binding.alloc_workspace(plan)

        def verify():
            binding.rpa_build_tables(new, kv, table, free, count, cu, kv, slots, count, page, ws)
            binding.rpa_build_tree(parents, cu, kv, None, mask, pos, ws)
            binding.rpa_append_rope(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], pos, slots, freq, q, k_pages,
                                    v_pages, workspace=ws)
            binding.rpa_forward_tree(q, k_pages, v_pages, table, cu, kv, mask, None, None, d ** -0.5, out, plan, ws)

        def keep():
            binding.rpa_commit_tree(k_pages, v_pages, slots, cu, path, ws)
            binding.rpa_trim_tables(drop, kv, table, free, count, kv, count, page, ws)

        trees = [ref.random_parents(t, rng) for t in nodes]
        parents.copy_(i32(sum(trees, [])))
        rows.copy_(torch.from_numpy(rng.standard_normal(rows.shape)))
        paths = []
        for t, p in zip(nodes, trees):  # from a random node up to its root
            j, way = int(rng.integers(t)), []
            while j >= 0:
                way.append(j)
                j = p[j]
            paths.append(way[::-1])
        path.copy_(i32([w + [-1] * (most - len(w)) for w in paths]))
        drop.copy_(i32([t - len(w) for t, w in zip(nodes, paths)]))
        appended = []
        for part in (verify, keep):
            if captured:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    part()
                g.replay()
            else:
                part()
            appended.append(k_pages.flatten(0, 1)[slots].cpu())
            assert binding.rpa_get_device_error(ws) == 0
        # The attention, over the rows as the cache holds them.
        b = ref.tree_batch(nodes, kv_host, hq, hkv, d, page, None, seed=0, spare=0)
        b.q = q.cpu()
        pos_host = np.concatenate([kv_host[s] + ref.tree_of(trees[s])[1] for s in range(seqs)])
        assert np.array_equal(pos.cpu().numpy(), pos_host)
        x = rows.double().cpu()
        near_turned(q, x[:, :hq], pos_host, freq.cpu().numpy(), False, 2.0 ** -8)
        near_turned(appended[0], x[:, hq:hq + hkv], pos_host, freq.cpu().numpy(), False, 2.0 ** -8)
        for s in range(seqs):
            b.sees[s] = ref.tree_of(trees[s])[0]
            mine = slice(int(cu_host[s]), int(cu_host[s + 1]))
            k_all = torch.cat([cached[s][0], appended[0][mine]])
            v_all = torch.cat([cached[s][1], rows.cpu()[mine, hq + hkv:]])
            key = np.arange(len(k_all))
            b.k_pages[b.table[s, key // page], key % page] = k_all
            b.v_pages[b.table[s, key // page], key % page] = v_all
        check(b, out)
        # The cache holds the context and the accepted nodes.
        kv_host = [k + len(w) for k, w in zip(kv_host, paths)]
        assert kv.tolist() == kv_host
        t = table.cpu().numpy()
        held = []
        for s in range(seqs):
            rows_s = [int(cu_host[s]) + j for j in paths[s]]
            key = np.arange(kv_host[s])
            k_now, v_now = (p.cpu()[t[s, key // page], key % page] for p in (k_pages, v_pages))
            assert torch.equal(v_now, torch.cat([cached[s][1], rows.cpu()[rows_s, hq + hkv:]]))
            assert torch.equal(k_now[:len(cached[s][0])], cached[s][0])
            near_turned(k_now[len(cached[s][0]):], x[rows_s, hq:hq + hkv], pos_host[rows_s], freq.cpu().numpy(), False, 2.0 ** -8)
            cached[s] = [k_now, v_now]
            held += t[s, :ref.ceil_div(kv_host[s], page)].tolist()
        assert sorted(held + free.cpu().tolist()[:int(count)]) == list(range(pool))
