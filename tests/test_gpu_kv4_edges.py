"""Attention over 4-bit pages where a user meets its edges: NaN that only some
rows see, probabilities far below a row's largest, lengths that disagree with
the plan, scales of zero and below.

Bounds are those of test_gpu_kv4.py, with the probabilities' own rounding: f16
(2^-11 of itself) on the split-KV kernels, bf16 (2^-8) where a prefill ran.
"""

from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import oracle
from ragged_paged_attention_rpa_gb300 import binding, build, workloads

from .test_gpu_kv4 import FEW, ROWS, Kv4Batch, batch, check, cuda, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def sees(b, s):
    """Mask [q_len, kv_len] of the keys each query of sequence s sees."""
    n, m = int(b.cu_q_lens[s + 1] - b.cu_q_lens[s]), int(b.kv_lens[s])
    back = (m - n + np.arange(n))[:, None] - np.arange(m)[None]
    w = 0 if b.window is None else int(b.window[s])
    return (back >= 0) & ((back < w) if w > 0 else True)


def slot(b, s, key):
    return b.page_table[s, key // b.page_size], key % b.page_size


def check_nan(b, out, want_nan, ref, prefill):
    """NaN exactly where `want_nan` says, the bound elsewhere."""
    got = out.float().cpu().numpy().reshape(want_nan.shape).astype(np.float64)
    assert np.array_equal(np.isnan(got), want_nan), \
        "%d NaN missing, %d too many" % ((want_nan & ~np.isnan(got)).sum(), (np.isnan(got) & ~want_nan).sum())
    got = np.where(want_nan, ref[0].reshape(want_nan.shape), got)
    check(b, torch.from_numpy(got), prefill=prefill, ref=ref)


# ---------------------------------------------------------------- NaN keys

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nan_keys", [[61, 62, 63, 64], [125, 126, 127, 128], [0, 189, 190, 191]])
def test_a_nan_key_reaches_the_prompt_rows_that_see_it(d, nan_keys):
    """Wherever in a key tile it lies, on 4-bit pages and on bf16 ones."""
    n = len(nan_keys)
    b = batch([193 + i for i in range(n)], [193 + i for i in range(n)], 4, 2, d, 16, seed=31)
    ref = reference(b)
    want = np.zeros((b.q.shape[0], 4, d), bool)
    for s, key in enumerate(nan_keys):
        page, at = slot(b, s, key)
        b.k_fp4_scale[page, 1, at, d // 16 - 1] = 255
        want[b.cu_q_lens[s] + key:b.cu_q_lens[s + 1], 2:] = True
    r = Kv4Batch(b)
    assert r.plan.info()["num_prefill_seqs"] == n
    check_nan(b, r.call(), want, ref, True)
    assert binding.rpa_get_device_error(r.ws) == 0


@pytest.mark.parametrize("pairs", [0, 2])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("nan_keys", [[61, 62, 63, 64], [125, 126, 127, 128]])
def test_a_nan_key_of_16_bit_pages_reaches_the_prompt_rows_that_see_it(d, pairs, nan_keys):
    n = len(nan_keys)
    b = workloads.make_batch([193 + i for i in range(n)], [193 + i for i in range(n)], num_q_heads=4,
                             num_kv_heads=2, head_dim=d, page_size=16, seed=32)
    want = np.zeros((b.q.shape[0], 4, d), bool)
    for s, key in enumerate(nan_keys):
        page, at = slot(b, s, key)
        b.k_pages[page, at, 1, 5] = 0x7FC0
        want[b.cu_q_lens[s] + key:b.cu_q_lens[s + 1], 2:] = True
    db = binding.Batch(b)
    plan = db.plan(prefill_pairs=pairs)
    ws = binding.alloc_workspace(plan)
    got = db.forward(plan, ws).float().cpu().numpy()
    assert binding.rpa_get_device_error(ws) == 0
    assert np.array_equal(np.isnan(got), want)


# ---------------------------------------------------------------- NaN values

VALUES = [
    # (q_lens, kv_lens, Hq, Hkv, D, P, windows, num_sms): what holds the rows
    ([3, 2], [300, 40], 2, 2, 64, 16, None, 0),                       # tiles of 8
    ([4, 16], [70, 500], 3, 1, 64, 32, [0, 9], 0),                    # of 16, of 64
    ([12, 7, 1], [513, 100, 30], 1, 1, 128, 16, [0, 5, 0], 0),        # of 16, of 8
    ([6, 4], [4000, 130], 4, 2, 128, 64, None, 0),                    # of 16, cut over CTAs
    ([8, 5], [700, 90], 1, 1, 256, 128, [0, 3], 0),                   # of 8
    ([5, 16], [90, 3000], 3, 1, 256, 16, None, 0),                    # two of 8; of 64
    ([40, 33], [2000, 33], 1, 1, 128, 64, [0, 6], 0),                 # of 64
    ([20, 30], [300, 65], 2, 2, 256, 16, [0, 9], 0),
    ([16, 9], [5000, 70], 4, 1, 64, 16, [700, 0], 0),
    ([3] * 30, [50 + 9 * i for i in range(30)], 2, 1, 128, 16, None, 1),  # whole segments, one CTA
    ([5] * 30, [50 + 9 * i for i in range(30)], 8, 2, 64, 16, None, 1),
]


def nan_values(ql, kv, hq, hkv, d, p, win, sms, seed, **plan_kw):
    """A block of V that reads as NaN makes NaN its 16 dimensions of the rows
    that see its key, and nothing else: not the rows for which the key lies in
    the future or before the window."""
    b = batch(ql, kv, hq, hkv, d, p, win, seed=seed)
    ref = reference(b)
    want = np.zeros((b.q.shape[0], hq, d), bool)
    group = hq // hkv
    rng = np.random.default_rng(seed)
    for s in range(len(ql)):
        if s % 3 == 2:
            continue
        first = kv[s] - ql[s]
        keys = {kv[s] - 1, first + ql[s] // 2, min(kv[s] - 1, first + 1), max(0, first - 3), int(rng.integers(0, kv[s]))}
        see = sees(b, s)
        for key in sorted(keys):
            g, blk = int(rng.integers(0, hkv)), int(rng.integers(0, d // 16))
            page, at = slot(b, s, key)
            b.v_fp4_scale[page, g, at, blk] = 255
            rows = b.cu_q_lens[s] + np.nonzero(see[:, key])[0]
            want[rows, g * group:(g + 1) * group, 16 * blk:16 * blk + 16] = True
    assert want.any() and not want.all()
    r = Kv4Batch(b, num_sms=sms, **plan_kw)
    prefill = r.plan.info()["num_prefill_seqs"] > 0
    assert prefill == (max(ql) * group > 128)
    out = r.call().clone()
    assert binding.rpa_get_device_error(r.ws) == 0
    check_nan(b, out, want, ref, prefill)
    assert bool((r.ws[:256] == 0).all())             # words of the header back at zero
    # Without them, on the same workspace, nothing of it is left.
    good = batch(ql, kv, hq, hkv, d, p, win, seed=seed)
    r.pool[3].copy_(cuda(good.v_fp4_scale))
    check(good, r.call(), prefill=prefill, ref=ref)
    # In a captured call, with and without.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.call()
    for scales, expect in ((b, want), (good, np.zeros_like(want)), (b, want)):
        r.pool[3].copy_(cuda(scales.v_fp4_scale))
        graph.replay()
        check_nan(b, r.out, expect, ref, prefill)


@pytest.mark.parametrize("case", range(len(VALUES)))
def test_a_nan_value_reaches_the_rows_that_see_it(case):
    nan_values(*VALUES[case], seed=1000 + case)


# ---------------------------------------------------------------- NaN values of prompts

PROMPT_VALUES = [
    ([200, 1], [333, 50], 2, 2, 128, 16, None, 0),                    # prompts
    ([150, 140], [150, 400], 8, 1, 256, 128, [0, 33], 0),
    ([300, 129], [300, 700], 4, 2, 64, 16, [7, 0], 0),
    ([260], [260], 128, 1, 64, 32, [100], 0),                         # G = 128
    ([129] * 5, [129, 140, 150, 333, 129], 256, 256, 64, 16, None, 0),  # more items than a launch takes
]


@pytest.mark.parametrize("dynamic", [0, -1])
@pytest.mark.parametrize("case", range(len(PROMPT_VALUES)))
def test_a_nan_value_reaches_the_prompt_rows_that_see_it(case, dynamic):
    nan_values(*PROMPT_VALUES[case], seed=1050 + case, prefill_dynamic=dynamic)


# ---------------------------------------------------------------- NaN anywhere

@pytest.mark.parametrize("seed", range(40))
def test_nan_blocks_anywhere(seed):
    """Random batches with NaN blocks of K (all of the rows that see the key) and
    of V (their 16 dimensions), wherever they lie."""
    rng = np.random.default_rng(7000 + seed)
    pick = lambda *a: a[int(rng.integers(len(a)))]
    d, p, hkv, group = pick(64, 128, 256), pick(16, 32, 128), pick(1, 2, 3), pick(1, 2, 3, 8, 16)
    ql = [pick(1, 2, 4, 8, int(rng.integers(9, 40)), int(rng.integers(40, 260))) for _ in range(int(rng.integers(1, 8)))]
    kv = [q + pick(0, int(rng.integers(0, 40)), int(rng.integers(0, 900))) for q in ql]
    win = pick(None, [pick(0, 1, 7, 60) for _ in ql])
    b = batch(ql, kv, hkv * group, hkv, d, p, win, seed=seed)
    ref = reference(b)
    want = np.zeros((b.q.shape[0], hkv * group, d), bool)
    for _ in range(int(rng.integers(1, 12))):
        s = int(rng.integers(len(ql)))
        key, g, blk = int(rng.integers(max(0, kv[s] - 300), kv[s])), int(rng.integers(hkv)), int(rng.integers(d // 16))
        page, at = slot(b, s, key)
        rows = b.cu_q_lens[s] + np.nonzero(sees(b, s)[:, key])[0]
        of_k = rng.random() < 0.2
        (b.k_fp4_scale if of_k else b.v_fp4_scale)[page, g, at, blk] = 255
        want[rows, g * group:(g + 1) * group, slice(None) if of_k else slice(16 * blk, 16 * blk + 16)] = True
    r = Kv4Batch(b, num_sms=pick(0, 0, 1, 9))
    out = r.call().clone()
    assert binding.rpa_get_device_error(r.ws) == 0
    check_nan(b, out, want, ref, r.plan.info()["num_prefill_seqs"] > 0)
    assert torch.equal(r.call().view(torch.int16), out.view(torch.int16))


# ---------------------------------------------------------------- small probabilities

@pytest.mark.parametrize("hq,tokens,d", [(1, 1, 64), (12, 1, 64), (12, 1, 128), (8, 1, 128), (8, 1, 256), (64, 1, 64),
                                         (64, 1, 128), (32, 1, 256)])
def test_probabilities_far_below_the_largest(hq, tokens, d):
    """One key takes nearly all of each row and has a value of zero; the output
    is what the others, 2^-20.4 of it each, add up to.  Their probabilities lie
    midway between two multiples of 2^-24 of the largest."""
    n, kv = 64, 200
    b = batch([tokens] * n, [kv] * n, hq, 1, d, 16, seed=5)
    gap = 24 - np.log2(12.5)
    k = np.zeros(b.k_fp4.shape[:3] + (d,))
    v = np.ones_like(k)
    k[..., 0] = -6.0
    for s in range(n):
        page, at = slot(b, s, 0)
        k[page, 0, at, 0] = 6.0
        v[page, 0, at] = 0.0
    q = np.zeros(b.q.shape, np.float32)
    q[..., 0] = 1.0
    b.q = oracle.round_bf16(q)
    b.k_fp4, b.k_fp4_scale = workloads.kv4_encode(k)
    b.v_fp4, b.v_fp4_scale = workloads.kv4_encode(v)
    b.sm_scale = float(np.float32(gap * np.log(2) / 12))
    r = Kv4Batch(b, num_sms=1)                       # whole segments
    assert r.plan.info()["num_prefill_seqs"] == 0
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, prefill=False)


@pytest.mark.parametrize("hq,tokens,d", [(1, 1, 64), (12, 1, 64), (8, 1, 128), (8, 1, 256), (64, 1, 64), (64, 1, 128), (32, 1, 256)])
@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 26 * 1.1, 2.0 ** 28 * 1.3, 2.0 ** 33])
def test_scores_whose_steps_pass_f16(hq, tokens, d, top):
    """Logits so large that fp32 holds them in steps of many: the largest key
    takes the row."""
    n, kv = 5, 300
    b = batch([tokens] * n, [kv] * n, hq, 1, d, 16, seed=6)
    k = np.zeros(b.k_fp4.shape[:3] + (d,))
    for s in range(n):
        for key in range(kv):                        # a third below the largest, or more
            page, at = slot(b, s, key)
            k[page, 0, at, 0] = [0.5, 1, 1.5, 2, 3, 4][key * 7 % 6]
            k[page, 0, at, 1] = 6.0                  # the block's scale is one
        page, at = slot(b, s, 37 * s + 5)
        k[page, 0, at, 0] = 6.0
    q = np.zeros(b.q.shape, np.float32)
    q[..., 0] = 1.0
    b.q = oracle.round_bf16(q)
    b.k_fp4, b.k_fp4_scale = workloads.kv4_encode(k)
    b.sm_scale = top / 6
    out = Kv4Batch(b).call().float().cpu().numpy()
    v = oracle.kv4_pool(b.v_fp4, b.v_fp4_scale)
    for s in range(n):
        page, at = slot(b, s, 37 * s + 5)
        want = np.broadcast_to(v[page, at, 0], out[s].shape)
        assert (np.abs(out[s] - want) <= 2.0 ** -8 * np.abs(want)).all()


# ---------------------------------------------------------------- lengths

@pytest.mark.parametrize("ql,kv", [([1, 1], [100, 50]), ([3, 1], [700, 60]), ([30, 17], [200, 90]), ([200], [300]),
                                   ([1, 200], [90, 300])])
def test_lengths_that_disagree_with_the_plan(ql, kv):
    """Device lengths other than the plan's set the error word, on whichever
    kernel: a step that the table build refused (no new token, the lengths as
    before), keys more or fewer, tokens fewer."""
    b = batch(ql, kv, 4, 2, 128, 16, seed=7, max_pages_per_seq=max(kv) // 16 + 2)
    r = Kv4Batch(b)
    db = r.db
    good = r.call().clone()
    assert binding.rpa_get_device_error(r.ws) == 0
    cu, lens = b.cu_q_lens.copy(), b.kv_lens.copy()
    last = np.zeros_like(lens)
    last[-1] = 1
    for new_cu, new_lens in ((0 * cu, lens - np.diff(cu)), (cu, lens + last), (cu, lens - last),
                             (np.concatenate([cu[:-1], cu[-1:] - 1]), lens - last),
                             (np.concatenate([cu[:-1], cu[-1:] - 1]), lens)):
        db.cu_q_lens.copy_(cuda(new_cu.astype(np.int32)))
        db.kv_lens.copy_(cuda(new_lens.astype(np.int32)))
        r.call()
        assert binding.rpa_get_device_error(r.ws) == binding.RPA_DEVERR_LENGTHS, (new_cu, new_lens)
    db.cu_q_lens.copy_(cuda(cu))
    db.kv_lens.copy_(cuda(lens))
    assert torch.equal(r.call(), good) and binding.rpa_get_device_error(r.ws) == 0


@pytest.mark.parametrize("ql,kv", [([200], [300]), ([1, 200], [90, 300]), ([5, 3], [90, 40])])
def test_device_lengths_past_the_plans_rows(ql, kv):
    """Device lengths that name rows behind the plan's, or before them: reported,
    and nothing is written there."""
    b = batch(ql, kv, 4, 2, 128, 16, seed=7, max_pages_per_seq=max(kv) // 16 + 2)
    r = Kv4Batch(b)
    q = torch.cat([r.db.q, r.db.q])
    out = torch.full_like(q, 3.0)
    cu, n = b.cu_q_lens, int(b.cu_q_lens[-1])
    last = np.zeros_like(cu)
    last[-1] = 1
    for moved in (cu + last, cu + 1, cu - 300):
        binding.rpa_forward_kv4(q, *r.pool, r.db.page_table, cuda(moved), cuda(b.kv_lens + last[1:]), None, b.sm_scale,
                                out, r.plan, r.ws)
        assert binding.rpa_get_device_error(r.ws) == binding.RPA_DEVERR_LENGTHS
        assert bool((out[n:] == 3.0).all())


def test_many_tiles_are_all_looked_at():
    """Every sequence's lengths, whichever CTA works on it."""
    b = batch([1] * 900, [20 + i % 40 for i in range(900)], 2, 2, 64, 16, seed=8)
    r = Kv4Batch(b)
    r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    for s in (0, 151, 152, 500, 863, 864, 899):
        r.db.kv_lens[s] += 1
        r.call()
        assert binding.rpa_get_device_error(r.ws) == binding.RPA_DEVERR_LENGTHS, s
        r.db.kv_lens[s] -= 1


# ---------------------------------------------------------------- logit scales

@pytest.mark.parametrize("scale", [0.0, -0.0, -0.125, -40.0])
def test_scales_of_zero_and_below(scale):
    """sm_scale is any number: the same on every kernel."""
    b = batch([1, 6, 33, 200], [90, 300, 100, 260], 2, 1, 128, 16, [0, 4, 0, 50], seed=9)
    b.sm_scale = scale
    k, v = oracle.kv4_pool(b.k_fp4, b.k_fp4_scale), oracle.kv4_pool(b.v_fp4, b.v_fp4_scale)
    q = oracle.bf16_bits_to_f32(b.q)
    meta = (b.page_table, b.cu_q_lens, b.kv_lens, b.window, b.sm_scale)
    ref = oracle.attention(q, k, v, *meta, precision=64)
    mag = oracle.attention(q, k, np.abs(v), *meta, precision=64)
    kmax = np.sqrt((k.astype(np.float64) ** 2).sum(-1).max())
    qn = np.sqrt((q.reshape(-1, 128).astype(np.float64) ** 2).sum(-1))[:, None]
    # The module's terms; the exponential's and the logit scale's rounding grow
    # with the scores, which |q| |k| |scale| bounds.
    ds = (128 + 2) * 2.0 ** -23 * abs(scale) * qn * kmax + 2.0 ** -21 * abs(scale) * qn * kmax
    r = Kv4Batch(b)
    info = r.plan.info()
    assert info["num_decode_seqs"] > 0 and info["num_prefill_seqs"] > 0
    got = r.call().float().cpu().numpy().reshape(-1, 128).astype(np.float64)
    assert binding.rpa_get_device_error(r.ws) == 0
    # A probability p of the largest that f16 holds as a subnormal is off by half
    # its step, 2^-25 over the largest's 2^10: 2^-35 of the largest, of at most 300
    # keys.  (At -40 a row's second key can have 2^-200 of the first, which is zero
    # in fp32 already; where the first key's value is zero the relative terms alone
    # would ask for it.)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * ds + 2.0 ** -16) * mag + 300 * 2.0 ** -35 * np.abs(v).max()
    assert (np.abs(got - ref) <= bound).all()


# ---------------------------------------------------------------- the binding

def test_refusals_of_tensors_too_small_for_the_plan():
    """Each tensor that the kernels index by sequence or by row."""
    b = batch([1, 200, 3], [40, 300, 70], 4, 2, 64, 16, [0, 9, 0], seed=3)
    r = Kv4Batch(b)
    db = r.db
    good = dict(q=db.q, page_table=db.page_table, cu_q_lens=db.cu_q_lens, kv_lens=db.kv_lens, window=db.window, out=r.out)

    def call(**changed):
        a = {**good, **changed}
        binding.rpa_forward_kv4(a["q"], *r.pool, a["page_table"], a["cu_q_lens"], a["kv_lens"], a["window"], b.sm_scale,
                                a["out"], r.plan, r.ws)
    call()
    wide = torch.cat([db.page_table, db.page_table], 1)        # rows of another length
    for changed in (dict(cu_q_lens=db.cu_q_lens[:3]), dict(kv_lens=db.kv_lens[:2]), dict(window=db.window[:2]),
                    dict(page_table=wide), dict(page_table=db.page_table[:2]), dict(page_table=db.page_table.view(-1)[:-1]),
                    dict(q=db.q[:203]), dict(out=r.out[:203]), dict(q=db.q.view(-1, 2, 128)),
                    dict(out=r.out.view(-1, 8, 32))):
        with pytest.raises(ValueError):
            call(**changed)
    # More than the plan has is no matter, nor are rows laid out flat.
    call(q=db.q.view(204, -1), out=r.out.view(-1), page_table=db.page_table.view(-1))
    call(cu_q_lens=torch.cat([db.cu_q_lens, db.cu_q_lens]), kv_lens=torch.cat([db.kv_lens, db.kv_lens]),
         page_table=torch.cat([db.page_table, db.page_table]))
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, r.out)


def test_a_prepared_call():
    """ForwardKv4Call: marshalled once, run again, under another plan of the
    same tensors; plans that they are too small for are refused."""
    b = batch([1, 5, 200], [400, 30, 300], 4, 2, 128, 16, seed=4)
    r = Kv4Batch(b)
    want = r.call().clone()
    db = r.db
    one = binding.rpa_plan(b.cu_q_lens, b.kv_lens, None, 4, 2, 128, 16, b.max_pages_per_seq, b.num_pages, num_sms=3,
                           kv_dtype=binding.RPA_DTYPE_FP4_E2M1)
    ws = torch.zeros(max(r.plan.workspace_bytes, one.workspace_bytes), dtype=torch.uint8, device="cuda")
    call = binding.ForwardKv4Call(db.q, *r.pool, db.page_table, db.cu_q_lens, db.kv_lens, None, b.sm_scale, r.out, r.plan, ws)
    for plan in (None, one, r.plan):
        r.out.fill_(float("nan"))
        call() if plan is None else call(plan)
        check(b, r.out)
    assert torch.equal(r.out, want) and binding.rpa_get_device_error(ws) == 0
    big = np.array([0, 1, 6, 206 + 1], np.int32)
    for cu, width, pages in ((big, b.max_pages_per_seq, b.num_pages), (b.cu_q_lens, b.max_pages_per_seq + 1, b.num_pages),
                             (b.cu_q_lens, b.max_pages_per_seq, b.num_pages + 1)):
        plan = binding.rpa_plan(cu, b.kv_lens, None, 4, 2, 128, 16, width, pages, kv_dtype=binding.RPA_DTYPE_FP4_E2M1)
        with pytest.raises(ValueError):
            call(plan)


# ---------------------------------------------------------------- each kernel's own bound

def run_and_check(b, **plan_kw):
    """The bound of the kernels that ran, and the same bits twice."""
    r = Kv4Batch(b, **plan_kw)
    out = r.call().clone()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, prefill=r.plan.info()["num_prefill_seqs"] > 0)
    assert torch.equal(r.call(), out)


@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_tokens_within_the_split_kernels_bound(case):
    ql, kv, hq, hkv, d, p, win = FEW[case]
    run_and_check(batch(ql, kv, hq, hkv, d, p, win, seed=340 + case))


@pytest.mark.parametrize("case", range(len(ROWS)))
def test_tens_of_rows_within_the_split_kernels_bound(case):
    ql, kv, hq, hkv, d, p, win = ROWS[case]
    run_and_check(batch(ql, kv, hq, hkv, d, p, win, seed=700 + case))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [3, 7, 14, 30])
def test_small_windows_within_the_split_kernels_bound(d, tokens):
    kv = [tokens + 20 + 5 * i for i in range(24)] + [1312]
    b = batch([tokens] * 25, kv, 1, 1, d, 16, [17, 2, 5, 33, 9] * 5, seed=800 + tokens)
    for kw in ({}, {"num_sms": 1}):
        run_and_check(b, **kw)


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(seed):
    """Heads, dimensions, pages, windows, lengths, SMs and their split drawn."""
    rng = np.random.default_rng(5000 + seed)
    pick = lambda *a: a[int(rng.integers(len(a)))]
    d, p, hkv = pick(64, 128, 256), pick(16, 32, 64, 128, 256), pick(1, 1, 2, 3, 8)
    group = pick(1, 2, 3, 4, 7, 8, 16, 40)
    n = int(rng.integers(1, 25))
    ql, kv = [], []
    for _ in range(n):
        q = pick(0, 1, 1, 1, 2, int(rng.integers(2, 17)), int(rng.integers(17, 200)))
        ql.append(q)
        kv.append(q + pick(0, int(rng.integers(0, 40)), int(rng.integers(0, 700)), int(rng.integers(0, 3000))))
    if not any(ql):
        ql[0], kv[0] = 1, kv[0] + 1
    win = pick(None, [int(rng.integers(0, 90)) for _ in range(n)], [pick(0, 1, 500) for _ in range(n)])
    run_and_check(batch(ql, kv, hkv * group, hkv, d, p, win, seed=seed), num_sms=pick(0, 0, 1, 7, 40),
                  decode_sms=pick(0, 0, -1))


# ---------------------------------------------------------------- at once

def test_calls_at_once():
    """Mixed batches from several host threads, and from one thread on two
    streams in turn, each with a workspace of its own: the bits of calls made
    one at a time.  One of them holds NaN, the others' headers do not hear of it."""
    runs = []
    for i in range(4):
        n = 30 + 7 * i
        kv = [40 + 61 * j % 900 for j in range(n)]
        ql = [1] * (n - 3) + [7, 150 + i, 20]
        kv[-3:] = [400, 500, 300]
        b = batch(ql, kv, 8, 2, 128, 16, [0] * n if i % 2 else [j % 3 * 50 for j in range(n)], seed=60 + i)
        if i == 2:
            for s in (3, n - 2):
                page, at = slot(b, s, kv[s] - 1)
                b.v_fp4_scale[page, 0, at, 2] = 255
        runs.append(Kv4Batch(b, decode_sms=20 if i != 1 else -1))
    want = [r.call().clone() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    errors = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(20):
                runs[i].call(stream=streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    def same():
        torch.cuda.synchronize()
        assert not errors, errors
        for i, r in enumerate(runs):
            assert binding.rpa_get_device_error(r.ws) == 0 and bool((r.ws[:256] == 0).all())
            assert torch.equal(r.out.view(torch.int16), want[i].view(torch.int16)), i
            r.out.zero_()
        torch.cuda.synchronize()
    for r in runs:
        r.out.zero_()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    same()
    for _ in range(10):
        for i in range(4):
            runs[i].call(stream=streams[i])
    same()
