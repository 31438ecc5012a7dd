"""Attention over 4-bit pages where a user meets its edges: NaN that only some
rows see, probabilities far below a row's largest, lengths that disagree with
the plan, scales of zero and below.

Bounds are those of test_gpu_kv4.py, with the probabilities' own rounding: f16
(2^-11 of itself) on the split-KV kernels, bf16 (2^-8) where a prefill ran.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from ragged_paged_attention_rpa_gb300 import binding, build, workloads

from .test_gpu_kv4 import Kv4Batch, batch, check, cuda, reference

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
