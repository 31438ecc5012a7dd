"""Attention by a host plan over device lengths that are not its own: those of a
step that rpa_build_tables refused (no new tokens), and lengths that name rows
behind the plan's.  The call ends, says so where it looks, and writes nothing
behind the plan's rows."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def refused(b):
    """The device's lengths after a table build without pages for the step."""
    i32 = lambda a: torch.from_numpy(np.array(a, np.int32)).cuda()
    new = np.diff(b.cu_q_lens)
    cu, kv, count = i32(np.full(len(new) + 1, 9)), i32(b.kv_lens - new), i32([0])
    slots = torch.full((int(new.sum()),), 9, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.rpa_build_tables(i32(new), kv, i32(b.page_table), i32(np.zeros(b.num_pages)), count, cu, kv, slots, count,
                             b.page_size, ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGES
    assert not bool(cu.any()) and bool((slots == -1).all())
    return cu, kv


def forward(b, cu, kv, **plan_kw):
    db = binding.Batch(b)
    plan = db.plan(**plan_kw)
    ws = binding.alloc_workspace(plan)
    q = torch.cat([db.q, db.q])
    out = torch.full_like(q, 3.0)
    binding.rpa_forward(q, db.k_pages, db.v_pages, db.page_table, cu, kv, db.window, b.sm_scale, out, plan, ws)
    err = binding.rpa_get_device_error(ws)
    assert bool((out[b.q.shape[0]:] == 3.0).all())
    return err, out[:b.q.shape[0]]


CUDA_CORE = [
    # (q_lens, kv_lens, Hq, Hkv, D, P, dtype)
    ([1, 1], [40, 33], 4, 2, 64, 16, "f32"),
    ([5, 1, 30], [33, 49, 65], 4, 2, 128, 16, "f32"),
    ([3, 1, 20], [20, 9, 33], 4, 1, 64, 8, "bf16"),
]


@pytest.mark.parametrize("case", range(len(CUDA_CORE)))
def test_the_cuda_core_path_ends(case):
    ql, kv, hq, hkv, d, p, dtype = CUDA_CORE[case]
    b = workloads.make_batch(ql, kv, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=p, seed=case, dtype=dtype,
                             max_pages_per_seq=12)
    err, out = forward(b, *refused(b))
    assert err == binding.RPA_DEVERR_LENGTHS and bool((out == 3.0).all())
    db = binding.Batch(b)
    last = torch.zeros_like(db.cu_q_lens)
    last[-1] = 1
    for cu, lens in ((db.cu_q_lens - 300, db.kv_lens), (db.cu_q_lens + 2, db.kv_lens), (db.cu_q_lens, 0 * db.kv_lens),
                     (db.cu_q_lens.flip(0), db.kv_lens)):
        assert forward(b, cu, lens)[0] == binding.RPA_DEVERR_LENGTHS
    forward(b, db.cu_q_lens + last, db.kv_lens + last[1:])
    err, out = forward(b, db.cu_q_lens, db.kv_lens)
    assert err == 0 and bool(torch.isfinite(out).all()) and not bool((out == 3.0).all())


PREFILL = [
    # (q_lens, kv_lens, Hq, Hkv, D, P, plan options): the single-SM kernel, its
    # static lists and split items, SM pairs, beside decode
    ([200], [300], 4, 2, 64, 16, {}),
    ([200, 70], [300, 90], 8, 1, 256, 16, dict(prefill_dynamic=-1)),
    ([200], [1500], 4, 2, 128, 16, dict(prefill_split=2)),
    ([300, 33], [300, 33], 4, 1, 128, 16, dict(prefill_pairs=2)),
    ([1] * 5 + [150], [40 + 16 * i for i in range(5)] + [170], 8, 2, 128, 32, {}),
]


@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_the_tensor_core_prefill_stays_inside(case):
    ql, kv, hq, hkv, d, p, kw = PREFILL[case]
    b = workloads.make_batch(ql, kv, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=p, seed=10 + case,
                             max_pages_per_seq=max(kv) // p + 2)
    err, good = forward(b, *(lambda db: (db.cu_q_lens, db.kv_lens))(binding.Batch(b)), **kw)
    assert err == 0 and bool(torch.isfinite(good).all())
    new = np.diff(b.cu_q_lens)
    if any(-(-k // p) > -(-(k - n) // p) for k, n in zip(kv, new)):
        assert forward(b, *refused(b), **kw)[0] == binding.RPA_DEVERR_LENGTHS
    db = binding.Batch(b)
    last = torch.zeros_like(db.cu_q_lens)
    last[-1] = 1
    for cu, lens in ((db.cu_q_lens + last, db.kv_lens + last[1:]), (db.cu_q_lens + 1, db.kv_lens),
                     (db.cu_q_lens - 300, db.kv_lens)):
        assert forward(b, cu, lens, **kw)[0] == binding.RPA_DEVERR_LENGTHS
