"""Random steps of the page tables against their definition: requests, page
sizes, lengths and padding drawn, apart and in place."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build

from .test_gpu_tables import build_ref, cuda, need_of, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("seed", range(40))
def test_random_steps(seed):
    rng = np.random.default_rng(9000 + seed)
    pick = lambda *a: a[int(rng.integers(len(a)))]
    seqs, p = pick(1, 2, 7, 511, 512, 513, 2047, 2048, 2049, 4100), pick(1, 2, 16, 64, 256, 1024)
    few = seqs > 600
    new = rng.integers(0, pick(1, 2, 20 if few else 300) + 1, seqs).tolist()
    prev = rng.integers(0, pick(1, 40, 60 if few else 1000) + 1, seqs).tolist()
    table, free, count = state(new, prev, p, need_of(new, prev, p) + pick(0, 3), seed)
    room, in_place = sum(new) + pick(0, 1, 777), bool(rng.integers(2))
    want = build_ref(new, prev, table, free, count, p, room)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    t, f, c0, kv0 = cuda(table), cuda(free), cuda([count]), cuda(prev)
    kv, c1 = (kv0, c0) if in_place else (cuda([9] * seqs), cuda([9]))
    cu, slots = cuda([9] * (seqs + 1)), cuda([9] * room, np.int64)
    binding.rpa_build_tables(cuda(new), kv0, t, f, c0, cu, kv, slots, c1, p, ws)
    assert binding.rpa_get_device_error(ws) == 0
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert cu.tolist() == want[1] and kv.tolist() == want[2] and slots.tolist() == want[3] and c1.item() == want[4]
    # Some of them end: their pages come back in order.
    done = (rng.random(seqs) < 0.4).astype(np.int64)
    h, stack = want[4], free.copy()
    for s in np.nonzero(done)[0]:
        n = -(-want[2][s] // p)
        stack[h:h + n] = want[0][s, :n]
        h += n
    binding.rpa_release_tables(cuda(done), kv, t, f, c1, kv, c1, p, ws)
    assert binding.rpa_get_device_error(ws) == 0 and bool((ws == 0).all())
    assert np.array_equal(f.cpu().numpy(), stack) and c1.item() == h
    assert kv.tolist() == [0 if d else x for d, x in zip(done, want[2])]
