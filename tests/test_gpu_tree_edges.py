"""Drafted trees at the edges of what their calls take: masks under windows, scales near zero, values
near the ends of their range, paths of requests whose lengths cannot be used.  The attention's bound is that of
test_gpu_tree.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build

from . import tree_reference as ref
from .test_gpu_tree import PATHS, Tree, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_any_mask_under_a_window(d, path, dtype):
    """The window bounds the context alone: a node sees the nodes of its mask however far back they lie."""
    rng = np.random.default_rng(d)
    nodes, ctx, windows = [130, 40, 70], [50, 0, 33], [2, 7, 1]
    b = ref.tree_batch(nodes, ctx, 6, 2, d, 16, windows, seed=d, sees=[rng.random((t, t)) < 0.2 for t in nodes],
                       dtype=dtype)
    b.pos[:] = np.concatenate([c + np.arange(t) for c, t in zip(ctx, nodes)])
    check(b, Tree(b).run(path=path))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-40, 2.0 ** -127, 2.0 ** -126, 2.0 ** -125])
def test_scales_near_zero(scale, path):
    """Scores of up to 2^125 that such a scale makes small, or nothing."""
    b = ref.tree_batch([9, 5], [12, 0], 8, 2, 64, 16, [0, 40], seed=3, scale=scale)
    b.q *= 2.0 ** 59
    b.k_pages *= 2.0 ** 59
    check(b, Tree(b).run(path=path))


def rising_scores(d, nodes, ctx, by, seed):
    """Scores (base 2) that rise from 0 to `by` along the keys, and positive values of about 1."""
    b = ref.tree_batch(nodes, ctx, 4, 1, d, 32, None, seed=seed, scale=0.5)
    b.q[:], b.k_pages[:] = 0, 0
    b.q[..., 0] = 2.8853900817779268   # 1 / (scale log2 e)
    for s, n in enumerate(b.kv):
        for key in range(n):
            page, i = ref.slot(b, s, key)
            b.k_pages[page, i, :, 0] = by * key / n
    b.v_pages = (1 + b.v_pages.abs() / 8).to(b.v_pages.dtype)
    return b


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("by", [0, 7, 15, 60])
@pytest.mark.parametrize("sms", [1, 0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_near_the_end_of_the_range(d, by, path, sms):
    """2^116 of them times 1500 keys stay below 2^128, whatever the scores do."""
    b = rising_scores(d, [20, 3], [1500, 700], by, 16)
    b.v_pages *= 2.0 ** 116
    check(b, Tree(b).run(path=path, num_sms=sms))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("by", [0, 15, 60])
@pytest.mark.parametrize("sms", [1, 0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_small_values(d, by, path, sms):
    b = rising_scores(d, [20, 3], [1500, 700], by, 17)
    b.v_pages *= 2.0 ** -116
    check(b, Tree(b).run(path=path, num_sms=sms))


def test_empty_paths_of_unusable_lengths_are_reported():
    pages = torch.arange(4 * 8 * 64, dtype=torch.float32).view(4, 8, 1, 64).cuda()
    slots = torch.arange(12, device="cuda")
    path = torch.tensor([[-1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    for cu, code in [([0, 6, 12], 0), ([0, 0, 0], 0), ([0, -6, 12], binding.RPA_DEVERR_LENGTHS),
                     ([0, 6, 13], binding.RPA_DEVERR_LENGTHS), ([0, 6, 5], binding.RPA_DEVERR_LENGTHS)]:
        k, v, ws = pages.clone(), -pages, torch.zeros(256, dtype=torch.uint8, device="cuda")
        binding.rpa_commit_tree(k, v, slots, torch.tensor(cu, dtype=torch.int32, device="cuda"), path, ws)
        assert binding.rpa_get_device_error(ws) == code, cu
        assert torch.equal(k, pages) and torch.equal(v, -pages)
