"""Drafted trees without a GPU: plans and the refusals of the five entry points, which
return before anything is enqueued."""

from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from ragged_paged_attention_rpa_gb300 import binding, build

INVALID, UNSUPPORTED = binding.RPA_ERR_INVALID_ARG, binding.RPA_ERR_UNSUPPORTED
A = 1 << 20  # an address that no check dereferences


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def plan(nodes=(8, 8), ctx=(100, 300), windows=None, hq=8, hkv=1, d=128, page=16, words=1, **kw):
    cu = np.concatenate([[0], np.cumsum(nodes)])
    kv = np.array(ctx) + nodes
    width = max(1, -(-int(kv.max()) // page)) if len(kv) else 1
    return binding.rpa_plan(cu, kv, windows, hq, hkv, d, page, width, 4096, tree_words=words,
                            **{"num_sms": 152, **kw})


def refused(status, fn, *args):
    with pytest.raises(binding.RpaError) as e:
        fn(*args)
    assert e.value.status == status


def test_plans():
    info = plan().info()
    assert info["path"] == binding.RPA_PATH_TC and info["num_decode_seqs"] == 2 and info["num_prefill_seqs"] == 0 and info["decode_kernel"] == 0
    assert plan(nodes=(0, 0)).workspace_bytes == 256
    assert plan(nodes=(), ctx=()).workspace_bytes == 256
    assert plan(dtype=binding.RPA_DTYPE_F32).info()["path"] == binding.RPA_PATH_SIMT
    assert plan(path=binding.RPA_PATH_SIMT).info()["path"] == binding.RPA_PATH_SIMT
    assert plan(page=8).info()["path"] == binding.RPA_PATH_SIMT
    assert plan(hq=130).info()["path"] == binding.RPA_PATH_SIMT
    assert plan(nodes=(64, 1)).info()["num_decode_seqs"] == 2
    assert plan(nodes=(1024, 0), words=16).info()["num_decode_seqs"] == 1


@pytest.mark.parametrize("kw,status", [
    (dict(words=17), INVALID), (dict(words=-1), INVALID), (dict(nodes=(65, 1)), INVALID), (dict(path=7), INVALID),
    (dict(q_block=16), UNSUPPORTED), (dict(kv_split=256), UNSUPPORTED), (dict(prefill_pairs=1), UNSUPPORTED),
    (dict(prefill_split=4), UNSUPPORTED), (dict(decode_sms=5), UNSUPPORTED), (dict(decode_kernel=1), UNSUPPORTED),
    (dict(prefill_dynamic=-1), UNSUPPORTED), (dict(prefill_grouping=-1), UNSUPPORTED),
    (dict(kv_dtype=binding.RPA_DTYPE_FP8_E4M3), UNSUPPORTED), (dict(kv_dtype=binding.RPA_DTYPE_FP4_E2M1), UNSUPPORTED),
    (dict(path=binding.RPA_PATH_TC, page=8), UNSUPPORTED), (dict(path=binding.RPA_PATH_TC, hq=130), UNSUPPORTED),
    (dict(path=binding.RPA_PATH_TC, dtype=binding.RPA_DTYPE_F32), UNSUPPORTED),
])
def test_plans_refused(kw, status):
    refused(status, lambda: plan(**kw))


def test_a_plan_serves_its_own_call_only():
    L = binding.lib()
    tree, flat = plan(), plan(words=0)
    ws = 1 << 21
    fwd = [A] * 6 + [2, 8, 1, 128, 16, None, 0.1, A, None, None, ws, 1 << 30]
    kvw = [A] * 8 + [2, 8, 1, 128, 16, None, 0.1, A, None, None, ws, 1 << 30]
    for fn, args, at in [(L.rpa_forward, fwd, 15), (L.rpa_forward_kv, kvw, 17), (L.rpa_forward_kv4, kvw, 17),
                         (L.rpa_forward_fp8kv, kvw, 17), (L.rpa_forward_decode_noalloc, fwd[:16], 15)]:
        args = list(args)
        args[at] = tree.handle
        assert fn(*args) == binding.RPA_ERR_PLAN_MISMATCH, fn
    norm = binding.QkvNorm(None, None, None, 1e-6, 1e4)
    qkv = [A] * 3 + [ctypes.byref(norm)] + [A] * 6 + [2, 8, 1, 128, 16, None, 0.1, A, None, tree.handle, ws, 1 << 30]
    assert L.rpa_forward_qkv(*qkv) == binding.RPA_ERR_PLAN_MISMATCH
    args = [A] * 8 + [2, 8, 1, 128, 16, None, 0.1, A, None, flat.handle, ws, 1 << 30]
    assert L.rpa_forward_tree(*args) == binding.RPA_ERR_PLAN_MISMATCH


def test_forward_tree_refusals():
    L, p = binding.lib(), plan(nodes=(64, 64), ctx=(5000, 900))
    good = [A] * 8 + [2, 8, 1, 128, 16, None, 0.1, A, None, p.handle, 1 << 21, p.workspace_bytes]

    def rc(at, value):
        args = list(good)
        args[at] = value
        return L.rpa_forward_tree(*args)

    for at, value in [(8, 3), (9, 16), (10, 2), (11, 64), (12, 32), (13, A)]:
        assert rc(at, value) == binding.RPA_ERR_PLAN_MISMATCH, at
    for at in (0, 1, 2, 3, 4, 5, 6, 15, 17, 18):
        assert rc(at, None) == INVALID, at
    for at, value in [(0, A + 8), (1, A + 64), (2, A + 16), (3, A + 2), (4, A + 1), (5, A + 2), (6, A + 4), (7, A + 2),
                      (15, A + 8), (18, (1 << 21) + 128)]:
        assert rc(at, value) == INVALID, at
    assert rc(19, p.workspace_bytes - 1) == binding.RPA_ERR_WORKSPACE_TOO_SMALL
    w = plan(windows=[0, 5])
    args = [A] * 7 + [None, 2, 8, 1, 128, 16, A, 0.1, A, None, w.handle, 1 << 21, w.workspace_bytes]
    assert L.rpa_forward_tree(*args) == INVALID  # a window without positions


def test_build_tree_refusals():
    L = binding.lib()
    good = [A] * 6 + [2, 16, 1, None, None]
    for at, value in [(0, None), (1, None), (2, None), (4, None), (5, None), (0, A + 1), (1, A + 2), (2, A + 2),
                      (3, A + 2), (4, A + 4), (5, A + 2), (6, -1), (7, -1), (8, 0), (8, 17), (9, A + 16)]:
        args = list(good)
        args[at] = value
        assert L.rpa_build_tree(*args) == INVALID, (at, value)
    assert L.rpa_build_tree(*([None] * 6 + [0, 0, 1, None, None])) == 0


def test_append_rope_refusals():
    L = binding.lib()
    rope = binding.Rope(A, 128, 0)
    # q, k, v, strides, positions, slots, rope, q_out, pages, scales, T, Hq, Hkv, D, P, N, dtype, kv_dtype, ws, stream
    far = 1 << 30
    good = [A, A, A, 1024, 128, 128, A, A, ctypes.byref(rope), far, far, far, None, None, 16, 8, 1, 128, 16, 64,
            binding.RPA_DTYPE_BF16, binding.RPA_DTYPE_BF16, None, None]

    def rc(**kw):
        args = list(good)
        for at, value in kw.items():
            args[int(at[1:])] = value
        return L.rpa_append_rope(*args)

    for at in (0, 1, 2, 6, 7, 8, 9, 10, 11):
        assert rc(**{"a%d" % at: None}) == INVALID, at
    for at, value in [(0, A + 8), (1, A + 8), (2, A + 8), (3, 1016), (3, 1028), (4, 120), (4, 132), (5, 127), (6, A + 2),
                      (7, A + 4), (9, far + 8), (10, far + 8), (11, far + 8), (12, A), (13, A), (14, -1), (15, -1),
                      (16, 0), (18, 0), (19, 0), (20, 5), (22, A + 64)]:
        assert rc(**{"a%d" % at: value}) == INVALID, (at, value)
    for at, value in [(17, 96), (18, 24), (21, binding.RPA_DTYPE_F32), (21, binding.RPA_DTYPE_FP4_E2M1), (16, 1 << 20)]:
        kw = {"a%d" % at: value}
        if at == 17:
            kw["a8"] = ctypes.byref(binding.Rope(A, 64, 0))
        assert rc(**kw) == UNSUPPORTED, (at, value)
    assert rc(a21=binding.RPA_DTYPE_FP8_E4M3) == INVALID              # e4m3 pages without scales
    for dims, status in [(144, INVALID), (-16, INVALID), (8, UNSUPPORTED), (24, UNSUPPORTED)]:
        assert rc(a8=ctypes.byref(binding.Rope(A, dims, 0))) == status, dims
    assert rc(a8=ctypes.byref(binding.Rope(None, 128, 0))) == INVALID
    # q_out over q in part, over k, over v; q in place at another stride.
    assert rc(a9=A + 16) == INVALID and rc(a0=far + 64) == INVALID
    assert rc(a1=far + 256) == INVALID and rc(a2=far + 16 * 2048 - 16) == INVALID
    assert rc(a9=A, a3=2048) == INVALID
    assert rc(a14=0) == 0


def test_commit_tree_refusals():
    L = binding.lib()
    good = [A] * 5 + [2, 16, 4, 1, 128, 16, 64, binding.RPA_DTYPE_BF16, None, None]
    for at, value in [(0, None), (1, None), (2, None), (3, None), (4, None), (0, A + 8), (1, A + 8), (2, A + 4),
                      (3, A + 2), (4, A + 2), (5, -1), (6, -1), (7, -1), (8, 0), (9, 0), (10, 24), (10, 0), (11, 0),
                      (12, 3), (12, 9), (13, A + 8)]:
        args = list(good)
        args[at] = value
        assert L.rpa_commit_tree(*args) == INVALID, (at, value)
    for at, value in [(7, 1025), (9, 12), (8, 1 << 20)]:
        args = list(good)
        args[at] = value
        assert L.rpa_commit_tree(*args) == UNSUPPORTED, (at, value)


def test_trim_tables_refusals():
    L = binding.lib()
    good = [A, A + 1024, A, A, A, A + 2048, A + 4096, 2, 16, 4, 64, 1 << 21, None]
    for at, value in [(0, None), (1, None), (2, None), (3, None), (4, None), (5, None), (6, None), (0, A + 1), (5, A + 2),
                      (7, -1), (8, 24), (8, 0), (9, 0), (10, 0), (11, None), (11, (1 << 21) + 8), (5, A + 1028)]:
        args = list(good)
        args[at] = value
        assert L.rpa_trim_tables(*args) == INVALID, (at, value)
    args = list(good)
    args[7] = (1 << 30) + 1
    args[5] = args[1]
    assert L.rpa_trim_tables(*args) == UNSUPPORTED


def test_schedules_cover_every_tile_once(tmp_path):
    """Random batches through the scheduler alone (tests/csrc/tree_plan_check.cpp)."""
    exe = str(tmp_path / "tree_plan_check")
    here = os.path.dirname(os.path.abspath(__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I" + build.INCLUDE, "-I" + build.CSRC, "-I" + cuda,
                    os.path.join(here, "csrc", "tree_plan_check.cpp"), os.path.join(build.CSRC, "plan_tree.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 3e38, -2.0 ** 121])
def test_scales_refused(scale):
    L, p = binding.lib(), plan(nodes=(64, 64), ctx=(5000, 900))
    args = [A] * 8 + [2, 8, 1, 128, 16, None, scale, A, None, p.handle, 1 << 21, p.workspace_bytes]
    assert L.rpa_forward_tree(*args) == INVALID
