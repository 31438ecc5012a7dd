"""The 4-bit KV format on the CPU (its definition, restated and pinned) and the
host checks of the entry points that use it: nothing here needs a GPU."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import oracle
from ragged_paged_attention_rpa_gb300 import binding, build, workloads
from ragged_paged_attention_rpa_gb300.binding import (RPA_DTYPE_FP4_E2M1, RPA_ERR_INVALID_ARG,
                                                      RPA_ERR_PLAN_MISMATCH, RPA_ERR_UNSUPPORTED,
                                                      RPA_ERR_WORKSPACE_TOO_SMALL, RpaError)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def held(x):
    x = np.asarray(x, dtype=np.float64)
    return oracle.decode_kv4(*workloads.kv4_encode(x)).astype(np.float64)


def test_scales_are_half_precision_bits():
    """A scale byte is the upper half of an f16's bits, shifted right by 7."""
    b = np.arange(0xE3, dtype=np.uint16)
    assert np.array_equal((b << 7).view(np.float16).astype(np.float64), workloads.KV4_SCALES)
    assert np.isnan(np.array([255 << 7], np.uint16).view(np.float16))[0]


def test_every_code_times_every_scale_is_exact_in_f16_and_bf16():
    v = np.multiply.outer(workloads.E2M1, workloads.KV4_SCALES)
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    assert np.array_equal(oracle.bf16_bits_to_f32(oracle.round_bf16(v.astype(np.float32))).astype(np.float64), v)


def test_exact_blocks_come_back():
    for s in (2.0 ** -14, 0.4375, 1.0, 13.0, 10240.0):
        x = np.concatenate([workloads.E2M1, -workloads.E2M1]) * s
        assert np.array_equal(held(x), x)


def test_ties_saturation_and_zero():
    x = np.zeros(16)
    x[:8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]   # scale 1; each other a midpoint
    assert held(x)[:8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]
    assert np.array_equal(held(np.zeros(32)), np.zeros(32))
    x = np.full(16, 1e6)
    assert np.array_equal(held(x), np.full(16, 61440.0))
    # amax / 6 = 1.0625, the midpoint of 1 and 1.125: scale 1, the largest code.
    assert np.array_equal(held(np.full(16, 6.375)), np.full(16, 6.0))
    assert np.array_equal(held(np.full(16, 6 * 2.0 ** -18)), np.zeros(16))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_with_a_bad_value_reads_as_nan(bad):
    x = np.ones(48)
    x[20] = bad
    got = held(x)
    assert np.isnan(got[16:32]).all() and np.isfinite(np.delete(got, np.s_[16:32])).all()


def test_error_of_a_block():
    """An element is off by at most half the widest code step of its scale (one
    scale), plus what the largest code cannot reach: scale off by at most 1/16
    of itself, so max|x| <= 6.375 scales."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((500, 64)) * np.exp2(rng.integers(-9, 9, (500, 1)))
    codes, scales = workloads.kv4_encode(x)
    s = np.repeat(workloads.KV4_SCALES[scales], 16, -1)
    assert (np.abs(oracle.decode_kv4(codes, scales) - x) <= s * (1 + 1e-12)).all()


def plan_of(ql=(1, 1), kv=(40, 9), hq=8, hkv=1, d=128, p=16, win=None, mpps=8, **kw):
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    return binding.rpa_plan(cu, np.array(kv, np.int32), win, hq, hkv, d, p, mpps, 64, num_sms=152,
                            **{"kv_dtype": RPA_DTYPE_FP4_E2M1, **kw})


def test_plan_reports_its_pages():
    info = plan_of((1, 3, 60), (40, 9, 100)).info()
    assert info["kv_dtype"] == RPA_DTYPE_FP4_E2M1 and info["path"] == binding.RPA_PATH_TC
    assert info["num_decode_seqs"] + info["num_prefill_seqs"] == 3
    assert info["num_prefill_seqs"] >= 1 and info["num_prefill_items"] >= 1
    # The workspace holds the prompt's visible pages widened to bf16.
    assert info["workspace_bytes"] >= 2 * 7 * 16 * 128 * 2


def test_plan_refuses_what_4_bit_pages_do_not_take():
    for kw in ({"dtype": binding.RPA_DTYPE_F32}, {"path": binding.RPA_PATH_SIMT}, {"p": 8, "mpps": 13},
               {"kv_split": 64}, {"decode_kernel": 1},
               {"prefill_pairs": 2}, {"prefill_split": 2}, {"q_block": 32},
               {"hq": 256, "hkv": 1}):
        with pytest.raises(RpaError) as e:
            plan_of((1, 60), (40, 100), **kw)
        assert e.value.status == RPA_ERR_UNSUPPORTED, kw
    with pytest.raises(RpaError) as e:
        plan_of(kv_dtype=4)
    assert e.value.status == RPA_ERR_INVALID_ARG
    assert plan_of((0, 0), (3, 0)).info()["workspace_bytes"] == 256


def addr(x):
    return ctypes.c_void_p(x)


FAKE, WS = addr(1 << 20), addr(1 << 21)


def changed(args, **at):
    out = list(args)
    for k, v in at.items():
        out[int(k[1:])] = v
    return out


def test_forward_kv4_checks_before_any_launch():
    L = binding.lib()
    p = plan_of()
    ok = [FAKE] * 8 + [2, 8, 1, 128, 16, None, 0.1, FAKE, None, p.handle, WS, p.workspace_bytes]
    f = L.rpa_forward_kv4
    assert f(*changed(ok, _17=None)) == RPA_ERR_INVALID_ARG
    for i in (8, 9, 10, 11, 12):
        assert f(*changed(ok, **{"_%d" % i: 3})) == RPA_ERR_PLAN_MISMATCH
    assert f(*changed(ok, _13=FAKE)) == RPA_ERR_PLAN_MISMATCH      # a window the plan has not
    assert f(*changed(ok, _18=addr((1 << 21) + 16))) == RPA_ERR_INVALID_ARG
    assert f(*changed(ok, _19=255)) == RPA_ERR_WORKSPACE_TOO_SMALL
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 15):
        assert f(*changed(ok, **{"_%d" % i: None})) == RPA_ERR_INVALID_ARG
        off = 8 if i in (0, 1, 2, 3, 4, 15) else 2
        assert f(*changed(ok, **{"_%d" % i: addr((1 << 20) + off)})) == RPA_ERR_INVALID_ARG
    # A bf16 plan, and this plan with the other entry points.
    other = plan_of(kv_dtype=0)
    assert f(*changed(ok, _17=other.handle, _19=1 << 24)) == RPA_ERR_PLAN_MISMATCH
    meta = [2, 8, 1, 128, 16, None, 0.1, FAKE, None, p.handle]
    assert L.rpa_forward(*[FAKE] * 6, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward_kv(*[FAKE] * 8, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward_fp8kv(*[FAKE] * 8, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward_decode_noalloc(*[FAKE] * 6, *meta) == RPA_ERR_PLAN_MISMATCH
    norm = binding.QkvNorm(None, None, None, 1e-6, 1e4)
    assert L.rpa_forward_qkv(*[FAKE] * 3, ctypes.byref(norm), *[FAKE] * 6, *meta, WS, 1 << 24) \
        == RPA_ERR_PLAN_MISMATCH


@pytest.mark.parametrize("name", ["rpa_write_kv4", "rpa_read_kv4"])
def test_cache_calls_check_before_any_launch(name):
    f = getattr(binding.lib(), name)
    ok = [FAKE] * 7 + [4, 2, 128, 16, 8, binding.RPA_DTYPE_BF16, None, None]
    for i, v, want in ((7, -1, RPA_ERR_INVALID_ARG), (8, 0, RPA_ERR_INVALID_ARG),
                       (9, 96, RPA_ERR_UNSUPPORTED), (9, 0, RPA_ERR_INVALID_ARG),
                       (10, 24, RPA_ERR_INVALID_ARG), (10, 8, RPA_ERR_UNSUPPORTED),
                       (10, 512, RPA_ERR_UNSUPPORTED), (11, 0, RPA_ERR_INVALID_ARG),
                       (12, binding.RPA_DTYPE_FP8_E4M3, RPA_ERR_INVALID_ARG),
                       (13, addr((1 << 21) + 16), RPA_ERR_INVALID_ARG)):
        assert f(*changed(ok, **{"_%d" % i: v})) == want, (i, v)
    for i in range(7):
        assert f(*changed(ok, **{"_%d" % i: None})) == RPA_ERR_INVALID_ARG
        assert f(*changed(ok, **{"_%d" % i: addr((1 << 20) + 4)})) == RPA_ERR_INVALID_ARG
    assert f(*changed([None] * 7 + ok[7:], _7=0)) == binding.RPA_OK   # no tokens, nothing to do


def test_table_calls_check_before_any_launch():
    L = binding.lib()
    a = [addr((1 << 20) + 4096 * i) for i in range(9)]
    build_ok = a + [4, 8, 16, 4, 32, WS, None]
    release_ok = a[:7] + [4, 16, 4, 32, WS, None]
    for f, ok, n, shape in ((L.rpa_build_tables, build_ok, 9, ((9, -1), (10, -1), (11, 12), (11, 0),
                                                               (12, 0), (13, 0))),
                            (L.rpa_release_tables, release_ok, 7, ((7, -1), (8, 12), (9, 0), (10, 0)))):
        for i, v in shape:
            assert f(*changed(ok, **{"_%d" % i: v})) == RPA_ERR_INVALID_ARG, (i, v)
        for i in range(n):
            assert f(*changed(ok, **{"_%d" % i: None})) == RPA_ERR_INVALID_ARG, i
            assert f(*changed(ok, **{"_%d" % i: addr(a[i].value + 2)})) == RPA_ERR_INVALID_ARG, i
        ws = len(ok) - 2
        assert f(*changed(ok, **{"_%d" % ws: None})) == RPA_ERR_INVALID_ARG
        assert f(*changed(ok, **{"_%d" % ws: addr((1 << 21) + 128)})) == RPA_ERR_INVALID_ARG
    # Sizes whose loop indices would leave 31 bits.
    most = (1 << 30) + 1
    for f, ok, sizes in ((L.rpa_build_tables, build_ok, (9, 10, 13)), (L.rpa_release_tables, release_ok, (7, 10))):
        kv = {"_5" if f is L.rpa_release_tables else "_6": addr(1 << 40)}  # apart from kv_lens_prev
        for i in sizes:
            assert f(*changed(ok, **kv, **{"_%d" % i: most})) == RPA_ERR_UNSUPPORTED, i
    # Lengths or the stack's height that overlap their inputs without being them.
    assert L.rpa_build_tables(*changed(build_ok, _6=addr(a[1].value + 4))) == RPA_ERR_INVALID_ARG
    assert L.rpa_release_tables(*changed(release_ok, _5=addr(a[1].value + 12))) == RPA_ERR_INVALID_ARG
