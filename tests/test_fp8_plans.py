"""A plan for fp8 pages with the entry points of 16-bit ones: refused on the
host, before any launch."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

from ragged_paged_attention_rpa_gb300 import binding, build
from ragged_paged_attention_rpa_gb300.binding import RPA_ERR_PLAN_MISMATCH

FAKE, WS = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_entry_points_of_16_bit_pages_refuse_an_fp8_plan():
    """rpa_forward_kv would write bf16 rows into pages of half their size."""
    L = binding.lib()
    plan = binding.rpa_plan(np.array([0, 1, 2], np.int32), np.array([40, 9], np.int32), None, 8, 1, 128, 16, 8, 64,
                            num_sms=152, kv_dtype=binding.RPA_DTYPE_FP8_E4M3)
    meta = [2, 8, 1, 128, 16, None, 0.1, FAKE, None, plan.handle]
    norm = binding.QkvNorm(None, None, None, 1e-6, 1e4)
    assert L.rpa_forward_kv(*[FAKE] * 8, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward(*[FAKE] * 6, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward_qkv(*[FAKE] * 3, ctypes.byref(norm), *[FAKE] * 6, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward_kv4(*[FAKE] * 8, *meta, WS, 1 << 24) == RPA_ERR_PLAN_MISMATCH
    assert L.rpa_forward_decode_noalloc(*[FAKE] * 6, *meta) == RPA_ERR_PLAN_MISMATCH
