"""More KV heads than the tensor-core work lists hold (they keep a head in eight
bits): such batches run on the CUDA-core path, prompts over 4-bit pages are
refused, and single tokens over them run as ever."""

from __future__ import annotations

import numpy as np
import pytest

from ragged_paged_attention_rpa_gb300 import binding, build, workloads
from ragged_paged_attention_rpa_gb300.binding import RPA_ERR_UNSUPPORTED, RPA_PATH_SIMT, RPA_PATH_TC, RpaError


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def plan_of(ql, kv, hkv, **kw):
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    return binding.rpa_plan(cu, np.array(kv, np.int32), None, hkv, hkv, 64, 16, 16, 64, num_sms=152, **kw)


@pytest.mark.parametrize("hkv,path", [(256, RPA_PATH_TC), (257, RPA_PATH_SIMT), (600, RPA_PATH_SIMT)])
def test_the_path_of_a_plan(hkv, path):
    for ql, kv in (([1, 1], [40, 9]), ([20], [30]), ([1, 20], [9, 30])):
        assert plan_of(ql, kv, hkv).info()["path"] == path
        if path == RPA_PATH_SIMT:
            with pytest.raises(RpaError) as e:
                plan_of(ql, kv, hkv, path=RPA_PATH_TC)
            assert e.value.status == RPA_ERR_UNSUPPORTED


def test_prompts_over_4_bit_pages_are_refused():
    kw = dict(kv_dtype=binding.RPA_DTYPE_FP4_E2M1)
    assert plan_of([129, 1], [129, 40], 256, **kw).info()["num_prefill_seqs"] == 1
    with pytest.raises(RpaError) as e:
        plan_of([129, 1], [129, 40], 257, **kw)
    assert e.value.status == RPA_ERR_UNSUPPORTED
    assert plan_of([1, 3], [90, 40], 257, **kw).info()["num_prefill_seqs"] == 0


@pytest.mark.gpu
def test_against_the_oracle():
    from .test_gpu_kv4 import Kv4Batch, batch, check
    from .test_gpu_parity import assert_bf16_close, oracle_rows, run_gpu
    b = workloads.make_batch([1, 5, 1], [70, 33, 9], num_q_heads=300, num_kv_heads=300, head_dim=64, page_size=16, seed=2)
    got, err, _ = run_gpu(b)
    assert err == 0
    assert_bf16_close(got, oracle_rows(b))
    b = batch([1, 5, 1], [70, 33, 9], 300, 300, 64, 16, seed=3)
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, prefill=False)
