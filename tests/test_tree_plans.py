"""Plans for drafted trees that are refused for their lengths (no GPU)."""

from __future__ import annotations

import pytest

from ragged_paged_attention_rpa_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def plan(kv_lens, **kw):
    """Two requests of 4 nodes under a table of 2^23 pages of 256."""
    return binding.rpa_plan([0, 4, 8], kv_lens, kw.pop("windows", None), 8, 2, 128, 256, 1 << 23, 64, tree_words=1,
                            num_sms=152, **kw)


@pytest.mark.parametrize("path", [binding.RPA_PATH_AUTO, binding.RPA_PATH_SIMT])
@pytest.mark.parametrize("windows", [None, [5, 1 << 30]])
@pytest.mark.parametrize("dtype", [binding.RPA_DTYPE_BF16, binding.RPA_DTYPE_F32])
def test_lengths_that_32_bits_cannot_step_past(dtype, windows, path):
    """The kernels' loops over a request's keys end at up to 256 keys behind the last."""
    kw = dict(dtype=dtype, windows=windows, path=path)
    assert plan([100, (1 << 31) - 1024], **kw).info()["num_decode_seqs"] == 2
    for length in ((1 << 31) - 1023, (1 << 31) - 256, (1 << 31) - 1):
        for lens in ([length, 100], [100, length]):
            with pytest.raises(binding.RpaError) as e:
                plan(lens, **kw)
            assert e.value.status == binding.RPA_ERR_UNSUPPORTED
