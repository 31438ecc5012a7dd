"""The order of a mixed batch's two parts on two streams (fork_join.h): whatever
fails from the fork on, the side stream is joined, and the first error returned.
Steps that note themselves stand in for the CUDA calls: nothing here needs a GPU."""

from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from ragged_paged_attention_rpa_gb300 import build

FORK, THERE, MARK, HERE, JOIN = (1 << i for i in range(5))


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("fork") / "libforkjoin.so")
    src = os.path.join(os.path.dirname(__file__), "csrc", "fork_join_check.cpp")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I" + build.CSRC, "-o", lib, src], check=True)
    f = ctypes.CDLL(lib).fork_join_check

    def call(fails):
        order = ctypes.create_string_buffer(16)
        err = f(ctypes.c_uint(fails), order)
        return err, order.value.decode()
    return call


@pytest.mark.parametrize("fails,err,order", [
    (0, 0, "ftmhj"),
    (FORK, 10, "f"),                  # nothing on the side stream yet
    (THERE, 11, "ftmj"),              # what it had enqueued is waited for
    (HERE, 13, "ftmhj"),
    (MARK, 12, "ftm"),                # no event to wait for
    (JOIN, 14, "ftmhj"),
    (THERE | MARK, 11, "ftm"),
    (THERE | JOIN, 11, "ftmj"),
    (HERE | JOIN, 13, "ftmhj"),
])
def test_order_and_error(run, fails, err, order):
    assert run(fails) == (err, order)
