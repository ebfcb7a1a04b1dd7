"""How many rows a call of kv_store_q4 takes: up to 2^34 values, where its header says."""
import ctypes
import os
import re

import pytest

from paged_attention_int8_gb300 import _lib, build as pkg_build


@pytest.mark.parametrize("hk,d", [(1, 64), (8, 128), (2, 256)])
def test_the_limit_is_refused(hk, d):
    pkg_build.build()
    lib, p = _lib.load(), ctypes.c_void_p(16)
    n = (1 << 34) // (hk * d)
    assert lib.pa_kv_store_q4(p, hk * d, p, hk * d, p, n, hk, d, p, p, p, p, 4, 16, None, None) \
        == _lib.Status.UNSUPPORTED
    assert "2^34" in lib.pa_last_error().decode()


def test_the_limit_is_the_documented_one():
    """(A call just below it would hold 64 GB: the check's own text.)"""
    with open(os.path.join(pkg_build.CSRC, "api.cu")) as f:
        body = f.read().split("pa_status pa_kv_store_q4(")[1].split("split the tokens")[0]
    assert re.search(r"num_tokens\) \* num_kv_heads >= \(int64_t\{1\} << 34\) / head_dim\)", body)
    with open(os.path.join(pkg_build.INCLUDE, "paq8.h")) as f:
        assert "num_tokens * num_kv_heads * head_dim below 2^34" in f.read()
