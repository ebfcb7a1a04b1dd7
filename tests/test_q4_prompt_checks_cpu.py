"""The entries of the 4-bit cache, of the read-back and of prompt_attention without a GPU:
what they refuse on the host, their no-ops, and the sizes of their workspaces."""
import ctypes

import pytest
import torch

from paged_attention_int8_gb300 import _lib, build as pkg_build

BAD, NOT = _lib.Status.INVALID_ARG, _lib.Status.UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return _lib.load()


def _values(defaults, kw, floats=()):
    """The call's arguments in order: pointers (16 or None) by their lower-case p_ names."""
    assert set(kw) <= set(defaults)
    out = []
    for name, x in {**defaults, **kw}.items():
        if name.startswith("p_"):
            out.append(None if x is None else ctypes.c_void_p(x))
        else:
            out.append(ctypes.c_float(x) if name in floats else x)
    return out


STORE = dict(p_key=16, kstride=256, p_value=16, vstride=256, p_slots=16, n=4, hk=2, d=128, p_kc=16,
             p_ks=16, p_vc=16, p_vs=16, nb=4, bs=16, p_status=None, p_stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(p_key=None), BAD), (dict(p_value=None), BAD), (dict(p_slots=None), BAD),
    (dict(p_kc=None), BAD), (dict(p_vs=None), BAD), (dict(n=-1), BAD), (dict(hk=0), BAD),
    (dict(nb=0), BAD), (dict(kstride=255), BAD), (dict(vstride=128), BAD), (dict(kstride=260), BAD),
    (dict(p_key=24), BAD), (dict(p_value=8), BAD), (dict(p_ks=8), BAD), (dict(p_slots=20), BAD),
    (dict(p_status=18), BAD), (dict(d=96), NOT), (dict(bs=64), NOT), (dict(nb=1 << 23), NOT),
    (dict(n=1 << 27), NOT),
])
def test_store_refuses(lib, kw, expect):
    assert lib.pa_kv_store_q4(*_values(STORE, kw)) == expect
    assert lib.pa_last_error().decode()


def test_store_of_no_tokens_is_a_no_op(lib):
    assert lib.pa_kv_store_q4(*_values(STORE, dict(n=0, p_key=None, p_slots=None))) == _lib.Status.OK


LOAD = dict(p_key=16, kstride=256, p_value=16, vstride=256, p_cu=16, p_lens=None, S=2, n=40,
            p_table=16, tstride=8, columns=8, hk=2, d=128, p_a=16, p_b=16, p_c=16, p_e=16, nb=16,
            bs=16, p_status=None, p_stream=None)


@pytest.mark.parametrize("name", ["pa_kv_load", "pa_kv_load_f8v4", "pa_kv_load_q4"])
@pytest.mark.parametrize("kw,expect", [
    (dict(p_key=None), BAD), (dict(p_value=None), BAD), (dict(p_cu=None), BAD),
    (dict(p_table=None), BAD), (dict(p_a=None), BAD), (dict(p_e=None), BAD), (dict(S=-1), BAD),
    (dict(n=-1), BAD), (dict(columns=0), BAD), (dict(columns=9), BAD), (dict(tstride=-8, columns=8), BAD),
    (dict(kstride=248), BAD), (dict(vstride=260), BAD), (dict(p_value=24), BAD), (dict(p_b=4), BAD),
    (dict(p_cu=18), BAD), (dict(p_lens=17), BAD), (dict(p_table=18), BAD), (dict(p_status=2), BAD),
    (dict(d=32), NOT), (dict(bs=8), NOT), (dict(nb=1 << 23), NOT), (dict(n=(1 << 31) - 2), NOT),
])
def test_load_refuses(lib, name, kw, expect):
    assert getattr(lib, name)(*_values(LOAD, kw)) == expect
    assert lib.pa_last_error().decode()


@pytest.mark.parametrize("name", ["pa_kv_load", "pa_kv_load_f8v4", "pa_kv_load_q4"])
@pytest.mark.parametrize("kw", [dict(S=0), dict(n=0, p_key=None)])
def test_load_of_nothing_is_a_no_op(lib, name, kw):
    assert getattr(lib, name)(*_values(LOAD, kw)) == _lib.Status.OK


ATTN = dict(p_q=16, p_kc=16, p_ks=16, p_vc=16, p_vs=16, p_cu=16, p_lens=16, p_table=16, tstride=8,
            columns=8, S=2, T=2, hq=8, hk=2, d=128, nb=16, bs=16, mq=1, ms=100, scale=0.1, ns=1,
            p_sinks=None, window=0, p_out=16, p_lse=16, p_ws=16, wsb=256, flags=0, p_stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(flags=2), BAD), (dict(flags=_lib.ATTN_NON_CAUSAL | 4), BAD), (dict(S=-1), BAD),
    (dict(T=-1), BAD), (dict(p_ws=None), BAD), (dict(wsb=255), BAD), (dict(window=-1), BAD),
    (dict(window=5, flags=_lib.ATTN_NON_CAUSAL), BAD), (dict(p_q=None), BAD), (dict(p_cu=None), BAD),
    (dict(p_lens=None), BAD), (dict(p_table=None), BAD), (dict(p_out=None), BAD),
    (dict(p_kc=None), BAD), (dict(p_vs=None), BAD), (dict(hk=0), BAD), (dict(hq=0), BAD),
    (dict(hq=7), BAD), (dict(hq=34), NOT), (dict(columns=0), BAD), (dict(columns=9), BAD),
    (dict(mq=0), BAD), (dict(ms=0), BAD), (dict(ms=0x7fffffff), BAD), (dict(ns=-1), BAD),
    (dict(ns=65), BAD), (dict(ns=2), BAD), (dict(ns=64, wsb=1 << 12), BAD), (dict(p_q=8), BAD),
    (dict(p_out=24), BAD), (dict(p_ws=8), BAD), (dict(p_lse=18), BAD), (dict(p_sinks=2), BAD),
    (dict(p_lens=6), BAD), (dict(d=80), NOT), (dict(bs=64), NOT), (dict(nb=1 << 23), NOT),
    (dict(T=1 << 28), NOT),
])
def test_attention_refuses(lib, kw, expect):
    assert lib.pa_paged_attention_q4(*_values(ATTN, kw, ("scale",))) == expect
    assert lib.pa_last_error().decode()


@pytest.mark.parametrize("kw", [dict(S=0), dict(T=0, p_q=None)])
def test_attention_of_nothing_is_a_no_op(lib, kw):
    assert lib.pa_paged_attention_q4(*_values(ATTN, kw, ("scale",))) == _lib.Status.OK


PROMPT = dict(p_q=16, qstride=1024, p_k=16, kstride=256, p_v=16, vstride=256, p_cu_q=16, p_cu_k=16,
              S=2, T=40, n=40, hq=8, hk=2, d=128, mq=30, mk=30, scale=0.1, p_sinks=None, window=0,
              p_out=16, p_lse=16, p_ws=16, wsb=256, flags=0, p_stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(flags=2), BAD), (dict(S=-1), BAD), (dict(T=-1), BAD), (dict(n=-1), BAD),
    (dict(p_ws=None), BAD), (dict(wsb=255), BAD), (dict(window=-1), BAD),
    (dict(window=5, flags=_lib.ATTN_NON_CAUSAL), BAD), (dict(p_q=None), BAD), (dict(p_k=None), BAD),
    (dict(p_v=None), BAD), (dict(p_cu_q=None), BAD), (dict(p_cu_k=None), BAD), (dict(p_out=None), BAD),
    (dict(hk=0), BAD), (dict(hq=0), BAD), (dict(hq=7), BAD), (dict(hq=258, qstride=1 << 16), NOT),
    (dict(d=96), NOT), (dict(mq=0), BAD), (dict(mk=-1), BAD), (dict(qstride=1016), BAD),
    (dict(kstride=248), BAD), (dict(vstride=128), BAD), (dict(qstride=1028), BAD),
    (dict(kstride=260), BAD), (dict(p_q=8), BAD), (dict(p_v=24), BAD), (dict(p_out=8), BAD),
    (dict(p_ws=8), BAD), (dict(p_lse=2), BAD), (dict(p_sinks=17), BAD), (dict(p_cu_k=18), BAD),
    (dict(qstride=1 << 36), NOT), (dict(T=1 << 28), NOT), (dict(n=0x7fffffff), NOT),
])
def test_prompt_refuses(lib, kw, expect):
    assert lib.pa_prompt_attention(*_values(PROMPT, kw, ("scale",))) == expect
    assert lib.pa_last_error().decode()


@pytest.mark.parametrize("kw", [dict(S=0), dict(T=0, p_q=None)])
def test_prompt_of_nothing_is_a_no_op(lib, kw):
    assert lib.pa_prompt_attention(*_values(PROMPT, kw, ("scale",))) == _lib.Status.OK


def test_workspace_sizes():
    one = _lib.paged_attention_q4_workspace_size
    assert one(4, 4, 8, 2, 128, 1, 100, 1) == 256
    assert one(4, 4, 8, 2, 128, 1, 100, 3) == 256 + 4 * 8 * 3 * 130 * 4
    auto = one(1, 1, 8, 2, 128, 1, 1 << 17)
    assert (auto - 256) % (8 * 130 * 4) == 0 and 1 < (auto - 256) // (8 * 130 * 4) <= 64
    for bad in ((0, 4, 8, 2, 128, 1, 100, 1), (4, 4, 7, 2, 128, 1, 100, 3), (4, 4, 8, 2, 96, 1, 100, 3),
                (4, 4, 8, 2, 128, 0, 100, 3), (4, 4, 8, 2, 128, 1, 100, 65)):
        assert one(*bad) == 256
    prompt = _lib.prompt_attention_workspace_size
    assert prompt(64, 1 << 16, 1 << 16, 8, 2, 128, 1024, 1024) == 256
    few = prompt(1, 40, 5000, 8, 2, 128, 40, 5000)
    assert (few - 256) % (40 * 8 * 130 * 4) == 0 and 1 < (few - 256) // (40 * 8 * 130 * 4) <= 64
    assert prompt(1, 40, 5000, 7, 2, 128, 40, 5000) == 256


def test_bindings_refuse_host_tensors():
    rows = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    codes = torch.zeros((2, 2, 16, 32), dtype=torch.uint8)
    ks = torch.zeros((2, 2, 2, 16, 2), dtype=torch.float16)
    vs = torch.zeros((2, 2, 2, 2, 16), dtype=torch.float16)
    cache = (codes, ks, codes.clone(), vs)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        _lib.kv_store_q4(rows, rows, torch.arange(4), *cache)
    for load in (_lib.kv_load, _lib.kv_load_f8v4, _lib.kv_load_q4):
        with pytest.raises(ValueError):
            load(rows, rows, cu, table, *cache)
    with pytest.raises(ValueError):
        _lib.paged_attention_q4(rows, *cache, cu, cu[1:], table, 4, 4)
    with pytest.raises(ValueError):
        _lib.prompt_attention(rows, rows, rows, cu, 4)


def test_bindings_are_public():
    import paged_attention_int8_gb300 as pkg
    for name in ("kv_store_q4", "kv_load", "kv_load_f8v4", "kv_load_q4", "paged_attention_q4",
                 "paged_attention_q4_workspace_size", "prompt_attention",
                 "prompt_attention_workspace_size"):
        assert name in pkg.__all__ and callable(getattr(pkg, name))
