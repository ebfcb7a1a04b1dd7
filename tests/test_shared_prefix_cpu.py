"""The shared-prefix serving calls without a GPU: argument checks of the C
entries and of the bindings, and the workspace rule."""
import ctypes

import pytest
import torch

from paged_attention_int8_gb300 import _lib, build as pkg_build

OK, BAD, UNS = _lib.Status.OK, _lib.Status.INVALID_ARG, _lib.Status.UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return _lib.load()


def _call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*a.values())


TABLES = dict(ctx=0x1000, q=0x2000, S=4, src=0x10000, sstride=8, rows=4, source_rows=None,
              shared=None, free=0x3000, num_free=9, head=0x4000, nb=10, bs=16, table=0x20000,
              stride=8, cu=0x5000, lens=0x6000, slots=0x7000, pos=0x8000, T=4, pairs=0x9000,
              next=0xA000, status=0xB000, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(ctx=None), BAD), (dict(q=None), BAD), (dict(src=None), BAD), (dict(table=None), BAD),
    (dict(cu=None), BAD), (dict(lens=None), BAD), (dict(slots=None), BAD), (dict(free=None), BAD),
    (dict(S=-1), BAD), (dict(T=-1), BAD), (dict(num_free=-1), BAD), (dict(rows=0), BAD),
    (dict(rows=3), BAD),                                   # fewer rows than sequences
    (dict(nb=0), BAD), (dict(sstride=0), BAD), (dict(stride=-2), BAD),
    (dict(bs=8), UNS), (dict(T=1 << 26), UNS), (dict(stride=1 << 26), UNS),
    (dict(ctx=0x1002), BAD), (dict(slots=0x7004), BAD), (dict(pos=0x8004), BAD),
    (dict(status=0xB001), BAD),
    (dict(shared=0xC000, pairs=None), BAD),                # a private page needs its copy
    (dict(next=0x4000), BAD),                              # next_free is free_head
    (dict(lens=0x1000), BAD),                              # seq_lens over context_lens
    (dict(cu=0x6004), BAD),                                # two outputs overlap
    (dict(table=0x10000, source_rows=0xD000), BAD),        # in place, rows moved
    (dict(table=0x10000, stride=16), BAD),                 # in place, another stride
    (dict(table=0x10040), BAD),                            # part of the source table
    (dict(S=0, cu=None), BAD),
])
def test_build_block_tables_refuses(lib, kw, expect):
    assert _call(lib.pa_build_block_tables, TABLES, kw) == expect
    assert lib.pa_last_error().decode()


COPY = dict(pairs=0x1000, n=4, hk=2, d=128, a=0x10000, b=0x20000, c=0x30000, e=0x40000, nb=4,
            bs=16, status=None, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(pairs=None), BAD), (dict(n=-1), BAD), (dict(a=None), BAD), (dict(b=None), BAD),
    (dict(c=None), BAD), (dict(e=None), BAD), (dict(hk=0), BAD), (dict(nb=0), BAD),
    (dict(d=96), UNS), (dict(bs=64), UNS), (dict(a=0x10008), BAD), (dict(pairs=0x1004), BAD),
    (dict(nb=1 << 30), UNS), (dict(n=(1 << 31) - 1, hk=8), UNS), (dict(status=0x1002), BAD),
])
def test_copy_blocks_refuses(lib, kw, expect):
    for fn in (lib.pa_copy_blocks, lib.pa_copy_blocks_f8v4):
        assert _call(fn, COPY, kw) == expect
        assert lib.pa_last_error().decode()


def test_copy_blocks_no_pairs_is_a_no_op(lib):
    for fn in (lib.pa_copy_blocks, lib.pa_copy_blocks_f8v4):
        assert _call(fn, COPY, dict(n=0, pairs=None)) == OK


ATTN = dict(q=16, kc=16, ks=16, vc=16, vs=16, cu=16, sl=16, bt=16, bts=8, groups=16, prefix=16,
            G=1, S=2, T=2, hq=8, hk=2, d=128, nb=16, bs=16, mq=1, mp=100, ms=10,
            scale=ctypes.c_float(0.1), sinks=None, out=16, lse=16, ws=16, wsb=1 << 20, flags=0,
            stream=None)


@pytest.mark.parametrize("kw,expect", [
    *[(dict([(n, None)]), BAD) for n in ("q", "kc", "ks", "vc", "vs", "cu", "sl", "bt", "groups",
                                         "prefix", "out", "ws")],
    (dict(G=0), BAD), (dict(G=-1), BAD), (dict(S=-1), BAD), (dict(T=-1), BAD), (dict(hq=7), BAD),
    (dict(hk=0), BAD), (dict(hq=34), UNS), (dict(d=80), UNS), (dict(bs=64), UNS),
    (dict(nb=0), BAD), (dict(bts=0), BAD), (dict(nb=1 << 30), UNS), (dict(mq=0), BAD),
    (dict(mp=-1), BAD), (dict(ms=0), BAD), (dict(out=8), BAD), (dict(lse=18), BAD),
    (dict(sinks=18), BAD), (dict(cu=18), BAD), (dict(groups=18), BAD), (dict(prefix=18), BAD),
    (dict(flags=1), BAD), (dict(wsb=255), BAD),
    (dict(wsb=256 + 2 * 8 * 2 * 130 * 4 - 1), BAD),       # below two triples per row
])
def test_shared_prefix_refuses(lib, kw, expect):
    for fn in (lib.pa_paged_attention_shared_prefix, lib.pa_paged_attention_shared_prefix_f8v4):
        assert _call(fn, ATTN, kw) == expect
        assert lib.pa_last_error().decode()


def test_shared_prefix_empty_batch_is_a_no_op(lib):
    for fn in (lib.pa_paged_attention_shared_prefix, lib.pa_paged_attention_shared_prefix_f8v4):
        assert _call(fn, ATTN, dict(S=0, T=0, q=None)) == OK


def test_workspace_size(lib):
    size = _lib.shared_prefix_workspace_size
    # a header and whole triples per row, at least two
    for args in ((1, 1, 1, 4, 2, 64, 1, 0, 1), (64, 64, 1, 32, 8, 128, 1, 8192, 1024),
                 (8, 40, 3, 64, 8, 256, 5, 100000, 100000), (2, 4096, 1, 32, 8, 128, 2048, 64, 9000)):
        s, t, g, hq, hk, d, *_ = args
        triple = t * hq * (d + 2) * 4
        assert (size(*args) - 256) % triple == 0 and size(*args) >= 256 + 2 * triple
    # sizes out of range
    assert size(0, 0, 0, 4, 2, 64, 1, 0, 1) == 256
    assert size(1, 1, 1, 5, 2, 64, 1, 0, 1) == 256
    assert size(1, 1, 1, 4, 2, 80, 1, 0, 1) == 256


def test_bindings_stand_in_the_package():
    import paged_attention_int8_gb300 as pkg
    for name in ("build_block_tables", "BlockTables", "copy_blocks", "copy_blocks_f8v4",
                 "paged_attention_shared_prefix", "paged_attention_shared_prefix_f8v4",
                 "shared_prefix_workspace_size"):
        assert name in pkg.__all__ and callable(getattr(pkg, name))


def test_bindings_refuse_host_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        _lib.build_block_tables(i32(2), i32(2), i32(2, 4), i32(3), 4, 16, 2)
    kc = torch.zeros((2, 2, 16, 64), dtype=torch.int8)
    vc = torch.zeros((2, 2, 64, 16), dtype=torch.int8)
    ks, vs = torch.zeros((2, 2, 16, 2)).half(), torch.zeros((2, 2, 2, 16)).half()
    with pytest.raises(ValueError):
        _lib.copy_blocks(i32(1, 2), kc, ks, vc, vs)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _lib.paged_attention_shared_prefix(q, kc, ks, vc, vs, i32(3), i32(2), i32(2, 1), i32(2),
                                           i32(1), 1, 1, 1)
    with pytest.raises((TypeError, ValueError)):
        _lib.paged_attention_shared_prefix(q, kc.float(), ks, vc, vs, i32(3), i32(2), i32(2, 1),
                                           i32(2), i32(1), 1, 1, 1)
