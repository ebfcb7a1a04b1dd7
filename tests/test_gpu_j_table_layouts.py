"""Block tables in the layouts that a caller's tensors take: one row of any strides,
one column, a slice of a wider table."""
from __future__ import annotations

from dataclasses import replace

import pytest
import torch

from paged_attention_int8_gb300 import _lib
from tests import _shared as S

pytestmark = pytest.mark.gpu


def _calls(b):
    """Every attention binding of the batch's format over its table."""
    longest = max(b.seq_lens)
    if b.fmt == "q8":
        yield lambda: _lib.paged_attention(b.q, *b.cache, b.cu, b.lens, b.table, max(b.q_lens),
                                           longest)
        yield lambda: _lib.paged_attention_noalloc(b.q, *b.cache, b.cu, b.lens, b.table,
                                                   max(b.q_lens), longest)
    else:
        yield lambda: _lib.paged_attention_f8v4(b.q, *b.cache, b.cu, b.lens, b.table,
                                                max(b.q_lens), longest)
    yield b.call


@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
def test_one_row_of_any_strides(cuda_device, fmt):
    """A table of one row made by a transpose: torch gives its rows a stride of one
    and calls it contiguous."""
    b = S.make(81, cuda_device, fmt, 8, 2, 128, 16, [(70, [(1, 45)])])
    ref = S.reference(b)
    column = b.table.reshape(-1, 1).contiguous()
    b.table = column.t()
    assert b.table.stride() == (1, 1) and b.table.shape[1] > 1 and b.table.is_contiguous()
    for call in _calls(b):
        S.check(b, *call(), ref=ref)


@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
def test_one_column_of_any_strides(cuda_device, fmt):
    """Short sequences, a page each, their column taken from a transposed row."""
    b = S.make(82, cuda_device, fmt, 8, 2, 128, 16, [(0, [(1, 9), (1, 16), (1, 3)])], columns=0)
    ref = S.reference(b)
    assert b.table.shape[1] == 1
    b.table = b.table.reshape(1, -1).contiguous().t()
    assert b.table.stride() == (1, 3)
    for call in _calls(b):
        S.check(b, *call(), ref=ref)


def test_tables_that_are_refused(cuda_device):
    b = S.make(83, cuda_device, "q8", 8, 2, 128, 16, [(20, [(1, 5), (1, 30)])])
    good = b.table
    for table in (good.t().contiguous().t(),             # the columns apart
                  good[:1].expand(2, -1),                # one row for both
                  good.as_strided((2, good.shape[1]), (1, 1)),
                  good.reshape(-1)):
        b.table = table
        for call in _calls(b):
            with pytest.raises(ValueError):
                call()


@pytest.mark.parametrize("fmt,d,hq,hk,n,q_len", [("q8", 128, 8, 2, 3, 1), ("q8", 256, 16, 2, 12, 1),
                                                 ("f8v4", 64, 4, 2, 3, 3), ("q8", 128, 16, 1, 20, 2),
                                                 ("q8", 128, 8, 2, 3, 20)])
def test_slice_of_a_wider_table(cuda_device, fmt, d, hq, hk, n, q_len):
    """The columns of a slice end where the slice does: keys past them are flagged and
    left out, though the wider table has entries there; the other rows are right."""
    b = S.make(84, cuda_device, fmt, hq, hk, d, 16, [(40, [(q_len, 30)] * n)], columns=0)
    ref = S.reference(b)
    columns = b.table.shape[1]
    wide = torch.zeros((n, columns + 9), dtype=torch.int32, device=cuda_device)
    wide[:, 4:4 + columns] = b.table
    b.table = wide[:, 4:4 + columns]
    S.check(b, *b.call(), ref=ref)
    lens = b.lens.clone()
    lens[1] = (columns + 3) * 16
    fn = (_lib.paged_attention_shared_prefix if fmt == "q8"
          else _lib.paged_attention_shared_prefix_f8v4)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device)
    out = torch.full_like(b.q, float("nan"))
    lse = torch.full(b.q.shape[:2], float("nan"), device=cuda_device)
    fn(b.q, *b.cache, b.cu, lens, b.table, b.groups, b.prefixes, *b.bounds, out=out, lse=lse,
       workspace=ws)
    with pytest.raises(_lib.PagedAttentionError) as err:
        _lib.check_status(ws)
    assert err.value.bits == _lib.DEV_BAD_BLOCK
    for t in (out, lse):  # the over-long sequence: any row, for the comparison of the others
        t[q_len:2 * q_len] = ref[0 if t is out else 1][q_len:2 * q_len].to(t)
    S.check(b, out, lse, ref=ref)


@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
def test_last_columns_of_a_wider_table(cuda_device, fmt):
    """A slice whose last row ends with the memory, on the current stream and on
    another."""
    b = S.make(85, cuda_device, fmt, 8, 2, 128, 16, [(40, [(1, 30), (1, 9), (1, 33)])], columns=0)
    # the pages of one group differ where the prefix ends inside one: each row by itself
    ref = S.reference(b)
    own = S.reference(replace(b, prefix=[0]))
    wide = torch.zeros((3, b.table.shape[1] + 9), dtype=torch.int32, device=cuda_device)
    wide[:, 9:] = b.table
    b.table = wide[:, 9:]
    *paged, shared = _calls(b)
    S.check(b, *shared(), ref=ref)
    for call in paged:
        S.check(b, *call(), ref=own)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = _lib.paged_attention if fmt == "q8" else _lib.paged_attention_f8v4
    out, lse = call(b.q, *b.cache, b.cu, b.lens, b.table, 1, max(b.seq_lens), stream=side)
    side.synchronize()
    S.check(b, out, lse, ref=own)
