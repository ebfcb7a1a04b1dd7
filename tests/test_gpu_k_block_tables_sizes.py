"""build_block_tables at the ends of its sizes: as many tokens as it takes, many
sequences beside long ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_attention_int8_gb300 import _lib
from tests import _harness as H

pytestmark = pytest.mark.gpu

MOST_TOKENS = 1 << 25


def test_as_many_padding_rows_as_it_takes(cuda_device):
    H.ensure_built()
    e = lambda *s: torch.empty(s, dtype=torch.int32, device=cuda_device)  # noqa: E731
    got = _lib.build_block_tables(e(0), e(0), e(1, 4), e(0), 3, 16, MOST_TOKENS)
    assert bool((got.slot_mapping == -1).all()) and bool((got.positions == 0).all())


def _plain(ctx, q, source, rows, free, bs, tokens):
    """The definition, in numpy: table (-1 where nothing is written), cu, slots, positions."""
    n, columns = len(ctx), source.shape[1]
    held, end = -(-ctx // bs), -(-(ctx + q) // bs)
    cu = np.concatenate([[0], np.cumsum(q)])
    at = np.concatenate([[0], np.cumsum(end - held)])
    table = np.full((n, columns), -1, np.int64)
    slots, pos = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int64)
    for s in range(n):
        table[s, :held[s]] = source[rows[s], :held[s]]
        table[s, held[s]:end[s]] = free[at[s]:at[s + 1]]
        x = np.arange(ctx[s], ctx[s] + q[s])
        slots[cu[s]:cu[s + 1]] = table[s, x // bs] * bs + x % bs
        pos[cu[s]:cu[s + 1]] = x
    return table, cu, slots, pos, at[n]


@pytest.mark.parametrize("n,columns,long_q,pad", [
    (1, (1 << 25) // 16, (1 << 25) - 700, 300),  # one prompt as long as it may be
    (3000, 9000, 90000, 40000),                  # more chunks than a row of blocks has
    (70000, 40, 500, 11),                        # many sequences
])
def test_many_tokens_and_sequences(cuda_device, n, columns, long_q, pad):
    H.ensure_built()
    rng = np.random.default_rng(n)
    bs = 16
    ctx = rng.integers(0, 30, n) if n > 1 else np.array([399])
    q = rng.integers(0, 3, n)
    q[n // 2] = long_q
    if n > 1:
        q[n - 1] = 7
        ctx[1] = bs * columns - 40  # a row of many held pages
    held = -(-ctx // bs)
    source = np.full((n, columns), -1, np.int64)
    source[np.arange(columns) < held[:, None]] = np.arange(held.sum())
    new = int((-(-(ctx + q) // bs) - held).sum())
    blocks = int(held.sum()) + new
    assert blocks * bs < 2 ** 31
    free = held.sum() + rng.permutation(new)
    rows = rng.permutation(n)
    tokens = int(q.sum()) + pad
    assert tokens <= MOST_TOKENS
    source[rows] = source.copy()  # the pages of s at row rows[s]
    want = _plain(ctx, q, source, rows, free, bs, tokens)
    i32 = lambda v: torch.from_numpy(np.ascontiguousarray(v).astype(np.int32)).to(cuda_device)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = _lib.build_block_tables(i32(ctx), i32(q), i32(source), i32(free), blocks, bs, tokens,
                                  source_rows=i32(rows), status=status)
    assert _lib.check_status(status) == 0
    for t, w in zip((got.block_table, got.cu_seqlens_q, got.slot_mapping, got.positions), want):
        assert torch.equal(t.cpu().to(torch.int64), torch.from_numpy(w))
    assert got.next_free.tolist() == [want[4]]


def test_as_many_sequences_as_it_takes(cuda_device):
    """2^18 sequences: right, and in milliseconds."""
    H.ensure_built()
    n, bs = 1 << 18, 16
    i = torch.arange(n, device=cuda_device)
    ctx, q = (i % 33).int(), (i % 3).int()
    source = (3 * i[:, None] + torch.arange(3, device=cuda_device)).int()
    held, end = (ctx + bs - 1) // bs, (ctx + q + bs - 1) // bs
    new = torch.where(q > 0, end - held, 0)
    free = 3 * n + torch.arange(int(new.sum()), device=cuda_device, dtype=torch.int32)
    tokens = int(q.sum())
    args = (ctx, q, source, free, 4 * n, bs, tokens)
    got = _lib.build_block_tables(*args)
    cu = torch.cumsum(q, 0, dtype=torch.int32)
    assert torch.equal(got.cu_seqlens_q[1:], cu) and torch.equal(got.seq_lens, ctx + q)
    assert got.next_free.tolist() == [free.numel()]
    at = (torch.cumsum(new, 0) - new)[:, None] + torch.arange(3, device=cuda_device) - held[:, None]
    page = torch.arange(3, device=cuda_device)[None]
    fresh = free[at.clamp(0, free.numel() - 1)]
    table = torch.where(page < held[:, None], source, fresh)
    table = torch.where(page < end[:, None], table, torch.full_like(table, -1))
    assert torch.equal(got.block_table, table)
    seq = torch.repeat_interleave(i, q.long())
    x = ctx[seq].long() + torch.arange(tokens, device=cuda_device) - (cu - q)[seq].long()
    assert torch.equal(got.positions, x)
    assert torch.equal(got.slot_mapping, table[seq, x // bs].long() * bs + x % bs)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    _lib.build_block_tables(*args, out=got)
    stop.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(stop) < 100  # ms


def test_results_that_are_not_wanted(cuda_device):
    """positions, copy_pairs and next_free may be None; the others are refused so."""
    H.ensure_built()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    args = (i32(3, 20), i32(1, 2), i32(7, -1, 8, 9).view(2, 2), i32(4, 5), 10, 16, 3)
    want = _lib.build_block_tables(*args)
    for at in range(7):
        out = [torch.full_like(t, -1) for t in want]
        out[at] = None
        if at in (0, 1, 2, 3):
            with pytest.raises(ValueError):
                _lib.build_block_tables(*args, out=out)
        else:
            got = _lib.build_block_tables(*args, out=out)
            assert got[at] is None
            for t, w in zip(got, want):
                assert t is None or torch.equal(t, w)
    # two at once
    for at in ((3, 4), (4, 5, 6)):
        out = [None if i in at else torch.full_like(t, -1) for i, t in enumerate(want)]
        if at[0] == 3:
            with pytest.raises(ValueError):
                _lib.build_block_tables(*args, out=out)
        else:
            assert torch.equal(_lib.build_block_tables(*args, out=out)[3], want[3])
