"""Groups whose bounds leave the batch or its order: every row that is not written is
flagged, every other row is right."""
from __future__ import annotations

import pytest
import torch

from paged_attention_int8_gb300 import _lib
from tests import _shared as S

pytestmark = pytest.mark.gpu


def _valid(groups, n):
    """Sequences whose group's bounds lie in the batch, by the last group that starts at
    or before each."""
    good = set()
    for s in range(n):
        g = max((i for i, x in enumerate(groups[:-1]) if x <= s), default=None)
        if g is not None and 0 <= groups[g] <= s < groups[g + 1] <= n:
            good.add(s)
    return good


@pytest.mark.parametrize("fmt,d,hq,hk,q_len", [("q8", 128, 8, 2, 1), ("q8", 256, 16, 2, 1),
                                               ("f8v4", 64, 4, 2, 3), ("q8", 128, 8, 2, 20)])
@pytest.mark.parametrize("groups", [[0, 20, 41], [0, 20, 2 ** 31 - 1], [-1, 20, 40], [-9, 20, 40],
                                    [0, 20, 30], [3, 20, 40], [0, 41, 41], [40, 40, 40],
                                    [0, 20, 40]], ids=str)
def test_group_bounds_outside_the_batch(cuda_device, fmt, d, hq, hk, q_len, groups):
    n = 40
    b = S.make(91, cuda_device, fmt, hq, hk, d, 16,
               [(64, [(q_len, 25)] * 20), (32, [(q_len, 21)] * 20)])
    _check_groups(b, S.reference(b), groups, _valid(groups, n), q_len)


@pytest.mark.parametrize("last", [40, 41, 2 ** 31 - 1])
def test_more_groups_than_a_warp(cuda_device, last):
    """Forty groups of one sequence, found by search; the last one's end past the batch."""
    b = S.make(92, cuda_device, "q8", 8, 2, 128, 16, [(40, [(1, 20)])] * 40)
    groups = list(range(40)) + [last]
    _check_groups(b, S.reference(b), groups, _valid(groups, 40), 1)


def _check_groups(b, ref, groups, valid, q_len):
    n = len(b.seq_lens)
    fn = (_lib.paged_attention_shared_prefix if b.fmt == "q8"
          else _lib.paged_attention_shared_prefix_f8v4)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=b.q.device)  # noqa: E731
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=b.q.device)
    out = torch.full_like(b.q, float("nan"))
    lse = torch.full(b.q.shape[:2], float("nan"), device=b.q.device)
    fn(b.q, *b.cache, b.cu, b.lens, b.table, i32(groups), b.prefixes, *b.bounds, out=out, lse=lse,
       workspace=ws)
    if len(valid) == n:
        assert _lib.check_status(ws) == 0
    else:
        with pytest.raises(_lib.PagedAttentionError) as err:
            _lib.check_status(ws)
        assert err.value.bits == _lib.DEV_BAD_SEQ
    for s in range(n):
        rows = slice(s * q_len, (s + 1) * q_len)
        if s not in valid:  # left as they were
            assert torch.isnan(out[rows].float()).all() and torch.isnan(lse[rows]).all()
            out[rows], lse[rows] = ref[0][rows].to(out), ref[1][rows].to(lse)
    S.check(b, out, lse, ref=ref)
