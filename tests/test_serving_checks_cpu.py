"""Argument checks of the attention and serving calls on the edges of their sizes and
layouts, without a GPU."""
import pytest
import torch

from paged_attention_int8_gb300 import _lib


def test_table_layouts():
    """Row strides that the attention calls take: those of a single row mean nothing."""
    t = torch.zeros((3, 8), dtype=torch.int32)
    layout = _lib._table_layout
    assert layout(t) == (3, 8, 8) and layout(t[:, 2:5]) == (3, 3, 8)
    assert layout(torch.zeros((8, 1)).t()) == (1, 8, 8)      # strides (1, 1)
    assert layout(t[1:2, :4]) == (1, 4, 4)
    assert layout(torch.zeros((1, 8)).t()) == (8, 1, 1)      # strides (1, 8)
    for bad in (t.t(), t[:1].expand(3, -1), t[:, ::2], t.as_strided((2, 8), (4, 1)), t[0]):
        with pytest.raises(ValueError):
            layout(bad)
