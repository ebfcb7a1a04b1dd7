"""Argument checks of the attention and serving calls on the edges of their sizes and
layouts, without a GPU."""
import ctypes

import pytest
import torch

from paged_attention_int8_gb300 import _lib, build as pkg_build


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return _lib.load()


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


VIEW = dict(q=16, kc=16, ks=16, vc=16, vs=16, cu=16, sl=16, bt=16, bts=8, cols=5, groups=16,
            prefix=16, G=1, S=2, T=2, hq=8, hk=2, d=128, nb=16, bs=16, mq=1, mp=100, ms=10,
            scale=ctypes.c_float(0.1), sinks=None, out=16, lse=16, ws=16, wsb=1 << 20, flags=0,
            stream=None)


@pytest.mark.parametrize("kw", [dict(cols=0), dict(cols=-3), dict(cols=9), dict(bts=4), dict(bts=0)])
def test_views_whose_columns_do_not_fit_their_rows(lib, kw):
    for fn in (lib.pa_paged_attention_shared_prefix_view,
               lib.pa_paged_attention_shared_prefix_f8v4_view):
        assert fn(*{**VIEW, **kw}.values()) == _lib.Status.INVALID_ARG
        assert "columns" in lib.pa_last_error().decode()


def test_rows_that_would_pass_the_end_of_their_memory():
    """The entries that a call may look up in a view of a wider table all stand in its
    memory: the view's own, or a copy's."""
    wide = torch.arange(24, dtype=torch.int32).reshape(3, 8)
    for view, copied in ((wide[:, :5], False), (wide[:2, 3:], False), (wide[:, 3:], True),
                         (wide[1:, 7:], True), (wide[1:2], False)):
        rows, columns, stride = _lib._table_layout(view)
        got, got_stride = _lib._table_in_bounds(view, rows, stride, None)
        assert torch.equal(got, view) and (got.data_ptr() != view.data_ptr()) == copied
        assert got_stride == (columns if copied else stride)
        assert got.storage_offset() + rows * got_stride <= got.untyped_storage().nbytes() // 4


def test_block_tables_of_too_many_sequences(lib):
    """The sums over earlier sequences are formed by every block: refused where they
    would keep the GPU for seconds and more."""
    far = 1 << 40
    args = dict(ctx=far, q=2 * far, S=(1 << 18) + 1, src=3 * far, sstride=8, rows=1 << 19,
                source_rows=None, shared=None, free=4 * far, num_free=9, head=5 * far, nb=10,
                bs=16, table=6 * far, stride=8, cu=7 * far, lens=8 * far, slots=9 * far,
                pos=10 * far, T=4, pairs=11 * far, next=12 * far, status=13 * far, stream=None)
    for n in ((1 << 18) + 1, 1 << 25, (1 << 31) - 1):
        args.update(S=n, rows=n)
        assert lib.pa_build_block_tables(*args.values()) == _lib.Status.UNSUPPORTED
        assert "sequences" in lib.pa_last_error().decode()


def test_sizes_that_no_product_holds(lib):
    """Sizes each in range whose products pass 64 bits: an answer, not a division by
    zero, and no size that wrapped around."""
    most = (1 << 31) - 1
    size = _lib.shared_prefix_workspace_size
    for args in ((1 << 30, most, 1, 1 << 19, 1 << 15, 64, most, 5, 5),
                 (1 << 30, most, 1, 1 << 30, 1 << 30, 64, 1 << 10, 5, 5),
                 (most, most, most, 16, 1, 256, most, most - 4096, most - 4096)):
        _, t, _, hq, _, d, *_ = args
        two = 256 + 2 * t * hq * (d + 2) * 4  # two triples a row, or all that a size_t holds
        assert size(*args) >= min(two, (1 << 64) - 1)
    for big in (dict(T=most), dict(S=most), dict(G=most), dict(S=1 << 30, T=1 << 30)):
        args = {**VIEW, **big, "mq": most, "hq": 1 << 19, "hk": 1 << 15}
        for fn in (lib.pa_paged_attention_shared_prefix_view,
                   lib.pa_paged_attention_shared_prefix_f8v4_view):
            assert fn(*args.values()) in (_lib.Status.UNSUPPORTED, _lib.Status.INVALID_ARG)


@pytest.mark.parametrize("n", [3, 16, 40])
def test_segments_follow_the_rows_of_a_pass(lib, n):
    """Heads of 256 channels take 8 rows a pass: a sequence of 16 rows fills as many
    blocks as two of 8, and has its keys cut into as many segments."""
    size = _lib.shared_prefix_workspace_size
    tokens = 4 * n
    assert size(n, tokens, 1, 8, 2, 256, 4, 0, 4096) == size(2 * n, tokens, 1, 8, 2, 256, 2, 0, 4096)


def test_streams_of_other_libraries_belong_to_the_tensors_device(monkeypatch):
    """An object with a stream's handle: its memory comes from the device that the
    tensors are on, whichever is current."""
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: made.append((h, device)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    _lib._allocating(type("Stream", (), {"cuda_stream": 0x1230})(), 3)
    assert made == [(0x1230, 3)]
    with _lib._allocating(None, 3):
        pass
    assert len(made) == 1
