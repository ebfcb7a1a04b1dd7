"""paged_attention_shared_prefix against a plain fp64 implementation, at the
sizes, lengths and masks where it can go wrong."""
import math

import pytest
import torch

from paged_attention_int8_gb300 import _lib
from tests import _shared as S

pytestmark = pytest.mark.gpu

LAYOUTS = [(4, 2, 64, 16), (8, 2, 128, 16), (8, 1, 128, 32), (4, 2, 256, 16), (2, 1, 256, 32),
           (3, 3, 64, 32), (7, 1, 128, 16), (32, 2, 128, 32), (6, 2, 256, 16), (16, 1, 64, 16)]
DECODE = [(70, [(1, 1), (1, 37), (1, 130)])]


@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
@pytest.mark.parametrize("hq,hk,d,bs", LAYOUTS)
def test_layouts(cuda_device, fmt, hq, hk, d, bs):
    b = S.make(hq * d + bs, cuda_device, fmt, hq, hk, d, bs, DECODE)
    S.check(b, *b.call())


# prefixes that end with a page, a tile, one key either side; one key; none
@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 63, 64, 65, 128, 300])
def test_prefix_lengths(cuda_device, fmt, prefix):
    b = S.make(prefix + 1, cuda_device, fmt, 4, 2, 128, 16,
               [(prefix, [(1, 1), (1, 2), (1, 16), (1, 63), (1, 64), (1, 65)])])
    S.check(b, *b.call())


# query chunks beside single tokens; empty queries; groups of one, empty groups
@pytest.mark.parametrize("fmt,d,bs", [("q8", 64, 16), ("q8", 128, 32), ("q8", 256, 16),
                                      ("f8v4", 128, 16), ("f8v4", 256, 32)])
def test_query_lengths_and_groups(cuda_device, fmt, d, bs):
    groups = [(33, [(1, 1), (5, 5), (0, 7), (17, 40)]), (0, [(3, 3)]), (64, []),
              (7, [(1, 90)]), (129, [(2, 3)] * 9)]
    b = S.make(d + bs, cuda_device, fmt, 8, 2, d, bs, groups, pad_rows=5)
    S.check(b, *b.call())


# groups whose rows fill one, several and parts of row blocks
@pytest.mark.parametrize("hq,hk,d,n", [(8, 2, 128, 3), (8, 2, 128, 16), (8, 2, 128, 33),
                                       (8, 1, 128, 33), (8, 1, 64, 70), (4, 2, 256, 40),
                                       (7, 1, 128, 39), (16, 1, 128, 17), (1, 1, 64, 300)])
@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
def test_group_sizes(cuda_device, fmt, hq, hk, d, n):
    b = S.make(n, cuda_device, fmt, hq, hk, d, 16, [(100, [(1, 1 + i % 5) for i in range(n)]),
                                                    (40, [(1, 3)] * 2)])
    S.check(b, *b.call())


# long prefixes and suffixes: many segments; the workspace down to one segment each
@pytest.mark.parametrize("fmt,d,bs", [("q8", 128, 16), ("q8", 256, 16), ("q8", 64, 32),
                                      ("f8v4", 128, 32)])
@pytest.mark.parametrize("squeeze", [False, True])
def test_segments(cuda_device, fmt, d, bs, squeeze):
    b = S.make(d, cuda_device, fmt, 4, 1, d, bs, [(2501, [(1, 1), (1, 1300), (4, 700)])])
    ws = None
    if squeeze:
        ws = torch.zeros(256 + b.q.shape[0] * b.hq * 2 * (d + 2) * 4, dtype=torch.uint8,
                         device=cuda_device)
    S.check(b, *b.call(workspace=ws))


# many groups: shares of several short prefixes each, last rows that fill less
# than half a block, more groups than a warp has lanes, prefixes of no key
@pytest.mark.parametrize("fmt,hq,hk,d,bs", [("q8", 16, 1, 64, 16), ("q8", 16, 4, 128, 32),
                                            ("f8v4", 16, 2, 128, 16), ("q8", 14, 2, 64, 32),
                                            ("q8", 16, 2, 256, 16), ("f8v4", 8, 1, 256, 32)])
@pytest.mark.parametrize("n_groups", [2, 31, 33, 70])
def test_many_groups(cuda_device, fmt, hq, hk, d, bs, n_groups):
    sizes = [(7 * i) % 9 + 5 for i in range(n_groups)]
    sizes[0] = 40
    groups = [((37 * i) % 230 if i % 5 else 0, [(1, 1 + (3 * j + i) % 4) for j in range(n)])
              for i, n in enumerate(sizes)]
    b = S.make(n_groups, cuda_device, fmt, hq, hk, d, bs, groups)
    ref = S.reference(b)
    S.check(b, *b.call(), ref=ref)
    # one segment each
    ws = torch.zeros(256 + b.q.shape[0] * b.hq * 2 * (d + 2) * 4, dtype=torch.uint8,
                     device=cuda_device)
    S.check(b, *b.call(workspace=ws), ref=ref)


# one group of several row blocks over a prefix of many tiles, its last block
# part full; every block's share crosses units
@pytest.mark.parametrize("fmt,d,n,prefix", [("q8", 128, 150, 1700), ("q8", 64, 90, 2500),
                                            ("f8v4", 128, 129, 1100), ("q8", 256, 70, 1500),
                                               ("f8v4", 256, 33, 900), ("q8", 256, 32, 4100)])
def test_shares_cross_units(cuda_device, fmt, d, n, prefix):
    b = S.make(n, cuda_device, fmt, 8, 2, d, 16, [(prefix, [(1, 1 + i % 3) for i in range(n)])])
    ref = S.reference(b)
    S.check(b, *b.call(), ref=ref)
    full = _lib.shared_prefix_workspace_size(n, n, 1, 8, 2, d, *b.bounds)
    triple = n * 8 * (d + 2) * 4
    for slots in (2, 3, 4):  # fewer and fewer segments
        ws = torch.zeros(min(full, 256 + slots * triple), dtype=torch.uint8, device=cuda_device)
        S.check(b, *b.call(workspace=ws), ref=ref)


# the bounds of the prefixes and suffixes are hints, that of the query lengths an upper bound
@pytest.mark.parametrize("bounds", [(6, 0, 1), (6, 64, 64), (999, 99999, 99999), (7, 1, 100000)])
def test_bounds_are_hints(cuda_device, bounds):
    b = S.make(5, cuda_device, "q8", 8, 2, 128, 16, [(700, [(1, 300), (6, 80), (1, 2)]),
                                                     (5, [(1, 900)])])
    S.check(b, *b.call(bounds=bounds))


@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sinks(cuda_device, fmt, d):
    sinks = [-math.inf, 0.0, 30.0, -1.5]
    b = S.make(d, cuda_device, fmt, 4, 2, d, 16, [(90, [(1, 1), (3, 70)])], sinks=sinks)
    S.check(b, *b.call())


# peaked rows: large scores of either sign, the maximum late in the suffix or in the prefix
@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
@pytest.mark.parametrize("q_scale", [0.01, 12.0])
def test_score_ranges(cuda_device, fmt, q_scale):
    b = S.make(3, cuda_device, fmt, 8, 2, 128, 16, [(500, [(1, 200), (1, 5), (8, 30)])],
               q_scale=q_scale, k_bias=2.0)
    S.check(b, *b.call())


def test_softmax_scale(cuda_device):
    b = S.make(9, cuda_device, "q8", 4, 2, 64, 16, DECODE)
    S.check(b, *b.call(softmax_scale=0.3), scale=0.3)


def test_same_as_paged_attention(cuda_device):
    """The call's contract: where the rows share every page of the prefix, it
    computes what paged_attention does (both against one fp64 result)."""
    b = S.make(11, cuda_device, "q8", 32, 8, 128, 16, [(992, [(1, 1 + 40 * i) for i in range(12)])])
    ref = S.reference(b)
    S.check(b, *b.call(), ref=ref)
    S.check(b, *_lib.paged_attention(b.q, *b.cache, b.cu, b.lens, b.table, 1, max(b.seq_lens)),
            ref=ref)


def test_rows_of_bad_sequences_stay(cuda_device):
    """A sequence shorter than its prefix and query, one no group holds: flagged,
    their rows left as they were, the others right."""
    b = S.make(13, cuda_device, "q8", 4, 2, 64, 16, [(40, [(1, 5), (1, 6)]), (20, [(1, 9)])])
    ref = S.reference(b)
    good = b.lens.clone()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=cuda_device)
    for case in ("short", "outside", "table", "column"):
        lens, groups, table = good.clone(), b.groups.clone(), b.table.clone()
        if case == "short":
            lens[1] = 40
        elif case == "outside":
            groups[1:] = torch.tensor([1, 1], dtype=torch.int32)
        elif case == "table":
            table[1, 2] = b.blocks
        else:
            table = table[:, :2].contiguous()
        out = torch.full_like(b.q, float("nan"))
        lse = torch.full(b.q.shape[:2], float("nan"), device=cuda_device)
        _lib.paged_attention_shared_prefix(b.q, *b.cache, b.cu, lens, table, groups, b.prefixes,
                                           *b.bounds, out=out, lse=lse, workspace=ws)
        with pytest.raises(_lib.PagedAttentionError) as err:
            _lib.check_status(ws)
        assert err.value.bits == (_lib.DEV_BAD_BLOCK if case in ("table", "column")
                                  else _lib.DEV_BAD_SEQ)
        if case in ("short", "outside"):
            bad = [1] if case == "short" else [1, 2]
            assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
            assert torch.isfinite(out[0].float()).all()
            assert (lse[0].double().cpu() - ref[1][0]).abs().max() < 1e-3
    S.check(b, *b.call(), ref=ref)


def test_query_longer_than_its_bound_is_flagged(cuda_device):
    b = S.make(15, cuda_device, "q8", 8, 2, 128, 16, [(40, [(1, 5), (6, 9), (2, 4)])])
    ref = S.reference(b)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=cuda_device)
    out = torch.full_like(b.q, float("nan"))
    lse = torch.full(b.q.shape[:2], float("nan"), device=cuda_device)
    _lib.paged_attention_shared_prefix(b.q, *b.cache, b.cu, b.lens, b.table, b.groups, b.prefixes,
                                       2, 40, 9, out=out, lse=lse, workspace=ws)
    with pytest.raises(_lib.PagedAttentionError) as err:
        _lib.check_status(ws)
    assert err.value.bits == _lib.DEV_BAD_SEQ
    assert torch.isnan(out[1:7].float()).all() and torch.isnan(lse[1:7]).all()
    for rows in ([0], [7, 8]):
        assert (lse[rows].double().cpu() - ref[1][rows]).abs().max() < 1e-3


def test_q_outside_fp16_is_flagged(cuda_device):
    b = S.make(17, cuda_device, "q8", 4, 2, 64, 16, DECODE)
    b.q[1, 2, 5] = 1e6
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=cuda_device)
    _lib.paged_attention_shared_prefix(b.q, *b.cache, b.cu, b.lens, b.table, b.groups, b.prefixes,
                                       *b.bounds, workspace=ws)
    with pytest.raises(_lib.PagedAttentionError) as err:
        _lib.check_status(ws)
    assert err.value.bits == _lib.DEV_BAD_Q


def test_graph_replay_with_new_lengths(cuda_device):
    """A captured call replayed after its inputs changed in place: lengths,
    prefixes, tables and queries come from device memory."""
    first = S.make(21, cuda_device, "q8", 8, 2, 128, 16, [(200, [(1, 30)] * 6)], columns=30)
    other = S.make(22, cuda_device, "q8", 8, 2, 128, 16, [(90, [(1, 100), (1, 3)]),
                                                          (17, [(1, 7)] * 4)], columns=30)
    ref = S.reference(other)
    blocks = max(first.blocks, other.blocks)
    cache = [torch.zeros((blocks, *t.shape[1:]), dtype=t.dtype, device=cuda_device)
             for t in first.cache]
    cols = max(first.table.shape[1], other.table.shape[1])
    table = torch.full((6, cols), -1, dtype=torch.int32, device=cuda_device)
    groups = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    prefixes = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    q, cu, lens = first.q.clone(), first.cu.clone(), first.lens.clone()
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device=cuda_device)
    bounds = (1, 256, 128)
    ws = torch.zeros(_lib.shared_prefix_workspace_size(6, 6, 2, 8, 2, 128, *bounds),
                     dtype=torch.uint8, device=cuda_device)

    def fill(b, gr, pr):
        for t, x in zip(cache, b.cache):
            t[:x.shape[0]] = x
        table.fill_(-1)
        table[:, :b.table.shape[1]] = b.table
        groups.copy_(torch.tensor(gr))
        prefixes.copy_(torch.tensor(pr))
        q.copy_(b.q), cu.copy_(b.cu), lens.copy_(b.lens)

    def call():
        _lib.paged_attention_shared_prefix(q, *cache, cu, lens, table, groups, prefixes, *bounds,
                                           out=out, lse=lse, workspace=ws)

    fill(first, [0, 6, 6], [200, 0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    S.check(first, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    fill(other, [0, 2, 6], [90, 17])
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert _lib.check_status(ws) == 0
        S.check(other, out, lse, ref=ref)


def test_two_calls_on_two_streams(cuda_device):
    """Calls that overlap on the GPU, each with its own workspace."""
    a = S.make(31, cuda_device, "q8", 32, 4, 128, 16, [(900, [(1, 50)] * 24)])
    b = S.make(32, cuda_device, "f8v4", 8, 2, 128, 16, [(700, [(1, 90)] * 20)])
    alone = [x.call() for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = []
    for x in (a, b):
        need = _lib.shared_prefix_workspace_size(len(x.seq_lens), x.q.shape[0], 1, x.hq, x.hk,
                                                 x.d, *x.bounds)
        args.append((torch.empty_like(x.q), torch.empty(x.q.shape[:2], device=cuda_device),
                     torch.zeros(need, dtype=torch.uint8, device=cuda_device)))
    torch.cuda.synchronize()
    for _ in range(8):
        for x, st, (o, z, w) in zip((a, b), streams, args):
            fn = (_lib.paged_attention_shared_prefix if x.fmt == "q8"
                  else _lib.paged_attention_shared_prefix_f8v4)
            fn(x.q, *x.cache, x.cu, x.lens, x.table, x.groups, x.prefixes, *x.bounds, out=o, lse=z,
               workspace=w, stream=st)
    torch.cuda.synchronize()
    for (o, z, w), (ro, rz) in zip(args, alone):
        assert torch.equal(o, ro) and torch.equal(z, rz)  # the same bits, run after run


def test_allocates_its_results_when_omitted(cuda_device):
    b = S.make(41, cuda_device, "q8", 4, 2, 64, 16, DECODE)
    args = (b.q, *b.cache, b.cu, b.lens, b.table, b.groups, b.prefixes, *b.bounds)
    S.check(b, *_lib.paged_attention_shared_prefix(*args))
    out = _lib.paged_attention_shared_prefix(*args, return_lse=False)
    assert torch.equal(out, _lib.paged_attention_shared_prefix(*args)[0])
