"""The serving calls where an index, an order or a stream could go wrong: offsets
past 32 bits, work that wraps around the grid, graphs, streams, odd scales."""
import pytest
import torch

from paged_attention_int8_gb300 import _lib, inputs
from tests import _harness as H
from tests import _shared as S

pytestmark = pytest.mark.gpu


# rows of 9 - 16, 17 - 24 and 25 - 32 a sequence, several segments, scores that grow
# along the keys (the running offset moves) and that shrink
@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
@pytest.mark.parametrize("hq,hk,d,bs,q_len", [(8, 1, 128, 16, 2), (8, 1, 128, 32, 3), (8, 1, 128, 16, 4),
                                              (8, 1, 128, 32, 4), (16, 2, 64, 16, 4), (8, 1, 256, 16, 4),
                                              (5, 1, 128, 16, 6), (16, 1, 64, 32, 2)])
@pytest.mark.parametrize("q_scale", [1.0, 10.0])
def test_row_tiles(cuda_device, fmt, hq, hk, d, bs, q_len, q_scale):
    b = S.make(hq + q_len, cuda_device, fmt, hq, hk, d, bs,
               [(70, [(q_len, 900), (1, 1), (q_len - 1, 333)]), (9, [(q_len, q_len)])],
               q_scale=q_scale, k_bias=2.0)
    S.check(b, *b.call())


@pytest.mark.parametrize("n_groups", [30, 31, 32, 33])
def test_groups_about_a_warp(cuda_device, n_groups):
    groups = [(11 * i % 97, [(1, 1 + i % 70)] * (1 + i % 3)) for i in range(n_groups)]
    b = S.make(n_groups, cuda_device, "q8", 4, 1, 64, 16, groups)
    S.check(b, *b.call())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.07])
def test_scales_of_zero_and_below(cuda_device, d, scale):
    """Masked keys stay masked under a scale that is not positive."""
    b = S.make(d, cuda_device, "q8", 8, 2, d, 16, [(75, [(1, 1), (1, 70), (3, 9), (20, 31)]),
                                                  (40, [(1, 5)] * 20)])
    S.check(b, *b.call(softmax_scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
def test_pages_past_four_gigabytes(cuda_device, fmt):
    """Pages at the end of a cache whose K alone takes more than 2^32 bytes."""
    hk, d, bs = 2, 128, 16
    b = S.make(3, cuda_device, fmt, 16, hk, d, bs, [(100, [(1, 40)] * 9), (30, [(2, 9)])])
    ref = S.reference(b)
    blocks = (1 << 20) + (1 << 17)
    shapes = (inputs.cache_shapes if fmt == "q8" else inputs.cache_shapes_f8v4)(blocks, hk, bs, d)
    big = [torch.empty(s, dtype=t.dtype, device=cuda_device) for s, t in zip(shapes, b.cache)]
    assert big[0].numel() > 1 << 32
    first = blocks - b.blocks
    for t, x in zip(big, b.cache):
        t[first:] = x
    small, b.cache = b.cache, big
    table = b.table.clone()
    b.table = torch.where(table >= 0, table + first, table)
    S.check(b, *b.call(), ref=ref)
    # the copy: from the far end to the near one and back to other far blocks
    copy = _lib.copy_blocks if fmt == "q8" else _lib.copy_blocks_f8v4
    pairs = torch.tensor([[first + i, i] for i in range(b.blocks)], dtype=torch.int32,
                         device=cuda_device)
    copy(pairs, *big)
    far = torch.tensor([[i, first - b.blocks + i] for i in range(b.blocks)], dtype=torch.int32,
                       device=cuda_device)
    copy(far, *big)
    for t, x in zip(big, small):
        assert torch.equal(t[:b.blocks], x) and torch.equal(t[first - b.blocks:first], x)


def _filled(blocks, hk, d, bs, device, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(-100, 100, s, generator=g, dtype=torch.int8).to(device) if i % 2 == 0
            else torch.randint(0, 9999, s, generator=g, dtype=torch.int16).to(device)
            for i, s in enumerate(inputs.cache_shapes(blocks, hk, bs, d))]


# more parts than a grid takes 32 times over; parts that end inside each array;
# blocks of many parts; a hole in every few pairs
@pytest.mark.parametrize("pairs,hk,d,bs", [(30000, 1, 64, 16), (9000, 2, 128, 16), (5, 64, 256, 32),
                                           (1, 13, 256, 32), (700, 7, 64, 32)])
def test_copies_of_all_sizes(cuda_device, pairs, hk, d, bs):
    H.ensure_built()
    blocks = 2 * pairs + 1
    cache = _filled(blocks, hk, d, bs, cuda_device, pairs)
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(5)).to(cuda_device)
    p = torch.stack([order[:pairs], order[pairs:2 * pairs]], 1).to(torch.int32)
    if pairs > 9:
        p[3::7, 0] = -1
        p[5::11, 1] = p[5::11, 0]
    want = [t.clone() for t in cache]
    real = (p[:, 0] >= 0) & (p[:, 0] != p[:, 1])
    for t in want:
        t[p[real, 1].long()] = t[p[real, 0].long()]
    _lib.copy_blocks(p, *cache)
    for t, w in zip(cache, want):
        assert torch.equal(t, w)


def test_copy_captured_and_replayed_with_other_pairs(cuda_device):
    H.ensure_built()
    cache = _filled(40, 2, 128, 16, cuda_device, 1)
    pairs = torch.full((6, 2), -1, dtype=torch.int32, device=cuda_device)
    _lib.copy_blocks(pairs, *cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.copy_blocks(pairs, *cache)
    for step in range(3):
        pairs.copy_(torch.tensor([[step, 10 + step], [-1, 4], [step, 20 + step], [30, 30], [7, 35],
                                  [8, 36 + step]]))
        want = [t.clone() for t in cache]
        for a, b in pairs.tolist():
            if a >= 0:
                for w in want:
                    w[b] = w[a]
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(cache, want):
            assert torch.equal(t, w)


@pytest.mark.parametrize("fmt,d,hq,hk,q_len", [("q8", 256, 16, 2, 1), ("f8v4", 128, 8, 1, 4),
                                               ("q8", 64, 16, 1, 3), ("q8", 128, 4, 4, 40)])
def test_two_graphs_that_share_a_workspace(cuda_device, fmt, d, hq, hk, q_len):
    """Each of two captured calls, replayed in turn on one stream, leaves its own result."""
    a = S.make(1, cuda_device, fmt, hq, hk, d, 16, [(300, [(q_len, 50 + i) for i in range(6)])])
    b = S.make(2, cuda_device, fmt, hq, hk, d, 16, [(90, [(q_len, 41)] * 2), (5, [(q_len, 200)])])
    ws = torch.zeros(max(_lib.shared_prefix_workspace_size(
        len(x.seq_lens), x.q.shape[0], len(x.prefix), hq, hk, d, *x.bounds) for x in (a, b)),
        dtype=torch.uint8, device=cuda_device)
    fn = (_lib.paged_attention_shared_prefix if fmt == "q8"
          else _lib.paged_attention_shared_prefix_f8v4)
    runs = []
    for x in (a, b):
        out, lse = torch.empty_like(x.q), torch.empty(x.q.shape[:2], device=cuda_device)

        def call(x=x, out=out, lse=lse):
            fn(x.q, *x.cache, x.cu, x.lens, x.table, x.groups, x.prefixes, *x.bounds, out=out,
               lse=lse, workspace=ws)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((x, S.reference(x), graph, out, lse))
    for x, ref, graph, out, lse in (*runs, *reversed(runs)):
        out.fill_(float("nan")), lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert _lib.check_status(ws) == 0
        S.check(x, out, lse, ref=ref)


def test_omitted_results_belong_to_the_calls_stream(cuda_device):
    """Results and workspace that a call allocates for another stream than the
    current one are not handed out again before that stream has used them."""
    b = S.make(51, cuda_device, "q8", 8, 2, 128, 16, [(400, [(1, 60)] * 20)])
    want = b.call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    ctx, one, free = i32([5, 40]), i32([1, 1]), torch.arange(30, dtype=torch.int32, device=cuda_device)
    source = i32([[7, -1, -1, -1], [8, 9, 10, -1]])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = _lib.paged_attention_shared_prefix(b.q, *b.cache, b.cu, b.lens, b.table, b.groups,
                                             b.prefixes, *b.bounds, stream=side)
    tables = _lib.build_block_tables(ctx, one, source, free, 30, 16, 2, stream=side)
    need = _lib.shared_prefix_workspace_size(20, 20, 1, 8, 2, 128, *b.bounds)
    for _ in range(4):  # what the current stream allocates meanwhile, overwritten
        other = [torch.full((need,), 0xFF, dtype=torch.uint8, device=cuda_device) for _ in range(3)]
        del other
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert tables.block_table.tolist() == [[7, -1, -1, -1], [8, 9, 10, -1]]
    assert tables.slot_mapping.tolist() == [7 * 16 + 5, 10 * 16 + 8]


@pytest.mark.parametrize("fmt,hq,hk,d,q_len", [("q8", 8, 2, 128, 1), ("q8", 8, 2, 256, 1),
                                               ("f8v4", 2, 2, 64, 3), ("q8", 16, 1, 128, 9)])
@pytest.mark.parametrize("n", [2, 24])
def test_lengths_past_the_table_end_there(cuda_device, fmt, hq, hk, d, q_len, n):
    """Lengths that no table row can hold (the largest int32): flagged, walked no
    further than the table's columns, and the other group's rows right."""
    b = S.make(61, cuda_device, fmt, hq, hk, d, 16, [(90, [(q_len, 33)] * n), (40, [(q_len, 30)] * n)])
    ref = S.reference(b)
    fn = (_lib.paged_attention_shared_prefix if fmt == "q8"
          else _lib.paged_attention_shared_prefix_f8v4)
    lens, prefixes = b.lens.clone(), b.prefixes.clone()
    lens[n:] = 2 ** 31 - 1
    good = n * q_len
    for prefix in (40, 2 ** 31 - 100):
        prefixes[1] = prefix
        ws = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device)
        out, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=cuda_device)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        fn(b.q, *b.cache, b.cu, lens, b.table, b.groups, prefixes, *b.bounds, out=out, lse=lse,
           workspace=ws)
        end.record()
        with pytest.raises(_lib.PagedAttentionError) as err:
            _lib.check_status(ws)
        assert err.value.bits == _lib.DEV_BAD_BLOCK
        assert start.elapsed_time(end) < 50  # ms; 2^31 keys would take seconds
        # fp32 sums; bf16 rounds |out| < 4 by 2^-7 at most, fp16 P and V' by 2^-10 of it
        assert (lse[:good].double().cpu() - ref[1][:good]).abs().max() < 1e-3
        assert (out[:good].double().cpu() - ref[0][:good]).abs().max() < 2e-2


def test_groups_that_name_no_sequence(cuda_device):
    """Group bounds out of order and past the batch: nothing out of range is read,
    the rows no group holds stay."""
    b = S.make(63, cuda_device, "q8", 8, 2, 128, 16, [(64, [(1, 20)] * 20), (32, [(1, 9)] * 20)])
    for groups in ([0, 40, 0], [40, 0, 40], [0, 41, 40], [-1, 20, 40], [0, 2 ** 31 - 1, 40]):
        ws = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device)
        out = torch.full_like(b.q, float("nan"))
        bad = torch.tensor(groups, dtype=torch.int32, device=cuda_device)
        cu = b.cu.clone()
        cu[-1] = 39
        _lib.paged_attention_shared_prefix(b.q, *b.cache, cu, b.lens, b.table, bad, b.prefixes,
                                           *b.bounds, out=out, workspace=ws)
        try:
            _lib.check_status(ws)
        except _lib.PagedAttentionError as err:
            assert err.bits & ~(_lib.DEV_BAD_SEQ | _lib.DEV_BAD_BLOCK) == 0
        assert torch.isnan(out[39].float()).all()


@pytest.mark.parametrize("fmt,d,hq,hk,n,q_len", [("q8", 128, 8, 1, 20, 1), ("q8", 256, 16, 2, 12, 1),
                                                 ("f8v4", 64, 4, 2, 3, 1), ("q8", 128, 8, 2, 3, 20),
                                                 ("q8", 128, 4, 2, 2, 1)])
@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "kernel", "branches", "call"])
def test_reads_what_was_written_just_before(cuda_device, fmt, d, hq, hk, n, q_len, before):
    """The call's kernels start only after the work before it on the stream: its
    inputs become right right before it, by every kind of work that can stand there,
    eagerly and in a captured graph."""
    b = S.make(71, cuda_device, fmt, hq, hk, d, 16, [(200, [(q_len, 50)] * n)])
    ref = S.reference(b)
    fn = (_lib.paged_attention_shared_prefix if fmt == "q8"
          else _lib.paged_attention_shared_prefix_f8v4)
    q, cu, lens, groups, prefixes = (torch.empty_like(t) for t in (b.q, b.cu, b.lens, b.groups,
                                                                   b.prefixes))
    pairs = list(zip((q, cu, lens, groups, prefixes), (b.q, b.cu, b.lens, b.groups, b.prefixes)))
    out, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=cuda_device)
    ws = torch.zeros(_lib.shared_prefix_workspace_size(n, b.q.shape[0], 1, hq, hk, d, *b.bounds),
                     dtype=torch.uint8, device=cuda_device)
    side = torch.cuda.Stream()
    other = torch.empty(1 << 24, device=cuda_device)

    def call(x=q):
        fn(x, *b.cache, cu, lens, b.table, groups, prefixes, *b.bounds, out=out, lse=lse,
           workspace=ws)

    def run():
        other.fill_(1.0)
        for t, x in pairs:
            t.copy_(x)
        if before == "memset":
            lse.view(torch.uint8).zero_()
        elif before == "kernel":
            for t, x in pairs:
                torch.add(x, 0, out=t)
        elif before == "branches":
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                other.mul_(2.0)
                q.copy_(b.q)
            cu.copy_(b.cu)
            main.wait_stream(side)
        elif before == "call":
            call(torch.zeros_like(q))
        call()

    def spoil():
        for t, _ in pairs:
            t.zero_()
        out.fill_(float("nan")), lse.fill_(float("nan"))

    def verify():
        torch.cuda.synchronize()
        assert _lib.check_status(ws) == 0
        S.check(b, out, lse, ref=ref)

    if before != "nothing":
        for _ in range(3):
            spoil()
            torch.cuda.synchronize()
            run()
            verify()
    for t, x in pairs:
        t.copy_(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call() if before == "nothing" else run()
    for _ in range(3):
        if before != "nothing":
            spoil()
        torch.cuda.synchronize()
        graph.replay()
        verify()


@pytest.mark.parametrize("before", ["memset", "copy", "kernel", "branches", "call"])
@pytest.mark.parametrize("captured", [False, True])
def test_tables_and_copies_follow_what_was_before(cuda_device, before, captured):
    """The same of the single-kernel calls: tables from lengths written just before,
    then a copy by the pairs they made, from blocks written just before."""
    H.ensure_built()
    dev = cuda_device
    n, columns, bs = 40, 300, 16
    ctx_good = torch.arange(n, dtype=torch.int32, device=dev) * 101 + 7
    one, free = torch.ones(n, dtype=torch.int32, device=dev), torch.arange(5000, 5100, dtype=torch.int32,
                                                                           device=dev)
    source = torch.arange(n * columns, dtype=torch.int32, device=dev).view(n, columns) % 4000
    blocks = 6000
    cache = _filled(blocks, 1, 64, bs, dev, 9)
    fresh = [t.clone() for t in cache]
    ctx = torch.zeros_like(ctx_good)
    side = torch.cuda.Stream()
    other = torch.empty(1 << 24, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    t = _lib.build_block_tables(ctx, one, source, free, blocks, bs, n,
                                source_rows=torch.arange(n, dtype=torch.int32, device=dev),
                                shared_lens=ctx_good)
    rows = torch.arange(n, dtype=torch.int32, device=dev)

    def run():
        other.fill_(1.0)
        ctx.copy_(ctx_good)
        for x, y in zip(cache, fresh):
            x.copy_(y)
        if before == "memset":
            t.copy_pairs.zero_()
        elif before == "kernel":
            torch.add(ctx_good, 0, out=ctx)
        elif before == "branches":
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                other.mul_(2.0)
                ctx.copy_(ctx_good)
            main.wait_stream(side)
        elif before == "call":
            _lib.copy_blocks(t.copy_pairs, *cache)
            for x, y in zip(cache, fresh):
                x.copy_(y)
        _lib.build_block_tables(ctx, one, source, free, blocks, bs, n, source_rows=rows,
                                shared_lens=ctx_good, out=t, status=status)
        _lib.copy_blocks(t.copy_pairs, *cache, status=status)

    # on the host: every sequence's last page is shared and partly filled, or full
    c = ctx_good.tolist()
    dealt, pairs = 5000, []
    for s in range(n):
        pairs.append([int(source[s, c[s] // bs]), dealt] if c[s] % bs else [-1, -1])
        dealt += 1
    want = [x.clone() for x in fresh]
    for a, b in pairs:
        if a >= 0:
            for x, y in zip(want, fresh):
                x[b] = y[a]
    run()
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(4):
        ctx.zero_(), t.copy_pairs.fill_(-1)
        for x in cache:
            x.zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert _lib.check_status(status) == 0
        assert t.copy_pairs.tolist() == pairs and t.seq_lens.tolist() == [x + 1 for x in c]
        for x, y in zip(cache, want):
            assert torch.equal(x, y)


# so many rows that a warp of the join takes two, four or more channel blocks in turn
@pytest.mark.parametrize("fmt,hq,hk,d,n,pad", [("q8", 64, 8, 128, 100, 0), ("f8v4", 64, 4, 128, 200, 3),
                                               ("q8", 32, 8, 256, 170, 1), ("q8", 16, 16, 64, 701, 5)])
def test_many_rows_to_join(cuda_device, fmt, hq, hk, d, n, pad):
    b = S.make(n, cuda_device, fmt, hq, hk, d, 16,
               [(30, [(1, 1 + i % 5) for i in range(n - 7)]), (17, [(1, 2)] * 7)], pad_rows=pad)
    S.check(b, *b.call())
