"""build_block_tables and copy_blocks against plain implementations, and a
serving loop of all the shared-prefix calls together."""
import random

import numpy as np
import pytest
import torch

from paged_attention_int8_gb300 import _lib, inputs
from tests import _harness as H
from tests import _shared as S

pytestmark = pytest.mark.gpu


def _plan(ctx, q, source, rows, shared, free, head, bs, tokens, table):
    """The definition, one sequence after the other (numpy; table written in
    place of a copy)."""
    table = table.copy()
    n = len(ctx)
    cu, slots = [0], np.full(tokens, -1, np.int64)
    pos, pairs = np.zeros(tokens, np.int64), np.full((n, 2), -1, np.int64)
    for s in range(n):
        c, ql = ctx[s], q[s]
        row = source[s if rows is None else rows[s]]
        held, end = -(-c // bs), -(-(c + ql) // bs)
        pages = list(row[:held])
        if ql and c % bs and shared is not None and shared[s] > c - c % bs:
            pairs[s] = pages[-1], free[head]
            pages[-1] = free[head]
            head += 1
        while len(pages) < end:
            pages.append(free[head])
            head += 1
        table[s, :len(pages)] = pages
        for i in range(ql):
            x = c + i
            slots[cu[-1] + i] = int(pages[x // bs]) * bs + x % bs
            pos[cu[-1] + i] = x
        cu.append(cu[-1] + ql)
    return table, cu, [a + b for a, b in zip(ctx, q)], slots, pos, pairs, [head]


def _case(seed, n, bs, ctx_max, q_max, rows=None, fork=False, pad=0):
    r = random.Random(seed)
    n_rows = rows or n
    row_of = [r.randrange(n_rows) for _ in range(n)] if fork else (
        r.sample(range(n_rows), n) if rows else None)
    row_ctx = [r.choice([0, 1, bs - 1, bs, bs + 1, r.randint(0, ctx_max)]) for _ in range(n_rows)]
    ctx = [row_ctx[s if row_of is None else row_of[s]] for s in range(n)]
    q = [r.choice([0, 1, 1, 1, bs, r.randint(0, q_max)]) for _ in range(n)]
    shared = None
    if fork:
        shared = [r.choice([0, c, c - c % bs, max(0, c - 1)]) for c in ctx]
    columns = max([-(-(a + b) // bs) for a, b in zip(ctx, q)]
                  + [-(-c // bs) for c in row_ctx]) + r.randrange(4) + 1
    blocks = sum(-(-c // bs) for c in row_ctx) + sum(-(-x // bs) + 1 for x in q) + 5
    ids = list(range(blocks))
    r.shuffle(ids)
    source = np.full((n_rows, columns), -1, np.int32)
    for i, c in enumerate(row_ctx):
        for p in range(-(-c // bs)):
            source[i, p] = ids.pop()
    head = r.randrange(3)
    free = np.array([-1] * head + ids, np.int32)
    return ctx, q, source, row_of, shared, free, head, blocks, sum(q) + pad


CASES = [dict(seed=1, n=1, bs=16, ctx_max=5, q_max=1), dict(seed=2, n=8, bs=16, ctx_max=200, q_max=1),
         dict(seed=3, n=9, bs=32, ctx_max=500, q_max=70, pad=13),
         dict(seed=4, n=100, bs=16, ctx_max=900, q_max=3, rows=130),
         dict(seed=5, n=257, bs=32, ctx_max=300, q_max=2, rows=20, fork=True),
         dict(seed=6, n=64, bs=16, ctx_max=64, q_max=2, rows=3, fork=True, pad=2000),
         dict(seed=7, n=5, bs=16, ctx_max=40000, q_max=5000, rows=6),
         dict(seed=8, n=3, bs=16, ctx_max=70000, q_max=40, rows=2, fork=True)]


def _run(dev, ctx, q, source, rows, shared, free, head, blocks, tokens, bs, in_place=False,
         defaults=False):
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    n = len(ctx)
    src = torch.from_numpy(source.copy()).to(dev)
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    out = None
    if not defaults:
        table = src if in_place else torch.full((n, source.shape[1]), -7, dtype=torch.int32,
                                                device=dev)
        out = (table, i32([9] * (n + 1)), i32([9] * n),
               torch.full((tokens,), 9, dtype=torch.int64, device=dev),
               torch.full((tokens,), 9, dtype=torch.int64, device=dev), i32([[9, 9]] * n),
               i32([9]))
    got = _lib.build_block_tables(i32(ctx), i32(q), src, torch.from_numpy(free).to(dev), blocks,
                                  bs, tokens, source_rows=i32(rows), shared_lens=i32(shared),
                                  free_head=i32([head]), out=out, status=status)
    assert _lib.check_status(status) == 0
    return got


def _same(got, want):
    for name, g, w in zip(got._fields, got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), np.asarray(w), err_msg=name)


@pytest.mark.parametrize("kw", CASES, ids=lambda k: f"{k['seed']}")
def test_build_block_tables(cuda_device, kw):
    H.ensure_built()
    ctx, q, source, rows, shared, free, head, blocks, tokens = _case(**kw)
    args = (ctx, q, source, rows, shared, free, head, blocks, tokens, kw["bs"])
    untouched = np.full((len(ctx), source.shape[1]), -7, np.int32)
    want = _plan(ctx, q, source, rows, shared, free, head, kw["bs"], tokens, untouched)
    _same(_run(cuda_device, *args), want)
    fresh = _plan(ctx, q, source, rows, shared, free, head, kw["bs"], tokens,
                  np.full_like(untouched, -1))
    _same(_run(cuda_device, *args, defaults=True), fresh)
    if rows is None:
        want = _plan(ctx, q, source, rows, shared, free, head, kw["bs"], tokens, source)
        _same(_run(cuda_device, *args, in_place=True), want)


# private copies of pages far down a wide row, the table extended in place
@pytest.mark.parametrize("bs", [16, 32])
def test_private_pages_in_place(cuda_device, bs):
    H.ensure_built()
    n, held = 21, 2100
    ctx = [held * bs - 1 - i for i in range(n)]
    q = [1 + 3 * (i % 2) for i in range(n)]
    r = np.random.default_rng(bs)
    blocks = n * (held + 3)
    ids = r.permutation(blocks).astype(np.int32)
    source = np.full((n, held + 2), -1, np.int32)
    source[:, :held] = ids[:n * held].reshape(n, held)
    args = (ctx, q, source, None, ctx, ids[n * held:], 0, blocks, sum(q), bs)
    want = _plan(ctx, q, source, None, ctx, ids[n * held:], 0, bs, sum(q), source)
    for _ in range(5):
        _same(_run(cuda_device, *args, in_place=True), want)


def test_no_sequence(cuda_device):
    H.ensure_built()
    e = lambda *s: torch.empty(s, dtype=torch.int32, device=cuda_device)  # noqa: E731
    got = _lib.build_block_tables(e(0), e(0), e(1, 4), e(0), 3, 16, 7)
    assert got.cu_seqlens_q.tolist() == [0] and got.slot_mapping.tolist() == [-1] * 7
    assert got.positions.tolist() == [0] * 7 and got.next_free.tolist() == [0]


@pytest.mark.parametrize("case,bit", [("negative", "BAD_SEQ"), ("query", "BAD_SEQ"),
                                      ("tokens", "BAD_SEQ"), ("row", "BAD_SEQ"),
                                      ("columns", "BAD_BLOCK"), ("old", "BAD_BLOCK"),
                                      ("freeid", "BAD_BLOCK"), ("free", "NO_BLOCKS"),
                                      ("head", "NO_BLOCKS")])
def test_bad_metadata_is_flagged(cuda_device, case, bit):
    """Bad entries set their bit, touch nothing out of bounds and leave the
    other sequences' results as they should be."""
    H.ensure_built()
    bs, dev = 16, cuda_device
    ctx, q, rows = [20, 33, 16], [1, 2, 16], [0, 1, 2]
    source = np.array([[1, 2, -1, -1], [3, 4, 5, -1], [6, -1, -1, -1]], np.int32)
    free, head, tokens, blocks = np.array([8, 9], np.int32), 0, 19, 10
    if case == "negative":
        ctx[1] = -4
    elif case == "query":
        q[1] = 1 << 30
    elif case == "tokens":
        tokens = 10
    elif case == "row":
        rows[1] = 3
    elif case == "columns":
        source = source[:, :1].copy()
    elif case == "old":
        source[1, 2] = 99
    elif case == "freeid":
        free[0] = 10
    elif case == "free":
        free = free[:0]
    elif case == "head":
        head = -1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    # guard rows around every output
    guard = lambda n, dt: torch.full((n + 64,), 77, dtype=dt, device=dev)  # noqa: E731
    g = [guard(3 * source.shape[1], torch.int32), guard(4, torch.int32), guard(3, torch.int32),
         guard(tokens, torch.int64), guard(tokens, torch.int64), guard(6, torch.int32),
         guard(1, torch.int32)]
    cut = [x[32:-32] for x in g]
    out = (cut[0].view(3, -1), cut[1], cut[2], cut[3], cut[4], cut[5].view(3, 2), cut[6])
    got = _lib.build_block_tables(i32(ctx), i32(q), torch.from_numpy(source).to(dev),
                                  torch.from_numpy(free).to(dev), blocks, bs, tokens,
                                  source_rows=i32(rows), free_head=i32([head]), out=out,
                                  status=status)
    with pytest.raises(_lib.PagedAttentionError) as err:
        _lib.check_status(status)
    assert err.value.bits == getattr(_lib, "DEV_" + bit)
    for x in g:
        assert (x[:32] == 77).all() and (x[-32:] == 77).all()
    slots = got.slot_mapping.tolist()
    if case != "columns":
        assert slots[0] == 2 * bs + 4  # the first sequence's token is right in every case
    if case in ("negative", "query"):
        assert got.seq_lens.tolist() == [21, 0, 32] and got.cu_seqlens_q.tolist() == [0, 1, 1, 17]
        assert got.block_table[2].tolist()[:2] == [6, 8] and slots[1:17] == list(range(128, 144))
        assert slots[17:] == [-1, -1]
    if case in ("free", "head", "freeid"):
        assert slots[3:] == [-1] * 16 and got.block_table[2].tolist()[:2] == [6, -1]
    if case in ("old", "row"):
        assert slots[1:3] == [-1, -1] and slots[3:] == list(range(128, 144))
    if case == "columns":
        assert slots[:3] == [-1] * 3


# ------------------------------------------------------------------ copies

@pytest.mark.parametrize("fmt", ["q8", "f8v4"])
@pytest.mark.parametrize("hk,d,bs", [(1, 64, 16), (2, 128, 16), (3, 256, 32), (8, 128, 32)])
@pytest.mark.parametrize("pairs", [1, 7, 60])
def test_copy_blocks(cuda_device, fmt, hk, d, bs, pairs):
    H.ensure_built()
    blocks = 2 * pairs + 3
    g = torch.Generator().manual_seed(pairs * d)
    shapes = (inputs.cache_shapes if fmt == "q8" else inputs.cache_shapes_f8v4)(blocks, hk, bs, d)
    dtypes = ((torch.int8, torch.int16, torch.int8, torch.int16) if fmt == "q8"
              else (torch.uint8, torch.uint8, torch.int16, torch.int16))
    cache = [torch.randint(0, 120, s, generator=g, dtype=t) for s, t in zip(shapes, dtypes)]
    perm = torch.randperm(blocks, generator=g)
    p = torch.stack([perm[:pairs], perm[pairs:2 * pairs]], 1)
    if pairs > 5:
        p[1, 0] = p[0, 0]                      # one source, two destinations
        p[2] = -1                              # padding
        p[3, 0] = -1                           # no source
        p[4, 1] = -5                           # no destination
        p[5, 1] = p[5, 0]                      # onto itself
    want = [t.clone() for t in cache]
    for a, b in p.tolist():
        if a >= 0 and b >= 0:
            for t, w in zip(cache, want):
                w[b] = t[a]
    dev = [t.to(cuda_device) for t in cache]
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    fn = _lib.copy_blocks if fmt == "q8" else _lib.copy_blocks_f8v4
    fn(p.to(torch.int32).to(cuda_device), *dev, status=status)
    assert _lib.check_status(status) == 0
    for t, w in zip(dev, want):
        assert torch.equal(t.cpu(), w)


def test_copy_blocks_flags_bad_ids_and_takes_no_pairs(cuda_device):
    H.ensure_built()
    cache = [t.clone() for t in inputs.empty_cache(4, 2, 16, 64, device=cuda_device)]
    cache[0].random_(-100, 100)
    before = [t.clone() for t in cache]
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    _lib.copy_blocks(torch.empty((0, 2), dtype=torch.int32, device=cuda_device), *cache,
                     status=status)
    assert _lib.check_status(status) == 0
    pairs = torch.tensor([[0, 4], [9, 1], [2, 3]], dtype=torch.int32, device=cuda_device)
    _lib.copy_blocks(pairs, *cache, status=status)
    with pytest.raises(_lib.PagedAttentionError) as err:
        _lib.check_status(status)
    assert err.value.bits == _lib.DEV_BAD_BLOCK
    for t, b in zip(cache, before):
        assert torch.equal(t[:3], b[:3]) and torch.equal(t[3], b[2])


# ------------------------------------------------------- a run of them all

@pytest.mark.parametrize("fmt,hq,hk,d,bs", [("q8", 8, 2, 128, 16), ("f8v4", 4, 2, 64, 32),
                                            ("q8", 4, 1, 256, 16)])
def test_fork_and_decode(cuda_device, fmt, hq, hk, d, bs):
    """Two prompts are stored, each is forked into samples, and the samples
    decode several steps: tables, copies, stores and shared attention, every
    step's attention against fp64 over rows kept on the host."""
    H.ensure_built()
    dev = cuda_device
    g = torch.Generator().manual_seed(7)
    prompts, samples, steps = [bs * 3 + 5, bs * 2], [5, 3], 3
    n = sum(samples)
    blocks, columns = 64, 12
    make = inputs.empty_cache if fmt == "q8" else inputs.empty_cache_f8v4
    cache = list(make(blocks, hk, bs, d, device=dev))
    store = _lib.kv_store if fmt == "q8" else _lib.kv_store_f8v4
    copy = _lib.copy_blocks if fmt == "q8" else _lib.copy_blocks_f8v4
    attend = (_lib.paged_attention_shared_prefix if fmt == "q8"
              else _lib.paged_attention_shared_prefix_f8v4)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    rows = lambda k: torch.randn((k, hk, d), generator=g).bfloat16()  # noqa: E731
    free = torch.randperm(blocks, generator=g).to(torch.int32).to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    # the prompts, prefilled
    t = _lib.build_block_tables(i32([0, 0]), i32(prompts), torch.full((2, columns), -1,
                                dtype=torch.int32, device=dev), free, blocks, bs, sum(prompts),
                                status=status)
    k, v = rows(sum(prompts)), rows(sum(prompts))
    store(k.to(dev), v.to(dev), t.slot_mapping, *cache, status=status)
    host_k, host_v = list(k.split(prompts)), list(v.split(prompts))
    # the samples: each on its prompt's pages, a page half full copied before it is written
    owner = [0] * samples[0] + [1] * samples[1]
    ctx = [prompts[o] for o in owner]
    host_k, host_v = [host_k[o] for o in owner], [host_v[o] for o in owner]
    source, source_rows, shared = t.block_table, i32(owner), i32(ctx)
    groups, prefixes = i32([0, samples[0], n]), i32(prompts)
    for step in range(steps):
        t2 = _lib.build_block_tables(i32(ctx), i32([1] * n), source, free, blocks, bs, n + 2,
                                     source_rows=source_rows, shared_lens=shared,
                                     free_head=t.next_free, status=status)
        copy(t2.copy_pairs, *cache, status=status)
        made = (t2.copy_pairs[:, 0] >= 0).tolist()
        assert made == [step == 0 and prompts[o] % bs != 0 for o in owner]
        k, v = rows(n + 2), rows(n + 2)
        store(k.to(dev), v.to(dev), t2.slot_mapping, *cache, status=status)
        for s in range(n):
            host_k[s] = torch.cat([host_k[s], k[s:s + 1]])
            host_v[s] = torch.cat([host_v[s], v[s:s + 1]])
        q = torch.randn((n + 2, hq, d), generator=g).bfloat16().to(dev)
        b = S.Batch(fmt, hq, hk, d, bs, prompts, [0, samples[0], n], [1] * n,
                    [c + 1 for c in ctx], cache, t2.block_table, q, t2.cu_seqlens_q, t2.seq_lens,
                    groups, prefixes, None, blocks)
        assert t2.seq_lens.tolist() == b.seq_lens and t2.positions.tolist() == ctx + [0, 0]
        S.check(b, *b.call(), where=f"step {step}")
        # the pages hold what was stored, position by position: against a cache of its own
        for s in range(n):
            own = list(make(columns, hk, bs, d, device=dev))
            m = ctx[s] + 1
            store(host_k[s].to(dev), host_v[s].to(dev), torch.arange(m, device=dev), *own)
            mine = S.Batch(fmt, hq, hk, d, bs, [0], [0, 1], [1], [m], own, None, q, None, None,
                           None, None, None, columns)
            a = S._rows(b, t2.block_table[s].cpu(), 0, m)
            w = S._rows(mine, torch.arange(columns), 0, m)
            assert torch.equal(a[0], w[0]) and torch.equal(a[1], w[1])
        # on: this step's table is the next one's source
        t, source, source_rows, shared = t2, t2.block_table, None, None
        ctx = [c + 1 for c in ctx]
    assert _lib.check_status(status) == 0


# --------------------------------------------------------- the bindings' checks

def test_bindings_refuse_what_the_calls_cannot_take(cuda_device):
    """Types, layouts and shapes, each refused before anything is launched."""
    H.ensure_built()
    dev = cuda_device
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    good = dict(context_lens=i32(2), query_lens=i32(2), source_table=i32(2, 4), free_blocks=i32(3),
                num_blocks=4, block_size=16, num_tokens=2)
    _lib.build_block_tables(**good)
    for bad in (dict(query_lens=i32(3)), dict(context_lens=i32(2).long()),
                dict(source_table=i32(4, 4)[:, ::2]), dict(source_table=i32(8)),
                dict(free_blocks=i32(3).cpu()), dict(source_rows=i32(1)), dict(shared_lens=i32(5)),
                dict(free_head=i32(0)), dict(num_tokens=-1), dict(query_lens=i32(4)[::2])):
        with pytest.raises((TypeError, ValueError)):
            _lib.build_block_tables(**{**good, **bad})
    out = list(_lib.build_block_tables(**good))
    for at, t in ((0, i32(3, 4)), (1, i32(2)), (2, i32(2).long()), (3, i32(2)), (3, i32(3).long()),
                  (5, i32(2, 3)), (6, i32(0))):
        with pytest.raises((TypeError, ValueError)):
            _lib.build_block_tables(**good, out=out[:at] + [t] + out[at + 1:])
    with pytest.raises(_lib.PagedAttentionError):  # next_free over free_head
        head = i32(1)
        _lib.build_block_tables(**good, free_head=head, out=out[:6] + [head])
    cache = inputs.empty_cache(4, 2, 16, 64, device=dev)
    pairs = i32(1, 2)
    _lib.copy_blocks(pairs, *cache)
    for args in ((pairs.long(), *cache), (i32(2), *cache), (pairs, cache[0].float(), *cache[1:]),
                 (pairs, cache[0], cache[1], cache[0], cache[3]), (pairs, cache[0].cpu(), *cache[1:]),
                 (pairs, cache[0].transpose(1, 2), *cache[1:]),
                 (pairs, cache[0], cache[1].float(), *cache[2:])):
        with pytest.raises((TypeError, ValueError)):
            _lib.copy_blocks(*args)
    b = S.make(1, dev, "q8", 4, 2, 64, 16, [(20, [(1, 5)])])
    args = dict(q=b.q, k_cache=b.cache[0], k_scale=b.cache[1], v_cache=b.cache[2],
                v_scale=b.cache[3], cu_seqlens_q=b.cu, seq_lens=b.lens, block_table=b.table,
                cu_groups=b.groups, prefix_lens=b.prefixes, max_query_len=1, max_prefix_len=20,
                max_suffix_len=5)
    _lib.paged_attention_shared_prefix(**args)
    for bad in (dict(q=b.q.float()), dict(q=b.q.cpu()), dict(seq_lens=b.lens.long()),
                dict(block_table=b.table.long()), dict(cu_groups=b.groups[:1]),
                dict(cu_seqlens_q=b.cu[:1]), dict(sinks=torch.zeros(3, device=dev)),
                dict(sinks=torch.zeros(4, device=dev).half()), dict(out=b.q.float()),
                dict(lse=torch.zeros((1, 3), device=dev)), dict(q=b.q[:, :, :32].contiguous()),
                dict(workspace=torch.zeros(64, dtype=torch.uint8)),
                dict(block_table=b.table.t().contiguous().t())):
        if "block_table" in bad and bad["block_table"].dtype == torch.int32 \
                and bad["block_table"].stride(1) == 1:
            continue
        with pytest.raises((TypeError, ValueError)):
            _lib.paged_attention_shared_prefix(**{**args, **bad})
    with pytest.raises(_lib.PagedAttentionError):  # too small for two triples a row
        _lib.paged_attention_shared_prefix(**args, workspace=torch.zeros(
            512, dtype=torch.uint8, device=dev))
