"""The 4-bit cache and prompt_attention as a server uses them: together over the life of
its sequences, captured and replayed, on other streams, with bad tables and lengths, and with
values where a narrow format could lose them.

Bounds per value as those of the single operators (half a bf16 step of the output, 2^-8; p and
p * scale in fp16, 2^-11 each; p in bf16 for prompts, 2^-8).  Below fp16's normal range p and
p * scale are off by 2^-25 against a largest p of at least 2^10: 2^-35 a key and unit of its
codes (15) and zero, or 2^-25 where a scale of 16 and more stands in the cache."""
import math

import pytest
import torch

from paged_attention_int8_gb300 import _lib
from tests import _harness as H
from tests import _q4

pytestmark = pytest.mark.gpu


def _i32(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


def _starts(lens, device):
    return torch.tensor([0] + list(lens)).cumsum(0).int().to(device)


def _table(lens, bs, spare=2, seed=0):
    """A table [S, most pages + 1] of pages in random order, and the pages of its cache."""
    pages = [-(-n // bs) for n in lens]
    perm = torch.randperm(sum(pages) + spare, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(lens), max(1, max(pages)) + 1), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(pages):
        table[s, :c] = perm[at:at + c]
        at += c
    return table, sum(pages) + spare


def _slots(table, bs, spans):
    """Slots of the tokens start .. end - 1 of every sequence."""
    pos = torch.cat([torch.arange(a, b) for a, b in spans])
    seq = torch.cat([torch.full((b - a,), s) for s, (a, b) in enumerate(spans)])
    return table[seq, pos // bs].long() * bs + pos % bs


def _compare(out, lse, q, parts, pos, lift=35, p_bits=None, **kw):
    """One sequence against 64 bits: parts as _q4.attention64's; p_bits: p's rounding of
    prompts (bf16), else that of the 4-bit attention."""
    ref, z, vc, vz, _, reach = _q4.attention64(q, parts, pos, **kw)
    d, n = q.shape[-1], parts[0].shape[0]
    scale = abs(kw.get("scale") or d ** -0.5)
    if p_bits is None:
        eps = 2.0 ** -17 * reach + scale * 2.0 ** -21 * (float(parts[0].abs().amax()) * d if n else 0.0)
    else:
        eps = d * 2.0 ** -23 * reach
    low = n * 2.0 ** -lift * (15 + (float(parts[3].abs().max()) if n else 0.0))
    if p_bits is None:
        tol = 1.01 * (2.0 ** -10 * vc + 2.0 ** -11 * vz) + low
    else:
        tol = 1.01 * 2.0 ** -p_bits * (vc + vz)
    tol = tol + 2.0 ** -8 * ref.abs() + (2 * eps[..., None] + 2.0 ** -20) * (vc + vz) + 1e-30
    err = (out.double() - ref).abs()
    assert not torch.isnan(out).any()
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    if lse is not None:
        e = (lse.double() - z).abs()
        assert (e <= eps + 2.0 ** -20 * (1 + z.abs())).all(), float(e.max())


# ----------------------------------------------------------------- values of all sizes

@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (8, 2, 128), (6, 2, 256), (32, 2, 128)])
@pytest.mark.parametrize("spread", [1e-3, 1e-2, 1.0])
@pytest.mark.parametrize("splits", [1, 4])
def test_small_weights_of_small_scales(cuda_device, hq, hk, d, spread, splits):
    """One key takes most of a row's weight, 5000 others share the rest."""
    H.ensure_built()
    n, bs = 5000, 16
    g = torch.Generator().manual_seed(d)
    key = (torch.randn((n, hk, d), generator=g) * 0.1)
    key[0] = 9.0 / math.sqrt(d)
    value = torch.randn((n, hk, d), generator=g) * spread
    q = (1 + 0.1 * torch.randn((1, hq, d), generator=g)).bfloat16().to(cuda_device)
    table, blocks = _table([n], bs, seed=d)
    cpu = _q4.empty_cache(blocks, hk, d, bs)
    _q4.store(cpu, key.bfloat16(), value.bfloat16(), _slots(table, bs, [(0, n)]))
    out, lse = _lib.paged_attention_q4(q, *[x.to(cuda_device) for x in cpu], _i32([0, 1], cuda_device),
                                       _i32([n], cuda_device), table.to(cuda_device), 1, n,
                                       num_splits=splits)
    parts = [x.to(cuda_device) for x in _q4.rows64(cpu, table[0], n)]
    _compare(out, lse, q, parts, n - 1)


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (8, 2, 128), (6, 2, 256), (32, 2, 128)])
@pytest.mark.parametrize("late", [0, 900])
def test_large_scales(cuda_device, hq, hk, d, late):
    """Values whose scales pass 16, from some key on: p * scale leaves what the lift allows."""
    H.ensure_built()
    n, bs = 1000, 32
    g = torch.Generator().manual_seed(d + late)
    key = torch.randn((n, hk, d), generator=g)
    value = torch.randn((n, hk, d), generator=g)
    value[late:] *= torch.tensor([20.0, 300.0, 5000.0, 10000.0])[torch.arange(n - late) % 4][:, None, None]
    q = torch.randn((3, hq, d), generator=g).bfloat16().to(cuda_device)
    table, blocks = _table([n], bs, seed=d)
    cpu = _q4.empty_cache(blocks, hk, d, bs)
    _q4.store(cpu, key.bfloat16(), value.bfloat16(), _slots(table, bs, [(0, n)]))
    assert all(torch.isfinite(x[table[0, :n // bs].long()]).all() for x in cpu[1::2])
    out, lse = _lib.paged_attention_q4(q, *[x.to(cuda_device) for x in cpu], _i32([0, 3], cuda_device),
                                       _i32([n], cuda_device), table.to(cuda_device), 3, n)
    parts = [x.to(cuda_device) for x in _q4.rows64(cpu, table[0], n)]
    _compare(out, lse, q, parts, n - 3, lift=25)


def test_a_group_with_a_nan_reads_back_as_nan(cuda_device):
    """... and no other group is touched by it."""
    H.ensure_built()
    hk, d, bs, n = 2, 128, 16, 40
    g = torch.Generator().manual_seed(5)
    key, value = (torch.randn((n, hk, d), generator=g).bfloat16() for _ in range(2))
    bad = [(0, 0, 0), (7, 1, 37), (20, 0, 95), (39, 1, 127)]  # token, head, channel
    table, blocks = _table([n], bs)
    slots = _slots(table, bs, [(0, n)])
    clean = _q4.empty_cache(blocks, hk, d, bs)
    _q4.store(clean, key, value, slots)
    for t, h, c in bad:
        key[t, h, c] = value[t, h, c] = float("nan")
    cache = [x.to(cuda_device) for x in _q4.empty_cache(blocks, hk, d, bs)]
    _lib.kv_store_q4(key.to(cuda_device), value.to(cuda_device), slots.to(cuda_device), *cache)
    rows = torch.zeros((2, n, hk, d), dtype=torch.bfloat16, device=cuda_device)
    _lib.kv_load_q4(rows[0], rows[1], _i32([0, n], cuda_device), table.to(cuda_device), *cache)
    kc, kz, vc, vz = _q4.rows64(clean, table[0], n)
    for got, want in ((rows[0].cpu(), (kc + kz).float().bfloat16()), (rows[1].cpu(), (vc + vz).float().bfloat16())):
        for t, h, c in bad:
            lo = c // 32 * 32
            assert torch.isnan(got[t, h, lo:lo + 32]).all()
            got[t, h, lo:lo + 32] = want[t, h, lo:lo + 32]
        assert torch.equal(got, want)


# ------------------------------------------------------------------- a server's round

@pytest.mark.parametrize("hq,hk,d,bs", [(8, 2, 64, 16), (32, 8, 128, 32), (28, 4, 128, 16), (6, 2, 256, 32)])
def test_prompts_chunks_and_decoding_together(cuda_device, hq, hk, d, bs):
    """Prompts attend to their own rows and are stored; their next chunks attend to the
    cached prefix, once read back as rows and once merged from two passes; then tokens
    are decoded one by one and a few at a time."""
    H.ensure_built()
    dev = cuda_device
    first, chunk, steps, draft = [37, 130, 5], [20, 64, 1], 2, 3
    total = [a + b + steps + draft for a, b in zip(first, chunk)]
    table, blocks = _table(total, bs, seed=d)
    cpu = _q4.empty_cache(blocks, hk, d, bs)
    cache = [x.to(dev) for x in cpu]
    tab = table.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    g = torch.Generator().manual_seed(d + hq)

    def fused(lens):
        rows = torch.randn((sum(lens), hq + 2 * hk, d), generator=g).bfloat16()
        return rows, rows.to(dev).split((hq, hk, hk), 1)

    def keep(rows, spans):
        slots = _slots(table, bs, spans)
        _, k, v = rows.to(dev).split((hq, hk, hk), 1)
        _lib.kv_store_q4(k, v, slots.to(dev), *cache, status=status)
        _q4.store(cpu, rows[:, hq:hq + hk], rows[:, hq + hk:], slots)

    def cached(s, n):
        return [x.to(dev) for x in _q4.rows64(cpu, table[s], n)]

    def plain(x):
        x = x.double()
        return x, torch.zeros_like(x)

    # the prompts
    rows, (q, k, v) = fused(first)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
    out, lse = _lib.prompt_attention(q, k, v, _starts(first, dev), max(first), workspace=ws)
    at = 0
    for n in first:
        span = slice(at, at + n)
        _compare(out[span], lse[span], q[span], plain(k[span]) + plain(v[span]), 0, p_bits=8)
        at += n
    keep(rows, [(0, n) for n in first])

    # the next chunk over the prefix's rows, read back in front of its own
    rows, (q, k, v) = fused(chunk)
    both = [a + b for a, b in zip(first, chunk)]
    cu_q, cu_k = _starts(chunk, dev), _starts(both, dev)
    wide = torch.full((2, sum(both), hk, d), float("nan"), dtype=torch.bfloat16, device=dev)
    _lib.kv_load_q4(wide[0], wide[1], cu_k, tab, *cache, load_lens=_i32(first, dev), status=status)
    at, ak = 0, 0
    for a, b in zip(first, chunk):
        wide[0, ak + a:ak + a + b], wide[1, ak + a:ak + a + b] = k[at:at + b], v[at:at + b]
        at, ak = at + b, ak + a + b
    out, lse = _lib.prompt_attention(q, wide[0], wide[1], cu_q, max(chunk), cu_seqlens_k=cu_k,
                                     max_key_len=max(both), workspace=ws)
    at, ak = 0, 0
    for s, (a, b) in enumerate(zip(first, chunk)):
        kc, kz, vc, vz = cached(s, a)
        assert torch.equal(wide[0, ak:ak + a], (kc + kz).float().bfloat16())
        assert torch.equal(wide[1, ak:ak + a], (vc + vz).float().bfloat16())
        _compare(out[at:at + b], lse[at:at + b], q[at:at + b],
                 plain(wide[0, ak:ak + a + b]) + plain(wide[1, ak:ak + a + b]), a, p_bits=8)
        at, ak = at + b, ak + a + b
    # and as two passes, merged.  The prefix's output is off as the 4-bit attention's, the
    # chunk's as the prompt's, each rounded to bf16, and their sum once more.
    o1, l1 = _lib.paged_attention_q4(q.contiguous(), *cache, cu_q, _i32(first, dev), tab, max(chunk), max(first),
                                     causal=False, workspace=ws)
    o2, l2 = _lib.prompt_attention(q, k, v, cu_q, max(chunk), workspace=ws)
    merged, lm = _lib.merge_attn_states(o1, l1, o2, l2)
    at = 0
    for s, (a, b) in enumerate(zip(first, chunk)):
        span = slice(at, at + b)
        parts = [torch.cat([x, y]) for x, y in zip(cached(s, a), plain(k[span]) + plain(v[span]))]
        ref, z, vc, vz, _, reach = _q4.attention64(q[span], parts, a)
        eps = max(2.0 ** -17, d * 2.0 ** -23) * reach + d ** -0.5 * 2.0 ** -21 * float(parts[0].abs().amax()) * d
        tol = (2.0 ** -8 * ref.abs() + (1.01 * (2.0 ** -7 + 2.0 ** -10 + 2.0 ** -11) + 4 * eps[..., None] + 2.0 ** -18)
               * (vc + vz) + a * 2.0 ** -35 * 25)
        assert ((merged.double()[span] - ref).abs() <= tol).all(), s
        assert ((lm.double()[span] - z).abs() <= 2 * eps + 2.0 ** -19 * (1 + z.abs())).all(), s
        at += b
    keep(rows, [(a, a + b) for a, b in zip(first, chunk)])

    # decoding: single tokens, then a few at once, each stored before it attends
    now = both
    for count in [1] * steps + [draft]:
        rows, (q, _, _) = fused([count] * 3)
        keep(rows, [(n, n + count) for n in now])
        now = [n + count for n in now]
        out, lse = _lib.paged_attention_q4(q.contiguous(), *cache, _starts([count] * 3, dev), _i32(now, dev), tab,
                                           count, max(now), workspace=ws)
        for s, n in enumerate(now):
            span = slice(s * count, (s + 1) * count)
            _compare(out[span], lse[span], q[span], cached(s, n), n - count)
    assert _lib.check_status(ws) == 0 and _lib.check_status(status) == 0


def _decode_inputs(device, lens, hq, hk, d, bs, seed):
    table, blocks = _table(lens, bs, seed=seed)
    g = torch.Generator().manual_seed(seed)
    cpu = _q4.empty_cache(blocks, hk, d, bs)
    n = sum(lens)
    _q4.store(cpu, torch.randn((n, hk, d), generator=g).bfloat16(), torch.randn((n, hk, d), generator=g).bfloat16(),
              _slots(table, bs, [(0, x) for x in lens]))
    q = torch.randn((len(lens), hq, d), generator=g).bfloat16().to(device)
    return q, [x.to(device) for x in cpu], cpu, table, _starts([1] * len(lens), device), _i32(lens, device)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_two_graphs_that_share_a_workspace(cuda_device, d):
    """A graph that stores a token, attends, reads back and attends to the rows; another of
    other sizes; replayed in turn with new tokens and lengths, against the calls made one by one."""
    H.ensure_built()
    dev, bs, hq, hk = cuda_device, 16, 8, 2
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device=dev)
    runs = []
    for lens in ([3000, 17, 800], [40, 2500]):
        q, cache, _, table, cu, sl = _decode_inputs(dev, [n + 8 for n in lens], hq, hk, d, bs, len(lens))
        sl.copy_(_i32(lens, dev))
        x = dict(q=q, cache=cache, table=table.to(dev), cu=cu, sl=sl, lens=list(lens), cpu_table=table,
                 kv=torch.zeros((2, len(lens), hk, d), dtype=torch.bfloat16, device=dev),
                 slots=torch.full((len(lens),), -1, dtype=torch.int64, device=dev), rows_cu=_starts(lens, dev),
                 rows=torch.zeros((2, sum(lens), hk, d), dtype=torch.bfloat16, device=dev),
                 out=torch.zeros_like(q), lse=torch.zeros(q.shape[:2], device=dev), out2=torch.zeros_like(q),
                 lse2=torch.zeros(q.shape[:2], device=dev))

        def step(x=x):
            _lib.kv_store_q4(x["kv"][0], x["kv"][1], x["slots"], *x["cache"])
            _lib.paged_attention_q4(x["q"], *x["cache"], x["cu"], x["sl"], x["table"], 1, 3008, out=x["out"],
                                    lse=x["lse"], workspace=ws)
            _lib.kv_load_q4(x["rows"][0], x["rows"][1], x["rows_cu"], x["table"], *x["cache"])
            _lib.prompt_attention(x["q"], x["rows"][0], x["rows"][1], x["cu"], 1, cu_seqlens_k=x["rows_cu"],
                                  max_key_len=3008, out=x["out2"], lse=x["lse2"], workspace=ws)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((x, step, graph))
    g = torch.Generator().manual_seed(1)
    names = ("out", "lse", "out2", "lse2", "rows")
    for turn in range(3):
        got = []
        for x, step, graph in runs:
            x["kv"].copy_(torch.randn(x["kv"].shape, generator=g).bfloat16())
            x["q"].copy_(torch.randn(x["q"].shape, generator=g).bfloat16())
            x["slots"].copy_(_slots(x["cpu_table"], bs, [(n + turn, n + turn + 1) for n in x["lens"]]))
            x["sl"].copy_(_i32([n + turn + 1 for n in x["lens"]], dev))
            graph.replay()
            got.append([x[n].clone() for n in names])
        torch.cuda.synchronize()
        for (x, step, graph), have in zip(runs, got):
            for n in names:
                x[n].fill_(-3.0)
            step()
            torch.cuda.synchronize()
            for n, h in zip(names, have):
                assert torch.equal(x[n], h), n
    assert _lib.check_status(ws) == 0


def test_streams_and_allocated_results(cuda_device):
    """On a stream of its own, as the current one and as an argument, with results and
    workspace allocated by the calls; equal calls give equal bits."""
    H.ensure_built()
    dev = cuda_device
    q, cache, cpu, table, cu, sl = _decode_inputs(dev, [900, 33, 4000], 8, 2, 128, 16, 3)
    tab = table.to(dev)
    want, wl = _lib.paged_attention_q4(q, *cache, cu, sl, tab, 1, 4000)
    for s, n in enumerate((900, 33, 4000)):
        _compare(want[s:s + 1], wl[s:s + 1], q[s:s + 1], [x.to(dev) for x in _q4.rows64(cpu, table[s], n)], n - 1)
    k, v = (torch.randn((600, 2, 128), device=dev).bfloat16() for _ in range(2))
    p = torch.randn((600, 8, 128), device=dev).bfloat16()
    pc = _i32([0, 100, 600], dev)
    pw, pl = _lib.prompt_attention(p, k, v, pc, 500)
    few, fl = _lib.prompt_attention(p[:20], k, v, _i32([0, 20], dev), 20, cu_seqlens_k=_i32([0, 600], dev),
                                    max_key_len=600)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for explicit in (False, True):
        for _ in range(3):
            with torch.cuda.stream(torch.cuda.current_stream() if explicit else side):
                stream = side if explicit else None
                a, al = _lib.paged_attention_q4(q, *cache, cu, sl, tab, 1, 4000, stream=stream)
                b, bl = _lib.prompt_attention(p, k, v, pc, 500, stream=stream)
                c, cl = _lib.prompt_attention(p[:20], k, v, _i32([0, 20], dev) if not explicit else pc_few, 20,
                                              cu_seqlens_k=_i32([0, 600], dev) if not explicit else kc_few,
                                              max_key_len=600, stream=stream)
                only = _lib.paged_attention_q4(q, *cache, cu, sl, tab, 1, 4000, stream=stream, return_lse=False)
            torch.cuda.synchronize()
            for x, y in ((a, want), (al, wl), (b, pw), (bl, pl), (c, few), (cl, fl), (only, want)):
                assert torch.equal(x, y)
        pc_few, kc_few = _i32([0, 20], dev), _i32([0, 600], dev)
        torch.cuda.synchronize()


# ------------------------------------------------------------------ tables and lengths

@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("q_len", [1, 5])
def test_keys_without_a_page_are_left_out(cuda_device, bs, splits, q_len):
    """A view of the table's first columns; an entry out of range in the middle."""
    H.ensure_built()
    dev, hq, hk, d, n = cuda_device, 8, 2, 128, 1000
    table, blocks = _table([n, n], bs, seed=bs)
    g = torch.Generator().manual_seed(bs)
    cpu = _q4.empty_cache(blocks, hk, d, bs)
    _q4.store(cpu, *(torch.randn((2 * n, hk, d), generator=g).bfloat16() for _ in range(2)),
              _slots(table, bs, [(0, n)] * 2))
    cache = [x.to(dev) for x in cpu]
    q = torch.randn((2 * q_len, hq, d), generator=g).bfloat16().to(dev)
    cu = _starts([q_len] * 2, dev)
    bad = table.clone()
    bad[0, 7], bad[1, 20] = blocks, -2
    columns = 30
    for tab, lens, gone in ((bad, [n, n], {0: 7, 1: 20}), (table, [n, 0x7fffffff], {})):
        view = tab.to(dev)[:, :columns] if not gone else tab.to(dev)
        ws = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
        out, lse = _lib.paged_attention_q4(q, *cache, cu, _i32(lens, dev), view, q_len, n, num_splits=splits,
                                           workspace=ws)
        with pytest.raises(_lib.PagedAttentionError) as e:
            _lib.check_status(ws)
        assert e.value.bits == _lib.DEV_BAD_BLOCK
        for s in range(2):
            limit = n if gone else min(n, columns * bs)
            keep = torch.ones(limit, dtype=torch.bool)
            if gone:
                keep[gone[s] * bs:(gone[s] + 1) * bs] = False
            parts = [x[keep.to(x.device)].to(dev) for x in _q4.rows64(cpu, table[s], limit)]
            for i in range(q_len):
                # of the keys with a page, those up to the query's own
                seen = int(keep[:n - q_len + i + 1].sum())
                row = slice(s * q_len + i, s * q_len + i + 1)
                _compare(out[row], lse[row], q[row], [x[:seen] for x in parts], seen - 1)


def test_lengths_that_are_flagged(cuda_device):
    H.ensure_built()
    dev = cuda_device
    q, cache, _, table, cu, sl = _decode_inputs(dev, [100, 50, 70], 8, 2, 64, 16, 9)
    q = q.repeat(2, 1, 1)
    tab = table.to(dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    cases = [([0, 3, 4, 5], [100, 50, 70], 1, _lib.DEV_BAD_SEQ, [0, 1, 2, 5]),  # longer than the call allows
             ([0, 1, 2, 3], [100, -1, 70], 1, _lib.DEV_BAD_SEQ, [1, 3, 4, 5]),
             ([0, 2, 4, 6], [1, 50, 70], 2, _lib.DEV_BAD_SEQ, [0, 1]),          # fewer keys than queries
             ([0, 2, 4, 9], [100, 50, 70], 5, _lib.DEV_BAD_SEQ, [4, 5])]        # past the rows
    for starts, lens, most, bits, untouched in cases:
        out = torch.full_like(q, 7.0)
        _lib.paged_attention_q4(q, *cache, _i32(starts, dev), _i32(lens, dev), tab, most, 100, out=out, workspace=ws)
        with pytest.raises(_lib.PagedAttentionError) as e:
            _lib.check_status(ws)
        assert e.value.bits == bits
        ws.zero_()
        kept = [i for i in range(6) if bool((out[i] == 7).all())]
        assert kept == untouched
    q[1, 3, 5] = 1e5
    _lib.paged_attention_q4(q[:3].contiguous(), *cache, cu, sl, tab, 1, 100, workspace=ws)
    with pytest.raises(_lib.PagedAttentionError) as e:
        _lib.check_status(ws)
    assert e.value.bits == _lib.DEV_BAD_Q


@pytest.mark.parametrize("splits", [1, 3])
def test_pages_before_a_window_are_not_needed(cuda_device, splits):
    H.ensure_built()
    dev = cuda_device
    q, cache, cpu, table, cu, sl = _decode_inputs(dev, [1000, 333], 8, 2, 128, 16, 4)
    tab = table.clone()
    tab[0, :(1000 - 70) // 16], tab[1, :(333 - 70) // 16] = 1 << 30, -1
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
    out, lse = _lib.paged_attention_q4(q, *cache, cu, sl, tab.to(dev), 1, 1000, sliding_window=70, workspace=ws,
                                       num_splits=splits)
    assert _lib.check_status(ws) == 0
    for s, n in enumerate((1000, 333)):
        _compare(out[s:s + 1], lse[s:s + 1], q[s:s + 1], [x.to(dev) for x in _q4.rows64(cpu, table[s], n)], n - 1,
                 window=70)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_that_leave_nothing_out(cuda_device, d):
    """The largest window, with queries in front of the first key among others."""
    H.ensure_built()
    dev, most = cuda_device, 0x7fffffff
    g = torch.Generator().manual_seed(d)
    q = torch.randn((300, 4, d), generator=g).bfloat16().to(dev)
    k, v = (torch.randn((520, 2, d), generator=g).bfloat16().to(dev) for _ in range(2))
    cu_q, cu_k = _i32([0, 10, 300], dev), _i32([0, 3, 520], dev)
    want = _lib.prompt_attention(q, k, v, cu_q, 290, cu_seqlens_k=cu_k, max_key_len=517)
    got = _lib.prompt_attention(q, k, v, cu_q, 290, cu_seqlens_k=cu_k, max_key_len=517, sliding_window=most)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0][:7] == 0).all() and torch.isinf(got[1][:7]).all() and torch.isfinite(got[1][7:]).all()
    q, cache, _, table, cu, sl = _decode_inputs(dev, [3000, 5], 4, 2, d, 16, 4)
    want = _lib.paged_attention_q4(q, *cache, cu, sl, table.to(dev), 1, 3000, num_splits=3)
    got = _lib.paged_attention_q4(q, *cache, cu, sl, table.to(dev), 1, 3000, num_splits=3, sliding_window=most)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits(cuda_device):
    """Pages behind the first 2^32 bytes of a cache, and rows 2^20 channels apart."""
    H.ensure_built()
    dev, hk, d, bs, n = cuda_device, 8, 128, 32, 130
    blocks = (1 << 32) // (hk * bs * (d // 2)) + 64
    pages = -(-n // bs)
    last = torch.arange(blocks - pages, blocks).flip(0).int()[None]
    cache = [torch.empty((blocks, hk, bs, d // 2), dtype=torch.uint8, device=dev),
             torch.empty((blocks, hk, 2, bs, d // 32), dtype=torch.float16, device=dev),
             torch.empty((blocks, hk, bs, d // 2), dtype=torch.uint8, device=dev),
             torch.empty((blocks, hk, 2, d // 32, bs), dtype=torch.float16, device=dev)]
    g = torch.Generator().manual_seed(2)
    key, value = (torch.randn((n, hk, d), generator=g).bfloat16() for _ in range(2))
    slots = _slots(last, bs, [(0, n)])
    _lib.kv_store_q4(key.to(dev), value.to(dev), slots.to(dev), *cache)
    cpu = _q4.empty_cache(pages, hk, d, bs)
    small = torch.arange(pages).flip(0).int()[None]
    _q4.store(cpu, key, value, _slots(small, bs, [(0, n)]))
    parts = [x.to(dev) for x in _q4.rows64(cpu, small[0], n)]
    q = torch.randn((1, 16, d), generator=g).bfloat16().to(dev)
    out, lse = _lib.paged_attention_q4(q, *cache, _i32([0, 1], dev), _i32([n], dev), last.to(dev), 1, n)
    _compare(out, lse, q, parts, n - 1)
    far = 2100  # rows in front: 2100 * 2^20 elements pass 2^31
    wide = torch.empty((far + n, 1 << 20), dtype=torch.bfloat16, device=dev)
    k = wide[:, :hk * d].view(-1, hk, d)
    v = wide[:, hk * d:2 * hk * d].view(-1, hk, d)
    cu_k = _i32([0, far, far + n], dev)
    _lib.kv_load_q4(k, v, cu_k, torch.cat([last, last]).to(dev), *cache, load_lens=_i32([0, n], dev))
    assert torch.equal(k[far:], (parts[0] + parts[1]).float().bfloat16())
    k[:far], v[:far] = 0, 0
    qs = torch.randn((far + n, 16 * d), generator=g).bfloat16().to(dev)
    wide[:, 4 * hk * d:4 * hk * d + 16 * d] = qs
    qw = wide[:, 4 * hk * d:4 * hk * d + 16 * d].view(-1, 16, d)
    out, lse = _lib.prompt_attention(qw, k, v, cu_k, far)
    zero = torch.zeros((n, hk, d), dtype=torch.float64, device=dev)
    _compare(out[far:], lse[far:], qw[far:], (k[far:].double(), zero, v[far:].double(), zero), 0, p_bits=8)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
def test_prompts_of_which_some_are_empty(cuda_device, hq, hk, d):
    """Sequences without queries, without keys, of one token, in any order; rows that none
    owns are left as they were."""
    H.ensure_built()
    dev = cuda_device
    q_lens, k_lens = [0, 5, 1, 0, 130, 1, 9, 0], [4, 0, 1, 0, 200, 300, 3, 0]
    g = torch.Generator().manual_seed(d)
    t, n = sum(q_lens) + 4, sum(k_lens) + 4
    q = torch.randn((t, hq, d), generator=g).bfloat16().to(dev)
    k, v = (torch.randn((n, hk, d), generator=g).bfloat16().to(dev) for _ in range(2))
    out = torch.full_like(q, 7.0)
    lse = torch.full((t, hq), 7.0, device=dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    _lib.prompt_attention(q, k, v, _starts(q_lens, dev), 130, cu_seqlens_k=_starts(k_lens, dev), max_key_len=300,
                          out=out, lse=lse, workspace=ws)
    assert _lib.check_status(ws) == 0
    at = ak = 0
    for a, b in zip(q_lens, k_lens):
        none = max(0, a - b)  # the first queries see no key
        assert (out[at:at + none] == 0).all() and (lse[at:at + none] == -math.inf).all()
        kk, vv = k[ak:ak + b].double(), v[ak:ak + b].double()
        span = slice(at + none, at + a)
        if a > none:
            _compare(out[span], lse[span], q[span], (kk, 0 * kk, vv, 0 * vv), b - (a - none), p_bits=8)
        at, ak = at + a, ak + b
    assert (out[at:] == 7).all() and (lse[at:] == 7).all()


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
@pytest.mark.parametrize("count", [2, 31, 32, 33, 70])
def test_many_prompts_of_uneven_lengths(cuda_device, hq, hk, d, count):
    H.ensure_built()
    dev = cuda_device
    g = torch.Generator().manual_seed(count + d)
    q_lens = torch.randint(0, 90, (count,), generator=g).tolist()
    k_lens = [a + int(b) for a, b in zip(q_lens, torch.randint(0, 300, (count,), generator=g))]
    t, n = sum(q_lens), sum(k_lens)
    q = torch.randn((t, hq, d), generator=g).bfloat16().to(dev)
    k, v = (torch.randn((n, hk, d), generator=g).bfloat16().to(dev) for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    out, lse = _lib.prompt_attention(q, k, v, _starts(q_lens, dev), 90, cu_seqlens_k=_starts(k_lens, dev),
                                     max_key_len=390, workspace=ws)
    assert _lib.check_status(ws) == 0
    at = ak = 0
    for a, b in zip(q_lens, k_lens):
        kk, vv = k[ak:ak + b].double(), v[ak:ak + b].double()
        if a:
            _compare(out[at:at + a], lse[at:at + a], q[at:at + a], (kk, 0 * kk, vv, 0 * vv), b - a, p_bits=8)
        at, ak = at + a, ak + b


@pytest.mark.parametrize("count,most,splits", [(3, 9, 64), (200, 40, 7), (40, 700, 3), (6, 5000, 0), (300, 100, 2)])
@pytest.mark.parametrize("d,bs,q_len", [(64, 16, 1), (128, 32, 1), (128, 16, 3), (256, 16, 1)])
def test_segments_of_all_sizes(cuda_device, count, most, splits, d, bs, q_len):
    """More segments than keys, more blocks than places, segments that hold nothing."""
    H.ensure_built()
    dev, hq, hk = cuda_device, 8, 2
    lens = torch.randint(q_len, most, (count,), generator=torch.Generator().manual_seed(count)).tolist()
    _, cache, cpu, table, _, sl = _decode_inputs(dev, lens, hq, hk, d, bs, count)
    g = torch.Generator().manual_seed(d)
    q = torch.randn((count * q_len, hq, d), generator=g).bfloat16().to(dev)
    out, lse = _lib.paged_attention_q4(q, *cache, _starts([q_len] * count, dev), sl, table.to(dev), q_len, most,
                                       num_splits=splits)
    for s in sorted({0, 1, 2, count // 2, count - 1}):
        span = slice(s * q_len, (s + 1) * q_len)
        _compare(out[span], lse[span], q[span], [x.to(dev) for x in _q4.rows64(cpu, table[s], lens[s])],
                 lens[s] - q_len)


# ------------------------------------------- long queries (D 128: another kernel above 64 rows)
# p and the values are rounded to fp16 there: 2^-11 each of p |v|

def _long(cpu, table, q, cu, lens, q_lens, out, lse, dev, causal=True, window=0, sinks=None, bits=10):
    at = 0
    for s, (n, a) in enumerate(zip(lens, q_lens)):
        if a:
            parts = [x.to(dev) for x in _q4.rows64(cpu, table[s], n)]
            span = slice(at, at + a)
            ref, z, vc, vz, va, reach = _q4.attention64(q[span], parts, n - a, causal, window, sinks)
            d = q.shape[-1]
            eps = 2.0 ** -16 * reach + d ** -0.5 * 2.0 ** -21 * (float(parts[0].abs().amax()) * d if n else 0.0)
            tol = (2.0 ** -8 * ref.abs() + (1.01 * 2.0 ** -bits + 2 * eps[..., None] + 2.0 ** -20) * (vc + vz)
                   + n * 2.0 ** -35 * (float((parts[2].abs() + parts[3].abs()).max()) if n else 0.0) + 1e-30)
            assert not torch.isnan(out[span]).any()
            err = (out[span].double() - ref).abs()
            assert (err <= tol).all(), (s, float((err - tol).max()), float(err.max()))
            none = torch.isinf(z)
            assert torch.equal(torch.isinf(lse[span]), none)
            e = torch.where(none, torch.zeros_like(z), (lse[span].double() - z).abs())
            assert (e <= eps + 2.0 ** -20 * (1 + torch.where(none, torch.zeros_like(z), z.abs()))).all()
        at += a


def _long_batch(lens, hk, bs, seed, value_scale=1.0):
    table, blocks = _table(lens, bs, seed=seed)
    g = torch.Generator().manual_seed(seed)
    cpu = _q4.empty_cache(blocks, hk, 128, bs)
    n = sum(lens)
    key = torch.randn((n, hk, 128), generator=g)
    value = torch.randn((n, hk, 128), generator=g) * value_scale
    _q4.store(cpu, key.bfloat16(), value.bfloat16(), _slots(table, bs, [(0, x) for x in lens]))
    return cpu, table


@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 2), (28, 4), (16, 1), (10, 2)])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("splits", [1, 3, 0, 64])
@pytest.mark.parametrize("window,causal", [(0, True), (1, True), (100, True), (0, False)])
def test_long_queries(cuda_device, hq, hk, bs, splits, window, causal):
    H.ensure_built()
    dev = cuda_device
    lens, q_lens = [130, 700, 66, 1025, 90, 0 if not causal else 3], [130, 33, 66, 70, 1, 3]
    cpu, table = _long_batch(lens, hk, bs, hq + bs)
    cache = [x.to(dev) for x in cpu]
    g = torch.Generator().manual_seed(hq)
    t = sum(q_lens)
    q = torch.randn((t + 2, hq, 128), generator=g).bfloat16().to(dev)
    sinks = (torch.randn(hq, generator=g) * 3).to(dev)
    sinks[0] = -math.inf
    cu = _starts(q_lens, dev)
    for sk in (None, sinks):
        out = torch.full_like(q, 7.0)
        lse = torch.full((t + 2, hq), 7.0, device=dev)
        ws = torch.zeros(_lib.paged_attention_q4_workspace_size(6, t + 2, hq, hk, 128, 130, 1025, splits),
                         dtype=torch.uint8, device=dev)
        ws[256:] = 0xFF
        _lib.paged_attention_q4(q, *cache, cu, _i32(lens, dev), table.to(dev), 130, 1025, out=out, lse=lse,
                                workspace=ws, num_splits=splits, sliding_window=window, causal=causal, sinks=sk)
        assert _lib.check_status(ws) == 0
        _long(cpu, table, q, cu, lens, q_lens, out, lse, dev, causal, window, sk)
        assert (out[t:] == 7).all() and (lse[t:] == 7).all()


@pytest.mark.parametrize("spread", [1e-3, 1.0, 3000.0])
def test_long_queries_over_small_and_large_values(cuda_device, spread):
    H.ensure_built()
    dev, hq, hk = cuda_device, 8, 2
    lens, q_lens = [3000, 200], [40, 100]
    cpu, table = _long_batch(lens, hk, 16, 3, spread)
    g = torch.Generator().manual_seed(4)
    q = (torch.randn((140, hq, 128), generator=g) * 2).bfloat16().to(dev)
    cu = _starts(q_lens, dev)
    out, lse = _lib.paged_attention_q4(q, *[x.to(dev) for x in cpu], cu, _i32(lens, dev), table.to(dev), 100, 3000)
    _long(cpu, table, q, cu, lens, q_lens, out, lse, dev)


def test_long_queries_without_some_pages(cuda_device):
    """Entries out of range, a table that ends early, pages before a window, q out of range."""
    H.ensure_built()
    dev, hq, hk, bs, n, a = cuda_device, 8, 2, 16, 900, 80
    cpu, table = _long_batch([n], hk, bs, 8)
    cache = [x.to(dev) for x in cpu]
    q = torch.randn((a, hq, 128), generator=torch.Generator().manual_seed(1)).bfloat16().to(dev)
    cu, sl = _i32([0, a], dev), _i32([n], dev)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=dev)
    bad = table.clone()
    bad[0, 9], bad[0, 20] = 1 << 30, -5
    keep = torch.ones(n, dtype=torch.bool)
    keep[9 * bs:10 * bs] = keep[20 * bs:21 * bs] = False
    for tab, k in ((bad.to(dev), keep), (table.to(dev)[:, :40], torch.arange(n) < 40 * bs)):
        out, lse = _lib.paged_attention_q4(q, *cache, cu, sl, tab, a, n, workspace=ws, causal=False)
        with pytest.raises(_lib.PagedAttentionError) as e:
            _lib.check_status(ws)
        assert e.value.bits == _lib.DEV_BAD_BLOCK
        ws.zero_()
        parts = [x[k].to(dev) for x in _q4.rows64(cpu, table[0], n)]
        _compare(out, lse, q, parts, 0, causal=False, p_bits=10)
    stale = table.clone()
    stale[0, :(n - a - 100) // bs] = -1
    out, lse = _lib.paged_attention_q4(q, *cache, cu, sl, stale.to(dev), a, n, workspace=ws, sliding_window=100)
    assert _lib.check_status(ws) == 0
    _long(cpu, table, q, cu, [n], [a], out, lse, dev, window=100)
    q[3, 1, 7] = 1e5
    _lib.paged_attention_q4(q, *cache, cu, sl, table.to(dev), a, n, workspace=ws)
    with pytest.raises(_lib.PagedAttentionError) as e:
        _lib.check_status(ws)
    assert e.value.bits == _lib.DEV_BAD_Q
    ws.zero_()
    _lib.paged_attention_q4(q, *cache, _i32([0, a + 1], dev), sl, table.to(dev), a + 1, n, workspace=ws)
    with pytest.raises(_lib.PagedAttentionError) as e:
        _lib.check_status(ws)
    assert e.value.bits == _lib.DEV_BAD_SEQ


def test_long_queries_captured(cuda_device):
    H.ensure_built()
    dev, hq, hk = cuda_device, 8, 2
    lens, q_lens = [2000, 300], [50, 90]
    cpu, table = _long_batch(lens, hk, 32, 12)
    cache, tab, cu, sl = [x.to(dev) for x in cpu], table.to(dev), _starts(q_lens, dev), _i32(lens, dev)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((140, hq, 128), generator=g).bfloat16().to(dev)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
    out, lse = torch.zeros_like(q), torch.zeros((140, hq), device=dev)

    def call():
        _lib.paged_attention_q4(q, *cache, cu, sl, tab, 90, 2000, out=out, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        q.copy_(torch.randn(q.shape, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        have = out.clone(), lse.clone()
        out.fill_(0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, have[0]) and torch.equal(lse, have[1])
        _long(cpu, table, q, cu, lens, q_lens, out, lse, dev)
