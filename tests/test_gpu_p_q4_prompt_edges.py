"""The 4-bit cache and prompt_attention where their documentation makes a promise that larger
tests do not reach: keys that are no numbers, values past what fp16 holds next to their
weights, queries far from 1, sequences whose bounds fall, and which outputs a value that is no
number can reach."""
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


def _filled(lens, hk, d, bs, key, value):
    """A cache that holds rows key, value [sum(lens), Hk, D], on the CPU, and its table."""
    pages = [-(-n // bs) for n in lens]
    perm = torch.randperm(sum(pages) + 1, generator=torch.Generator().manual_seed(d)).int()
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(pages):
        table[s, :c] = perm[at:at + c]
        at += c
    pos = torch.cat([torch.arange(n) for n in lens])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)])
    cpu = _q4.empty_cache(sum(pages) + 1, hk, d, bs)
    _q4.store(cpu, key.bfloat16(), value.bfloat16(), table[seq, pos // bs].long() * bs + pos % bs)
    return cpu, table


def _flagged(status, bits):
    with pytest.raises(_lib.PagedAttentionError) as e:
        _lib.check_status(status)
    assert e.value.bits == bits


# --------------------------------------------------- keys and values that are no numbers

@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (8, 2, 128), (6, 2, 256)])
@pytest.mark.parametrize("count", [1, 3, 70])
@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("sink", [False, True])
def test_a_key_that_is_no_number(cuda_device, hq, hk, d, count, splits, sink):
    """Rows that see it have neither an output nor an lse, whatever the segments; the rows
    before it and the other sequences are what they are without it."""
    H.ensure_built()
    dev, lens, bad = cuda_device, [400, 350, 77], 400 - 1 - count // 2
    g = torch.Generator().manual_seed(d)
    key, value = (torch.randn((sum(lens), hk, d), generator=g) for _ in range(2))
    q = torch.randn((3 * count, hq, d), generator=g).bfloat16().to(dev)
    sinks = torch.randn(hq, generator=g).to(dev) if sink else None
    got = []
    for nan in (False, True):
        key[bad, 0, 5] = float("nan") if nan else 0.5
        cpu, table = _filled(lens, hk, d, 16, key, value)
        got.append(_lib.paged_attention_q4(q, *[x.to(dev) for x in cpu], _starts([count] * 3, dev), _i32(lens, dev),
                                           table.to(dev), count, 400, num_splits=splits, sinks=sinks))
    (want, want_lse), (out, lse) = got
    first = bad - (400 - count)  # query that sees it first
    heads = slice(0, hq // hk)   # of kv head 0
    assert torch.isnan(out[first:count, heads]).all() and torch.isnan(lse[first:count, heads]).all()
    assert torch.equal(lse[count:], want_lse[count:]) and torch.equal(out[count:], want[count:])
    assert torch.equal(lse[:, heads.stop:], want_lse[:, heads.stop:])
    assert torch.equal(out[:, heads.stop:], want[:, heads.stop:])
    # queries before it share a block with those that see it, and so where its maxima move: each of the
    # two results is within half a bf16 step and 2^-10 of sum p |c s| + 2^-11 of sum p |z| (under 9)
    a, b = out[:first, heads].float(), want[:first, heads].float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -9 * 9).all()
    assert ((lse[:first, heads] - want_lse[:first, heads]).abs() <= 2e-3).all()


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
@pytest.mark.parametrize("q_len,k_len", [(300, 300), (9, 3000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_key_of_a_prompt_that_is_no_number(cuda_device, hq, hk, d, q_len, k_len, bad):
    """As test_a_key_that_is_no_number; the second sizes go in segments.  (Infinite keys: the queries
    have both signs, so that their scores are inf - inf.)"""
    H.ensure_built()
    dev = cuda_device
    g = torch.Generator().manual_seed(d)
    q = torch.randn((q_len, hq, d), generator=g).bfloat16().to(dev)
    k, v = (torch.randn((k_len, hk, d), generator=g).bfloat16().to(dev) for _ in range(2))
    assert _lib.prompt_attention_workspace_size(1, q_len, k_len, hq, hk, d, q_len, k_len) > 256 or q_len == k_len

    def call(keys):
        return _lib.prompt_attention(q, keys, v, _i32([0, q_len], dev), q_len, cu_seqlens_k=_i32([0, k_len], dev),
                                     max_key_len=k_len)

    want, want_lse = call(k)
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
    at = k_len - 5
    k[at, 0] = bad
    out, lse = call(k)
    first, heads = q_len - 5, slice(0, hq // hk)
    assert torch.isnan(out[first:, heads]).all() and torch.isnan(lse[first:, heads]).all()
    assert torch.equal(out[:first], want[:first]) and torch.equal(lse[:first], want_lse[:first])
    assert torch.equal(out[:, heads.stop:], want[:, heads.stop:])
    assert torch.equal(lse[:, heads.stop:], want_lse[:, heads.stop:])


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
def test_scores_of_minus_infinity(cuda_device, hq, hk, d):
    """Weights that are all zero give 0 and -inf in one segment as in several."""
    H.ensure_built()
    dev = cuda_device
    q = torch.ones((5, hq, d), device=dev).bfloat16()
    k = torch.full((4000, hk, d), -float("inf"), device=dev).bfloat16()
    v = torch.randn((4000, hk, d), device=dev).bfloat16()
    need = _lib.prompt_attention_workspace_size(1, 5, 4000, hq, hk, d, 5, 4000)
    assert need > 256
    for size in (256, need):
        ws = torch.zeros(size, dtype=torch.uint8, device=dev)
        out, lse = _lib.prompt_attention(q, k, v, _i32([0, 5], dev), 5, cu_seqlens_k=_i32([0, 4000], dev),
                                         max_key_len=4000, workspace=ws)
        assert _lib.check_status(ws) == 0
        assert (out == 0).all() and (lse == -math.inf).all()


# ----------------------------------------------------------------- values and queries of all sizes

@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (8, 2, 128), (6, 2, 256), (32, 2, 128)])
@pytest.mark.parametrize("count", [1, 3])
@pytest.mark.parametrize("splits", [1, 3])
def test_the_largest_scales(cuda_device, hq, hk, d, count, splits):
    """Values up to 9e5 over zeros that fp16 holds: steps of up to 6e4, near its largest number.

    p and p * scale are rounded to fp16, 2^-11 each; p below its normal range to 2^-25 against a
    largest p of at least 1 / 4: 2^-23 a key of its largest value."""
    H.ensure_built()
    dev, n = cuda_device, 1000
    g = torch.Generator().manual_seed(d + count)
    key = torch.randn((n, hk, d), generator=g)
    value = torch.rand((n, hk, d), generator=g) * 9e5
    value[..., ::32] = 0  # a group's lowest
    q = (torch.randn((count, hq, d), generator=g) * 0.5).bfloat16().to(dev)
    cpu, table = _filled([n], hk, d, 16, key, value)
    held = [x[table[0].long()][:n // 16] for x in cpu[1::2]]
    assert all(torch.isfinite(x).all() for x in held) and float(held[1][:, :, 0].max()) > 5e4
    out, lse = _lib.paged_attention_q4(q, *[x.to(dev) for x in cpu], _i32([0, count], dev), _i32([n], dev),
                                       table.to(dev), count, n, num_splits=splits)
    parts = [x.to(dev) for x in _q4.rows64(cpu, table[0], n)]
    ref, z, vc, vz, _, reach = _q4.attention64(q, parts, n - count)
    eps = 2.0 ** -17 * reach
    tol = (2.0 ** -8 * ref.abs() + 1.01 * (2.0 ** -10 * vc + 2.0 ** -11 * vz)
           + (2 * eps[..., None] + 2.0 ** -20) * (vc + vz)
           + n * 2.0 ** -23 * float((parts[2].abs() + parts[3].abs()).max()))
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), float((err - tol).max())
    assert ((lse.double() - z).abs() <= eps + 2.0 ** -20 * (1 + z.abs())).all()


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (8, 2, 128), (6, 2, 256), (16, 1, 128)])
@pytest.mark.parametrize("count", [1, 3, 70])
@pytest.mark.parametrize("size", [1e-30, 1e-5, 1e-3, 1.0, 1e4])
def test_queries_of_all_sizes(cuda_device, hq, hk, d, count, size):
    """Queries whose size a softmax_scale takes back: no bit of theirs is lost.

    A score: exact products summed in fp32 (32 of a group on the tensor core, then the groups): under
    2^-16 of scale * sum |q| (|c s| + |z|).  The rest as in the other tests, p and the values
    in fp16 (2^-11 each)."""
    H.ensure_built()
    dev, lens = cuda_device, [300, 90]
    g = torch.Generator().manual_seed(d + count)
    key, value = (torch.randn((sum(lens), hk, d), generator=g) for _ in range(2))
    q = (torch.randn((2 * count, hq, d), generator=g) * size).bfloat16().to(dev)
    scale = d ** -0.5 / size
    cpu, table = _filled(lens, hk, d, 16, key, value)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
    out, lse = _lib.paged_attention_q4(q, *[x.to(dev) for x in cpu], _starts([count] * 2, dev), _i32(lens, dev),
                                       table.to(dev), count, 300, softmax_scale=scale, workspace=ws)
    assert _lib.check_status(ws) == 0
    for s, n in enumerate(lens):
        span = slice(s * count, (s + 1) * count)
        parts = [x.to(dev) for x in _q4.rows64(cpu, table[s], n)]
        ref, z, vc, vz, _, reach = _q4.attention64(q[span], parts, n - count, scale=scale)
        eps = 2.0 ** -16 * reach
        tol = (2.0 ** -8 * ref.abs() + (1.01 * 2.0 ** -10 + 2 * eps[..., None] + 2.0 ** -20) * (vc + vz)
               + n * 2.0 ** -35 * (15 + float((parts[2].abs() + parts[3].abs()).max())))
        err = (out[span].double() - ref).abs()
        assert (err <= tol).all(), (s, float((err - tol).max()), float(err.max()))
        assert ((lse[span].double() - z).abs() <= eps + 2.0 ** -20 * (1 + z.abs())).all(), s


# ---------------------------------------------------------------- bounds out of range

# starts of sequences over 40 rows: a falling one last, in the middle, beside many, and none within
BAD_STARTS = [[0, 40, 20], [0, 20, 10, 40], list(range(30)) + [25, 30, 31, 32, 33, 40],
              list(range(20)) + [10] + list(range(20, 40)), [100, 120], [-50, -20, 40]]


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256), (128, 1, 256)])
@pytest.mark.parametrize("starts", BAD_STARTS)
def test_prompt_bounds_that_are_flagged(cuda_device, hq, hk, d, starts):
    H.ensure_built()
    dev = cuda_device
    q = torch.randn((40, hq, d), device=dev).bfloat16()
    k = torch.randn((40, hk, d), device=dev).bfloat16()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
    cu = _i32(starts, dev)
    flat = _i32([0] * len(starts), dev)
    for cu_k in (cu, flat):
        _lib.prompt_attention(q, k, k, cu, 40, cu_seqlens_k=cu_k, max_key_len=40, workspace=ws)
        _flagged(ws, _lib.DEV_BAD_SEQ)
        assert _lib.check_status(ws) == 0


def test_a_bad_prompt_keeps_no_other_from_its_rows(cuda_device):
    """Tiles of one token: as many items as tokens, whatever the sequences that are left out."""
    H.ensure_built()
    dev = cuda_device
    q = torch.randn((4, 128, 256), device=dev).bfloat16()
    k = torch.randn((4, 1, 256), device=dev).bfloat16()
    for starts, own in (([0, 9, 2, 4], [2, 3]), ([0, 2, 4, 9], [0, 1, 2, 3]), ([-1, 0, 2, 4], [0, 1, 2, 3])):
        ws = torch.zeros(256, dtype=torch.uint8, device=dev)
        out = torch.full_like(q, 7.0)
        lse = torch.full((4, 128), 7.0, device=dev)
        _lib.prompt_attention(q, k, k, _i32(starts, dev), 9, cu_seqlens_k=_i32([0] * 4, dev), max_key_len=9, out=out,
                              lse=lse, workspace=ws)
        _flagged(ws, _lib.DEV_BAD_SEQ)
        for i in range(4):  # the queries see no key
            assert (out[i] == (0 if i in own else 7)).all() and (lse[i] == (-math.inf if i in own else 7)).all()


@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32), (256, 16)])
@pytest.mark.parametrize("starts", BAD_STARTS)
def test_read_back_bounds_that_are_flagged(cuda_device, d, bs, starts):
    H.ensure_built()
    dev, hk = cuda_device, 2
    cache = [x.to(dev) for x in _q4.empty_cache(3, hk, d, bs, fill=0)]
    rows = torch.full((2, 40, hk, d), 7.0, dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    table = torch.arange(3, dtype=torch.int32, device=dev).repeat(len(starts) - 1, 1)
    for lens in (None, _i32([0] * (len(starts) - 1), dev)):
        _lib.kv_load_q4(rows[0], rows[1], _i32(starts, dev), table, *cache, load_lens=lens, status=status)
        _flagged(status, _lib.DEV_BAD_SEQ)
    _lib.kv_load_q4(rows[0], rows[1], _i32([0, 3, 6], dev), table[:1].repeat(2, 1), *cache,
                    load_lens=_i32([0, 4], dev), status=status)
    _flagged(status, _lib.DEV_BAD_SEQ)


@pytest.mark.parametrize("hq,hk,d,most", [(4, 2, 64, 40), (16, 1, 64, 40), (8, 2, 128, 10), (8, 2, 128, 40),
                                          (6, 2, 256, 40), (16, 1, 256, 2)])
@pytest.mark.parametrize("starts", BAD_STARTS)
def test_cached_bounds_that_are_flagged(cuda_device, hq, hk, d, most, starts):
    H.ensure_built()
    dev = cuda_device
    cache = [x.to(dev) for x in _q4.empty_cache(4, hk, d, 16, fill=0)]
    for x in cache[1::2]:
        x.fill_(1.0)
    q = torch.randn((40, hq, d), device=dev).bfloat16()
    n = len(starts) - 1
    table = torch.arange(4, dtype=torch.int32, device=dev).repeat(n, 1)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=dev)
    for splits in (1, 3):
        _lib.paged_attention_q4(q, *cache, _i32(starts, dev), _i32([60] * n, dev), table, most, 60, workspace=ws,
                                num_splits=splits)
        _flagged(ws, _lib.DEV_BAD_SEQ)
    # a sequence without queries asks for nothing
    _lib.paged_attention_q4(q, *cache, _i32([0, 0, 2, 2], dev), _i32([-5, 60, 0], dev), table[:1].repeat(3, 1), most,
                            60, workspace=ws)
    assert _lib.check_status(ws) == 0


# ----------------------------------------------------------------- what reaches what

@pytest.mark.parametrize("hq,hk,d", [(2, 2, 64), (4, 1, 64), (3, 3, 128), (8, 2, 128), (16, 1, 128), (2, 2, 256),
                                     (6, 1, 256), (100, 1, 128)])
@pytest.mark.parametrize("window", [0, 70, 200])
@pytest.mark.parametrize("prefix", [0, 77])
def test_which_outputs_a_value_reaches(cuda_device, hq, hk, d, window, prefix):
    """A value row that holds no number reaches the queries that see its key, and of those that do
    not only queries of the same tile of 128 / (q heads a kv head) query tokens, up to 15
    keys in front of what its last query sees, and (with a window) of the same one or two
    tiles, back to the 128 keys in which the window of their first query begins."""
    H.ensure_built()
    dev, n = cuda_device, 600
    g = torch.Generator().manual_seed(d + hq)
    q = torch.randn((n, hq, d), generator=g).bfloat16().to(dev)
    k, v = (torch.randn((n + prefix, hk, d), generator=g).bfloat16().to(dev) for _ in range(2))
    cu_q, cu_k = _i32([0, n], dev), _i32([0, n + prefix], dev)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)  # one segment

    def call(values):
        r = _lib.prompt_attention(q, k, values, cu_q, n, cu_seqlens_k=cu_k, max_key_len=n + prefix,
                                  sliding_window=window, workspace=ws)
        assert _lib.check_status(ws) == 0
        return r

    want, want_lse = call(v)
    tile = 128 // (hq // hk)
    block = tile * (1 if d == 256 else 2)
    for j in (0, 130, 301, 447, n + prefix - 1):
        for bad in (float("nan"), float("inf")):
            values = v.clone()
            values[j] = bad
            out, lse = call(values)
            assert torch.equal(lse, want_lse)
            finite = torch.isfinite(out).flatten(1).any(1).tolist()
            same = (out == want).flatten(1).all(1).tolist()
            for i in range(n):
                at = prefix + i  # the last key of query i
                if j <= at and (not window or j > at - window):
                    assert not finite[i], (j, i)
                    continue
                end = prefix + min(i // tile * tile + tile, n)  # behind the last key of its tile
                first = max(0, prefix + i // block * block - window + 1) if window else 0
                if j >= -(-end // 16) * 16 or j < first // 128 * 128:
                    assert same[i], (j, i)


# ----------------------------------------------------------------- large groups

def _prompts(device, hq, hk, d, q_lens, k_lens, sinks=None, window=0, room=None):
    g = torch.Generator().manual_seed(hq + d)
    t, n = sum(q_lens), sum(k_lens)
    q = torch.randn((t, hq, d), generator=g).bfloat16().to(device)
    k, v = (torch.randn((n, hk, d), generator=g).bfloat16().to(device) for _ in range(2))
    most = max(q_lens), max(k_lens)
    size = _lib.prompt_attention_workspace_size(len(q_lens), t, n, hq, hk, d, *most)
    ws = torch.full((size if room is None else room,), 0xFF, dtype=torch.uint8, device=device)
    ws[:4] = 0
    out = torch.full_like(q, float("nan"))
    lse = torch.full((t, hq), float("nan"), device=device)
    _lib.prompt_attention(q, k, v, _starts(q_lens, device), most[0], cu_seqlens_k=_starts(k_lens, device),
                          max_key_len=most[1], sinks=sinks, sliding_window=window, out=out, lse=lse, workspace=ws)
    assert _lib.check_status(ws) == 0
    at = ak = 0
    for a, b in zip(q_lens, k_lens):
        # in 64 bits, all heads at once
        qq = q[at:at + a].double()
        kk, vv = (x[ak:ak + b].double().repeat_interleave(hq // hk, 1) for x in (k, v))
        key, pos = torch.arange(b, device=device)[None], b - a + torch.arange(a, device=device)[:, None]
        seen = (key <= pos) & (key > pos - (window or b + 1))
        x = torch.einsum("ihd,jhd->hij", qq, kk) * d ** -0.5
        reach = torch.einsum("ihd,jhd->hij", qq.abs(), kk.abs()).masked_fill(~seen, 0) * d ** -0.5
        reach = torch.cat([reach, reach.new_zeros((hq, a, 1))], 2).amax(2).T
        extra = x.new_full((hq, a, 1), -math.inf) if sinks is None else sinks.double().view(hq, 1, 1).expand(hq, a, 1)
        z = torch.logsumexp(torch.cat([x.masked_fill(~seen, -math.inf), extra], 2), 2).T
        p = torch.exp(x - z.T[..., None]).masked_fill(~seen, 0)
        ref, va = (torch.einsum("hij,jhd->ihd", p, y) for y in (vv, vv.abs()))
        eps = d * 2.0 ** -23 * reach  # D exact products summed in fp32
        tol = 2.0 ** -8 * ref.abs() + (1.01 * 2.0 ** -8 + 2 * eps[..., None] + 2.0 ** -20) * va + 1e-30
        assert ((out[at:at + a].double() - ref).abs() <= tol).all(), (a, b)
        empty = torch.isinf(z)
        assert torch.equal(torch.isinf(lse[at:at + a]), empty)
        e = torch.where(empty, torch.zeros_like(z), (lse[at:at + a].double() - z).abs())
        assert (e <= eps + 2.0 ** -20 * (1 + torch.where(empty, torch.zeros_like(z), z.abs()))).all(), (a, b)
        at, ak = at + a, ak + b
    return size


@pytest.mark.parametrize("hq,hk", [(32, 2), (65, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("count", [1, 5, 32, 33])
def test_prompts_of_large_groups(cuda_device, hq, hk, d, count):
    """Tiles of 8 tokens down to one, sequences in order of their keys and (33) in their own."""
    H.ensure_built()
    dev = cuda_device
    g = torch.Generator().manual_seed(count + hq)
    q_lens = [70] if count == 1 else torch.randint(0, 9, (count,), generator=g).tolist()
    k_lens = [90] if count == 1 else [max(0, a + int(b)) for a, b in zip(q_lens, torch.randint(-2, 200, (count,),
                                                                                              generator=g))]
    sinks = (torch.randn(hq, generator=g) * 2).to(dev)
    for kw in ({}, dict(sinks=sinks, window=40)):
        _prompts(dev, hq, hk, d, q_lens, k_lens, room=256, **kw)


@pytest.mark.parametrize("hq,hk", [(16, 1), (65, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_of_large_groups_in_segments(cuda_device, hq, hk, d):
    H.ensure_built()
    for q_lens, k_lens, window in (([3], [3000], 0), ([2, 0, 1], [2500, 7, 1300], 0), ([4, 1], [3001, 2], 700)):
        size = _prompts(cuda_device, hq, hk, d, q_lens, k_lens, window=window)
        assert size > 256 + sum(q_lens) * hq * (d + 2) * 4  # more than one segment
