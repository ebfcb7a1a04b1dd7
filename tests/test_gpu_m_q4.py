"""The 4-bit cache on the GPU: the store bit for bit, the read-back of all formats bit for
bit, and attention against 64 bits.

Bounds of the attention, per value.  A score's error: 32 exact products summed in fp32 by
the tensor core (each addition off by at most 2^-23 of the group's absolute sum: 2^-18),
the group sums and the zeros' part less again: under 2^-17 of scale * sum |q| (|c s| +
|z|); q / 16 in fp16 is off by at most 2^-25 below its normal range, 2^-21 of q.  The
output: half a bf16 step (2^-8 of the value), p and p * scale rounded to fp16 (2^-11
each: 2^-10 of sum p |c s|, 2^-11 of sum p |z|; below the normal range 2^-25 a key,
against a largest p of at least 1), the scores' errors (p off by that factor), ex2 2^-22."""
import math
import random

import pytest
import torch

from paged_attention_int8_gb300 import _lib, inputs
from tests import _harness as H
from tests import _q4

pytestmark = pytest.mark.gpu


def _table(pages, spare, seed):
    n = sum(pages) + spare
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(pages), max(1, max(pages)) + 1), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(pages):
        table[s, :c] = perm[at:at + c]
        at += c
    return table, n


def _rows(n, hk, d, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    bias = torch.randn((hk, d), generator=g) * math.sqrt(2)
    k = (torch.randn((n, hk, d), generator=g) * spread + bias).bfloat16()
    return k, torch.randn((n, hk, d), generator=g).bfloat16()


def _batch(device, lens, hk, d, bs, seed=0):
    """A filled cache on the device, its CPU copy, and the table."""
    H.ensure_built()
    table, blocks = _table([-(-n // bs) for n in lens], 3, seed)
    cache = _q4.empty_cache(blocks, hk, d, bs)
    key, value = _rows(sum(lens), hk, d, seed + 1)
    pos = torch.cat([torch.arange(n) for n in lens])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)])
    slots = table[seq, pos // bs].long() * bs + pos % bs
    _q4.store(cache, key, value, slots)
    return [t.to(device) for t in cache], cache, table


# ------------------------------------------------------------------------ store

@pytest.mark.parametrize("d,bs,hk", [(64, 16, 2), (64, 32, 1), (128, 16, 3), (128, 32, 8),
                                     (256, 16, 2), (256, 32, 1)])
@pytest.mark.parametrize("n", [1, 77])
def test_store_bit_for_bit(cuda_device, d, bs, hk, n):
    H.ensure_built()
    key, value = _rows(n, hk, d, 11 * d + n)
    # groups on which ties fall: multiples of the step's half, a constant, zeros, steps below 1e-8
    half = torch.arange(32).float() % 31 * 0.5
    key[0, 0, :32] = half.bfloat16()
    value[-1, -1, -32:] = (half * 0.0625 - 0.5).bfloat16()
    key[-1, 0, 32:64] = 3.0
    value[0, 0, :32] = 0.0
    value[0, 0, 32:64] = (torch.arange(32).float() * 1e-9).bfloat16()
    blocks = n // bs + 3
    slots = torch.randperm(blocks * bs, generator=torch.Generator().manual_seed(n))[:n]
    if n > 1:
        slots[5] = -1
    want = _q4.empty_cache(blocks, hk, d, bs)
    got = [t.to(cuda_device) for t in want]
    _q4.store(want, key, value, slots)
    # rows of a wider buffer
    wide = torch.zeros((n, 2 * hk + 1, d), dtype=torch.bfloat16, device=cuda_device)
    wide[:, :hk], wide[:, hk:2 * hk] = key.to(cuda_device), value.to(cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    _lib.kv_store_q4(wide[:, :hk], wide[:, hk:2 * hk], slots.to(cuda_device), *got, status=status)
    assert _lib.check_status(status) == 0
    for a, b in zip(got, want):
        a = a.cpu()
        assert torch.equal(a if a.dtype == torch.uint8 else a.view(torch.int16),
                           b if b.dtype == torch.uint8 else b.view(torch.int16))


def test_store_flags_slots_past_the_cache(cuda_device):
    H.ensure_built()
    cache = [t.to(cuda_device) for t in _q4.empty_cache(2, 1, 64, 16)]
    key, value = _rows(3, 1, 64, 5)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    slots = torch.tensor([32, 1 << 40, 3], device=cuda_device)
    _lib.kv_store_q4(key.to(cuda_device), value.to(cuda_device), slots, *cache, status=status)
    with pytest.raises(_lib.PagedAttentionError) as e:
        _lib.check_status(status)
    assert e.value.bits == _lib.DEV_BAD_SLOT
    want = _q4.empty_cache(2, 1, 64, 16)
    _q4.store(want, key, value, torch.tensor([-1, -1, 3]))
    assert torch.equal(cache[0].cpu(), want[0]) and torch.equal(cache[2].cpu(), want[2])


# -------------------------------------------------------------------- read-back

def _dequantized(fmt, cache, table_row, n):
    """Rows [n, Hk, D] of a cache in fp64 (exact), for K and V."""
    if fmt == "q4":
        kc, kz, vc, vz = _q4.rows64(cache, table_row, n)
        return kc + kz, vc + vz
    bs = cache[0].shape[2]
    ids = table_row[:-(-n // bs)].long()
    if fmt == "q8":
        k = cache[0][ids].double() * cache[1][ids].double().repeat_interleave(32, -1)
        v = cache[2][ids].double() * cache[3][ids].double().repeat_interleave(32, -2)
        v = v.transpose(-1, -2)
    else:
        k = cache[0][ids].view(torch.float8_e4m3fn).double()
        nib = torch.stack([cache[1][ids] & 15, cache[1][ids] >> 4], -1).flatten(-2).double()
        v = nib * cache[2][ids].double()[:, :, None] + cache[3][ids].double()[:, :, None]
        v = v.transpose(-1, -2)
    return [x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n] for x in (k, v)]


@pytest.mark.parametrize("fmt", ["q8", "f8v4", "q4"])
@pytest.mark.parametrize("d,bs,hk", [(64, 16, 3), (128, 32, 2), (256, 16, 1), (64, 32, 1), (128, 16, 8),
                                     (256, 32, 2)])
def test_load_bit_for_bit(cuda_device, fmt, d, bs, hk):
    H.ensure_built()
    lens = [0, 1, bs, 3 * bs + 5, 0, 2 * bs - 1]
    part = [0, 1, 0, 2 * bs + 3, 0, 2 * bs - 1]  # what the second call loads
    table, blocks = _table([-(-n // bs) for n in lens], 2, d)
    key, value = _rows(sum(lens), hk, d, d + bs)
    pos = torch.cat([torch.arange(n) for n in lens])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)])
    slots = (table[seq, pos // bs].long() * bs + pos % bs).to(cuda_device)
    if fmt == "q8":
        cache = inputs.empty_cache(blocks, hk, bs, d, device=cuda_device)
        store, load = _lib.kv_store, _lib.kv_load
    elif fmt == "q4":
        cache = [t.to(cuda_device) for t in _q4.empty_cache(blocks, hk, d, bs)]
        store, load = _lib.kv_store_q4, _lib.kv_load_q4
    else:
        u8, f16 = torch.uint8, torch.float16
        z = lambda dt, *s: torch.zeros((blocks, hk, *s), dtype=dt, device=cuda_device)  # noqa: E731
        cache = [z(u8, bs, d), z(u8, d, bs // 2), z(f16, bs), z(f16, bs)]
        store, load = _lib.kv_store_f8v4, _lib.kv_load_f8v4
    store(key.to(cuda_device), value.to(cuda_device), slots, *cache)
    cpu = [t.cpu() for t in cache]
    if fmt == "q8":
        cpu = [t.view(torch.float16) if t.dtype == torch.int16 else t for t in cpu]
    start = 2  # rows before the first sequence belong to none
    cu = [start]
    for n in lens:
        cu.append(cu[-1] + n)
    for wanted in (lens, part):
        buf = torch.full((cu[-1] + 3, 2 * hk, d), 7.0, dtype=torch.bfloat16, device=cuda_device)
        want = buf.cpu().clone()
        for s, n in enumerate(wanted):
            if n:
                k, v = _dequantized(fmt, cpu, table[s], n)
                want[cu[s]:cu[s] + n, :hk] = k.float().bfloat16()
                want[cu[s]:cu[s] + n, hk:] = v.float().bfloat16()
        status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        load(buf[:, :hk], buf[:, hk:], torch.tensor(cu, dtype=torch.int32, device=cuda_device),
             table.to(cuda_device)[:, :-1], *cache, status=status,
             load_lens=None if wanted is lens else torch.tensor(part, dtype=torch.int32, device=cuda_device))
        assert _lib.check_status(status) == 0
        assert torch.equal(buf.cpu().view(torch.int16), want.view(torch.int16))


def test_load_flags_what_it_leaves_out(cuda_device):
    lens = [20, 20, 20, 20]
    cache, cpu, table = _batch(cuda_device, lens, 2, 64, 16)
    table[1, 1] = 10 ** 6          # a page outside the cache: its rows stay
    cu = torch.tensor([0, 20, 40, 60, 500], dtype=torch.int32)  # the last sequence leaves the rows
    load = torch.tensor([20, 20, 21, 20], dtype=torch.int32)   # the third asks for too many
    out = torch.full((2, 100, 2, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    _lib.kv_load_q4(out[0], out[1], cu.to(cuda_device), table.to(cuda_device), *cache,
                    load_lens=load.to(cuda_device), status=status)
    with pytest.raises(_lib.PagedAttentionError) as e:
        _lib.check_status(status)
    assert e.value.bits == _lib.DEV_BAD_BLOCK | _lib.DEV_BAD_SEQ
    k, v = _dequantized("q4", cpu, table[0], 20)
    assert torch.equal(out[0, :20].cpu(), k.float().bfloat16())
    k, v = _dequantized("q4", cpu, table[1, :1], 16)
    assert torch.equal(out[1, 20:36].cpu(), v.float().bfloat16())
    assert (out[:, 36:] == 7).all()


# -------------------------------------------------------------------- attention

def check(q, cpu, table, lens, q_lens, out, lse, scale=None, causal=True, window=0, sinks=None):
    """out and lse of every sequence against 64 bits."""
    at = 0
    d = q.shape[-1]
    for s, (n, ql) in enumerate(zip(lens, q_lens)):
        parts = [x.to(q.device) for x in _q4.rows64(cpu, table[s], n)]
        ref, z, vc, vz, va, reach = _q4.attention64(q[at:at + ql], parts, n - ql, causal, window,
                                                    sinks, scale)
        eps = 2.0 ** -17 * reach + (d ** -0.5 if scale is None else abs(scale)) * 2.0 ** -21 * (
            parts[0].abs().amax() * d if n else 0.0)
        low = n * 2.0 ** -25 * (15 * 1.0 + (float(parts[3].abs().max()) if n else 0.0))
        tol = (2.0 ** -8 * ref.abs() + 1.01 * (2.0 ** -10 * vc + 2.0 ** -11 * vz)
               + (2 * eps[..., None] + 2.0 ** -20) * (vc + vz) + low)
        err = (out[at:at + ql].double() - ref).abs()
        assert not torch.isnan(out[at:at + ql]).any(), f"sequence {s}"
        assert (err <= tol).all(), (s, float((err - tol).max()), float(err.max()))
        got = lse[at:at + ql].double()
        empty = torch.isinf(z)
        assert torch.equal(torch.isinf(got), empty)
        e = torch.where(empty, torch.zeros_like(z), (got - z).abs())
        assert (e <= eps + 2.0 ** -21 * (1 + torch.where(empty, torch.zeros_like(z), z.abs()))).all(), s
        at += ql


def _run(device, hq, hk, d, bs, lens, q_lens, seed=0, pad=0, table_extra=0, **kw):
    cache, cpu, table = _batch(device, lens, hk, d, bs, seed)
    g = torch.Generator().manual_seed(seed + 7)
    t = sum(q_lens) + pad
    q = torch.randn((t, hq, d), generator=g).bfloat16().to(device)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    out = torch.full((t, hq, d), float("nan"), dtype=torch.bfloat16, device=device)
    lse = torch.full((t, hq), float("nan"), device=device)
    sinks = kw.pop("sinks", None)
    if sinks is not None:
        sinks = (torch.randn(hq, generator=g) * 3).to(device)
        sinks[0] = -math.inf
    ws = torch.full((_lib.paged_attention_q4_workspace_size(len(lens), t, hq, hk, d, max(q_lens), max(lens) or 1,
                                                                kw.get("num_splits", 0)),), 0xFF,
                    dtype=torch.uint8, device=device)
    ws[:4] = 0
    _lib.paged_attention_q4(q, *cache, torch.tensor(cu, dtype=torch.int32, device=device),
                            torch.tensor(lens, dtype=torch.int32, device=device), table.to(device),
                            max(q_lens), max(lens) or 1, sinks=sinks, out=out, lse=lse,
                            workspace=ws, **kw)
    assert _lib.check_status(ws) == 0
    check(q, cpu, table, lens, q_lens, out, lse, causal=kw.get("causal", True),
          window=kw.get("sliding_window", 0), sinks=sinks, scale=kw.get("softmax_scale"))
    assert torch.isnan(out[sum(q_lens):]).all() and torch.isnan(lse[sum(q_lens):]).all()


HEADS = [(4, 2, 64), (8, 1, 128), (28, 4, 128), (6, 2, 256), (16, 1, 64), (3, 3, 128), (32, 2, 256)]


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("splits", [1, 5, 0])
def test_single_tokens(cuda_device, hq, hk, d, bs, splits):
    _run(cuda_device, hq, hk, d, bs, [1, 15, 16, 17, 63, 64, 65, 129, 300, 1500], [1] * 10, seed=hq + d,
         num_splits=splits, pad=2)


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("splits", [1, 3])
def test_several_tokens(cuda_device, hq, hk, d, splits):
    _run(cuda_device, hq, hk, d, 16, [5, 40, 1, 200, 333, 90], [5, 3, 1, 17, 70, 0], seed=d,
         num_splits=splits, pad=3)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (32, 4, 128), (6, 2, 256)])
@pytest.mark.parametrize("q_lens", [[1] * 4, [3, 1, 9, 20]])
@pytest.mark.parametrize("window,sinks", [(0, True), (1, False), (16, True), (37, False), (10000, True)])
@pytest.mark.parametrize("splits", [1, 4])
def test_sinks_and_windows(cuda_device, hq, hk, d, q_lens, window, sinks, splits):
    _run(cuda_device, hq, hk, d, 32, [3, 64, 129, 700], q_lens, seed=window, sinks=sinks or None,
         sliding_window=window, num_splits=splits)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("q_lens", [[1] * 4, [3, 1, 9, 20]])
@pytest.mark.parametrize("sinks", [None, True])
def test_non_causal_and_empty(cuda_device, splits, q_lens, sinks):
    _run(cuda_device, 8, 2, 128, 16, [0, 2, 100, 0], q_lens, causal=False, num_splits=splits, sinks=sinks)


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.3])
def test_scales_and_sharp_rows(cuda_device, scale):
    _run(cuda_device, 8, 2, 64, 16, [300, 77], [1, 4], softmax_scale=scale, num_splits=2)
