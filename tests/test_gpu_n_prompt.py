"""prompt_attention on the GPU against 64 bits.

Bounds per value.  A score: D exact products summed in fp32 by the tensor core, each addition
off by at most 2^-23 of the sum of their sizes: D * 2^-23 of scale * sum |q| |k|.  The output:
half a bf16 step (2^-8 of the value), p rounded to bf16 (2^-8 of each term, sum p |v| in the
worst case), the scores' errors and ex2's 2^-22 on each p."""
import math

import pytest
import torch

from paged_attention_int8_gb300 import _lib
from tests import _harness as H
from tests import _q4

pytestmark = pytest.mark.gpu


def check(q, k, v, q_lens, k_lens, out, lse, causal=True, window=0, sinks=None, scale=None):
    at = ak = 0
    d = q.shape[-1]
    for s, (ql, kl) in enumerate(zip(q_lens, k_lens)):
        kk, vv = k[ak:ak + kl].double(), v[ak:ak + kl].double()
        zero = torch.zeros_like(kk)
        ref, z, va, _, _, reach = _q4.attention64(q[at:at + ql], (kk, zero, vv, zero), kl - ql, causal,
                                                  window, sinks, scale)
        eps = d * 2.0 ** -23 * reach
        tol = 2.0 ** -8 * ref.abs() + (1.01 * 2.0 ** -8 + 2 * eps[..., None] + 2.0 ** -20) * va + 1e-30
        got = out[at:at + ql].double()
        assert not torch.isnan(got).any(), f"sequence {s}"
        err = (got - ref).abs()
        assert (err <= tol).all(), (s, float((err - tol).max()), float(err.max()))
        empty = torch.isinf(z)
        g = lse[at:at + ql].double()
        assert torch.equal(torch.isinf(g), empty), s
        z0 = torch.where(empty, torch.zeros_like(z), z)
        e = torch.where(empty, torch.zeros_like(z), (g - z).abs())
        assert (e <= eps + 2.0 ** -20 * (1 + z0.abs())).all(), (s, float(e.max()))
        at, ak = at + ql, ak + kl


def run(device, hq, hk, d, q_lens, k_lens=None, seed=0, pad=0, fused=False, sinks=None, hint=None,
        spread=1.0, **kw):
    H.ensure_built()
    g = torch.Generator().manual_seed(seed)
    k_lens = q_lens if k_lens is None else k_lens
    t, n = sum(q_lens) + pad, sum(k_lens) + pad
    if fused:
        assert q_lens == k_lens
        rows = torch.randn((t, hq + 2 * hk, d), generator=g).bfloat16().to(device)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
    else:
        q, k, v = (torch.randn((m, h, d), generator=g).bfloat16().to(device)
                   for m, h in ((t, hq), (n, hk), (n, hk)))
        q = (q.float() * spread).bfloat16()
    cu = lambda lens: torch.tensor([0] + lens, device=device).cumsum(0).int()  # noqa: E731
    out = torch.full((t, hq, d), float("nan"), dtype=torch.bfloat16, device=device)
    lse = torch.full((t, hq), float("nan"), device=device)
    if sinks is not None:
        sinks = (torch.randn(hq, generator=g) * 3).to(device)
        sinks[0] = -math.inf
    hint = (max(q_lens), max(k_lens)) if hint is None else hint
    ws = torch.full((_lib.prompt_attention_workspace_size(len(q_lens), t, n, hq, hk, d, *hint),), 0xFF,
                    dtype=torch.uint8, device=device)
    ws[:4] = 0
    # rows that no sequence owns, and the rows behind each sequence's last, hold no number
    if pad:
        k[sum(k_lens):], v[sum(k_lens):] = float("nan"), float("nan")
    _lib.prompt_attention(q, k, v, cu(q_lens), hint[0], cu_seqlens_k=None if fused else cu(k_lens),
                          max_key_len=hint[1], sinks=sinks, out=out, lse=lse, workspace=ws, **kw)
    assert _lib.check_status(ws) == 0
    check(q, k, v, q_lens, k_lens, out, lse, causal=kw.get("causal", True),
          window=kw.get("sliding_window", 0), sinks=sinks, scale=kw.get("softmax_scale"))
    assert torch.isnan(out[sum(q_lens):]).all() and torch.isnan(lse[sum(q_lens):]).all()


HEADS = [(4, 2, 64), (16, 16, 64), (8, 2, 128), (7, 1, 128), (3, 3, 128), (6, 2, 256), (8, 1, 256)]


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_one_short_prompt(cuda_device, hq, hk, d):
    run(cuda_device, hq, hk, d, [40])


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("fused", [False, True])
def test_packed_prompts(cuda_device, hq, hk, d, fused):
    run(cuda_device, hq, hk, d, [1, 127, 128, 129, 0, 17, 400, 255, 64, 2], seed=d, pad=5, fused=fused)


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_long_prompt(cuda_device, hq, hk, d):
    run(cuda_device, hq, hk, d, [1501, 700], seed=d + 1)


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_chunks_behind_prefixes(cuda_device, hq, hk, d):
    # queries fewer than keys, none, more than keys (the first see none), no keys at all
    run(cuda_device, hq, hk, d, [100, 1, 0, 50, 30, 5, 130], [1100, 300, 64, 20, 0, 5, 131], seed=3, pad=2)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(0, True), (1, None), (100, True), (128, None), (100000, None)])
def test_sinks_and_windows(cuda_device, hq, hk, d, window, sinks):
    run(cuda_device, hq, hk, d, [300, 5, 140], [700, 5, 100], seed=window, sinks=sinks,
        sliding_window=window)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
@pytest.mark.parametrize("sinks", [None, True])
def test_non_causal(cuda_device, hq, hk, d, sinks):
    run(cuda_device, hq, hk, d, [130, 3, 40, 1], [300, 0, 17, 1], causal=False, sinks=sinks)


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("q_lens,k_lens", [([40], [5000]), ([1], [3001]), ([3, 70, 1], [9000, 2000, 40]),
                                           ([200], [200])])
def test_few_rows_over_many_keys(cuda_device, hq, hk, d, q_lens, k_lens):
    # key segments, joined; rows that some segments hold nothing for (the window, the sinks)
    for kw in ({}, dict(sinks=True), dict(sliding_window=700), dict(causal=False, sinks=True)):
        run(cuda_device, hq, hk, d, q_lens, k_lens, seed=d, pad=1, hint=(max(q_lens), 100000), **kw)


def test_a_small_workspace_takes_fewer_segments(cuda_device):
    H.ensure_built()
    q = torch.randn((20, 8, 128), device=cuda_device).bfloat16()
    k = torch.randn((8000, 2, 128), device=cuda_device).bfloat16()
    cu = torch.tensor([0, 20], dtype=torch.int32, device=cuda_device)
    cuk = torch.tensor([0, 8000], dtype=torch.int32, device=cuda_device)
    need = _lib.prompt_attention_workspace_size(1, 20, 8000, 8, 2, 128, 20, 8000)
    assert need > 256 + 20 * 8 * 8 * 130 * 4
    for size in (need, need // 2, 256 + 20 * 8 * 2 * 130 * 4, 256 + 20 * 8 * 2 * 130 * 4 - 4, 256):
        ws = torch.zeros(size, dtype=torch.uint8, device=cuda_device)
        out, lse = _lib.prompt_attention(q, k, k, cu, 20, cu_seqlens_k=cuk, max_key_len=8000, workspace=ws)
        assert _lib.check_status(ws) == 0
        check(q, k, k, [20], [8000], out, lse)


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.25])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
def test_scales_and_growing_scores(cuda_device, hq, hk, d, scale):
    # sharp rows: the maximum moves from tile to tile
    run(cuda_device, hq, hk, d, [900], softmax_scale=scale, spread=2.0)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 2, 128), (6, 2, 256)])
def test_no_keys_at_all(cuda_device, hq, hk, d):
    run(cuda_device, hq, hk, d, [5, 9], [0, 0], hint=(9, 0))


def test_other_sequences_stay_out(cuda_device):
    """Keys and values of the sequences around one hold infinities and no numbers."""
    H.ensure_built()
    for d in (64, 128, 256):
        g = torch.Generator().manual_seed(d)
        q, k, v = (torch.randn((400, 4, d), generator=g).bfloat16().to(cuda_device) for _ in range(3))
        cu = torch.tensor([0, 130, 263, 400], dtype=torch.int32, device=cuda_device)
        want, wl = _lib.prompt_attention(q, k, v, cu, 137)
        for bad in (float("nan"), float("inf"), -float("inf")):
            k2, v2 = k.clone(), v.clone()
            for x in (k2, v2):
                x[:130], x[263:] = bad, bad
            out, lse = _lib.prompt_attention(q, k2, v2, cu, 137)
            assert torch.equal(out[130:263], want[130:263]) and torch.equal(lse[130:263], wl[130:263])


def test_bad_bounds_are_flagged(cuda_device):
    H.ensure_built()
    q = torch.randn((64, 2, 64), device=cuda_device).bfloat16()
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    out = torch.full_like(q, 7.0)
    good = torch.tensor([0, 20, 64], dtype=torch.int32, device=cuda_device)
    for cu_q, cu_k in ((good, [0, 20, 65]), (good, [0, 70, 64]), ([0, 20, 80], good), ([-4, 20, 64], good)):
        cu_q, cu_k = (torch.as_tensor(x, dtype=torch.int32, device=cuda_device) for x in (cu_q, cu_k))
        _lib.prompt_attention(q, q, q, cu_q, 64, cu_seqlens_k=cu_k, max_key_len=64, out=out, workspace=ws)
        with pytest.raises(_lib.PagedAttentionError) as e:
            _lib.check_status(ws)
        assert e.value.bits == _lib.DEV_BAD_SEQ
