"""The 4-bit format for the tests: a quantizer and page packer of its own, dequantized
rows in 64 bits, and attention over rows in 64 bits with the bounds of a comparison."""
from __future__ import annotations

import math

import torch

K_ORDER, V_ORDER = 8, 4  # channels of a lane's run in a key row and in a value row


def nibble_of_channel(d, run):
    """Position of each channel's code in its row."""
    c = torch.arange(d)
    return ((c % 32 // run) * (d // 32) + c // 32) * run + c % run


def quantize(x):
    """Rows [..., D] (bf16) -> codes [..., D] (natural order), scales and zeros [..., G] fp16."""
    y = x.float().unflatten(-1, (-1, 32))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = torch.clamp((hi - lo) * torch.tensor(1 / 15), min=torch.tensor(1e-8))
    v = ((y - lo) / s).double()  # the fp32 quotient
    code = torch.floor(v + 0.5).clamp(0, 15).to(torch.uint8)  # v >= 0: half away is half up
    return code.flatten(-2), s.squeeze(-1).half(), lo.squeeze(-1).half()


def pack(codes, run):
    """Codes [..., D] in natural order -> bytes [..., D / 2] in the row's order."""
    d = codes.shape[-1]
    row = torch.empty_like(codes)
    row[..., nibble_of_channel(d, run).to(codes.device)] = codes
    return row[..., 0::2] | (row[..., 1::2] << 4)


def unpack(rows, run):
    """The inverse of pack."""
    nib = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)
    return nib[..., nibble_of_channel(nib.shape[-1], run).to(rows.device)]


def empty_cache(nb, hk, d, bs, device="cpu", fill=0xA5):
    g = d // 32
    codes = lambda: torch.full((nb, hk, bs, d // 2), fill, dtype=torch.uint8, device=device)  # noqa: E731
    scales = lambda *s: torch.full((nb, hk, 2, *s), float("nan"), dtype=torch.float16, device=device)  # noqa: E731
    return [codes(), scales(bs, g), codes(), scales(g, bs)]


def store(cache, key, value, slots):
    """kv_store_q4 on the CPU, row by row of the format's definition."""
    bs = cache[0].shape[2]
    real = slots >= 0
    block, off = slots[real] // bs, slots[real] % bs
    for i, (x, run) in enumerate(((key, K_ORDER), (value, V_ORDER))):
        code, s, z = quantize(x[real])
        cache[2 * i][block, :, off] = pack(code, run)
        sz = torch.stack([s, z], 2)  # [n, Hk, 2, G]
        if i == 0:
            cache[1][block, :, :, off] = sz
        else:
            cache[3][block, :, :, :, off] = sz


def rows64(cache, table_row, n):
    """(codes * scale, zero) of keys 0 .. n - 1, for K and for V: fp64 [n, Hk, D] each."""
    nb, hk, bs, half = cache[0].shape
    ids = table_row[:-(-n // bs)].long()
    out = []
    for i, run in ((0, K_ORDER), (2, V_ORDER)):
        code = unpack(cache[i][ids], run).double()
        sz = cache[i + 1][ids].double()
        if i == 2:
            sz = sz.transpose(-1, -2)
        sz = sz.repeat_interleave(32, -1)  # [p, Hk, 2, bs, D]
        for x in (code * sz[:, :, 0], sz[:, :, 1]):
            out.append(x.transpose(1, 2).reshape(-1, hk, 2 * half)[:n])
    return out


def attention64(q, parts, q_pos, causal=True, window=0, sinks=None, scale=None):
    """Attention of q [n, Hq, D] over rows given as parts (kc, kz, vc, vz) [L, Hk, D] (key =
    kc + kz, value = vc + vz), query i at position q_pos + i, in 64 bits.  Returns out, lse
    and, of the same shapes, sum p |vc|, sum p |vz|, sum p |v| and the largest
    |scale| * sum |q| (|kc| + |kz|) of a row's keys."""
    n, hq, d = q.shape
    kc, kz, vc, vz = parts
    length, hk = kc.shape[:2]
    scale = d ** -0.5 if scale is None else scale
    rep = hq // hk
    key = torch.arange(length, device=q.device)[None]
    pos = q_pos + torch.arange(n, device=q.device)[:, None]
    seen = torch.ones((n, length), dtype=torch.bool, device=q.device)
    if causal:
        seen = key <= pos
        if window:
            seen = seen & (key > pos - window)
    res = [torch.zeros((n, hq, d), dtype=torch.float64, device=q.device) for _ in range(4)]
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    reach = torch.zeros((n, hq), dtype=torch.float64, device=q.device)
    for h in range(hq):
        qh, g = q[:, h].double(), h // rep
        x = qh @ (kc[:, g] + kz[:, g]).T * scale
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        extra = torch.full((n, 1), -math.inf if sinks is None else float(sinks[h]),
                           dtype=torch.float64, device=q.device)
        z = torch.logsumexp(torch.cat([x, extra], 1), 1)
        p = torch.where(torch.isinf(z)[:, None], torch.zeros_like(x), torch.exp(x - z[:, None]))
        lse[:, h] = z
        a = qh.abs() @ (kc[:, g].abs() + kz[:, g].abs()).T * abs(scale)
        if length:
            reach[:, h] = torch.where(seen, a, torch.zeros_like(a)).amax(1)
        for r, v in zip(res, (vc[:, g] + vz[:, g], vc[:, g].abs(), vz[:, g].abs(),
                              (vc[:, g] + vz[:, g]).abs())):
            r[:, h] = p @ v
    return res[0], lse, res[1], res[2], res[3], reach
