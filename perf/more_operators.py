"""Cases and plain forms of the operators around a 4-bit cache and a prompt.

A server that keeps its cache in 4 bits runs four operators that the 8-bit
path has no form of:

* ``kv_store_q4``: new K/V rows quantised to 4-bit codes as they are written
  into the paged cache, one scale and zero per (token, kv head, 32 channels);
* ``kv_load`` / ``kv_load_f8v4`` / ``kv_load_q4``: pages of a cache read back
  as packed bf16 rows (a cached prefix that a prompt's next chunk attends to, a
  cache that moves to another format);
* ``paged_attention_q4``: attention over the 4-bit cache, single tokens and
  several tokens a request;
* ``prompt_attention``: causal attention of packed prompts of different
  lengths over their own bf16 K/V rows, with or without a prefix before them.

Each case has a plain form in elementary torch operations (fp32, one rounding
at the end) and the call a user makes of the package (``own``).
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # three short prompts written, and read back as later steps will see them: latency
        dict(name="store_small", op="store", hk=2, d=64, bs=16, seqs=3, ctx=0, qlen=50, pad=0, lens=1),
        # chunks of prompts appended to cached prefixes, the token batch padded; the prefix and the
        # chunk come back as the rows that the chunk's attention takes
        dict(name="store_chunks", op="store", hk=8, d=128, bs=16, seqs=16, ctx=2048, qlen=2048,
             pad=333, lens=2),
        # the 8-bit prefixes of a few requests of uneven lengths
        dict(name="load_q8", op="load", fmt="q8", hk=8, d=128, bs=16, seqs=8, ctx=4096, lens=3),
        # long documents held in 4 bits
        dict(name="load_q4", op="load", fmt="q4", hk=8, d=128, bs=32, seqs=12, ctx=32768, lens=4),
        # two short requests decoding: latency
        dict(name="attn_tiny", op="attn", hq=4, hk=2, d=64, bs=16, seqs=2, ctx=100, qlen=1,
             sinks=False, window=0, lens=5),
        # a decode batch of requests of very different lengths
        dict(name="attn_decode", op="attn", hq=32, hk=8, d=128, bs=16, seqs=64, ctx=8192, qlen=1,
             sinks=False, window=0, lens=6),
        # a few requests deep into long documents, heads of 256 channels
        dict(name="attn_long", op="attn", hq=32, hk=8, d=256, bs=16, seqs=6, ctx=131072, qlen=1,
             sinks=False, window=0, lens=7),
        # up to five draft tokens a request verified together, with sinks
        dict(name="attn_verify", op="attn", hq=64, hk=8, d=128, bs=32, seqs=48, ctx=6001, qlen=5,
             sinks=True, window=0, lens=8),
        # three short prompts: latency
        dict(name="prompt_tiny", op="prompt", hq=4, hk=2, d=64, seqs=3, qlen=60, prefix=0, window=0,
             sinks=False, lens=9),
        # packed prompts of uneven lengths, sliced out of a fused projection
        dict(name="prompt_packed", op="prompt", hq=32, hk=8, d=128, seqs=8, qlen=4096, prefix=0,
             window=0, sinks=False, lens=10),
        # one long document
        dict(name="prompt_long", op="prompt", hq=32, hk=8, d=128, seqs=1, qlen=16384, prefix=0,
             window=0, sinks=False, lens=11),
        # chunks of prompts after their prefixes, heads of 256 channels
        dict(name="prompt_chunk_d256", op="prompt", hq=16, hk=4, d=256, seqs=4, qlen=1024,
             prefix=6000, window=0, sinks=False, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# q heads, kv heads, channels: the framework's layouts, one q head per kv head,
# odd and large group sizes
_HEADS = ((4, 2, 64), (32, 8, 128), (64, 8, 128), (32, 8, 256), (16, 16, 64), (28, 4, 128),
          (32, 2, 128), (6, 2, 256))


def draw(rng):
    op = rng.choice(("store", "load", "attn", "attn", "prompt", "prompt"))
    lens = rng.randrange(1 << 20)
    hq, hk, d = rng.choice(_HEADS)
    bs = rng.choice((16, 32))
    small = 128 // d if d <= 128 else 0.5  # heads of more channels: fewer rows
    small *= 8 / max(hk, 8)
    if op == "store":
        seqs = _log(rng, 1, 64)
        qlen = _log(rng, 1, max(2, int(24000 * small / seqs)))
        return dict(op=op, hk=hk, d=d, bs=bs, seqs=seqs, ctx=rng.choice((0, 0, _log(rng, 1, qlen + 1))),
                    qlen=qlen, pad=rng.choice((0, 0, 5, 77)), lens=lens)
    if op == "load":
        seqs = _log(rng, 1, 64)
        return dict(op=op, fmt=rng.choice(("q8", "f8v4", "q4", "q4")), hk=hk, d=d, bs=bs, seqs=seqs,
                    ctx=_log(rng, 1, int(160000 * small / seqs)), lens=lens)
    if op == "attn":
        qlen = rng.choice((1, 1, 1, 3, 8, 40, 300))
        seqs = _log(rng, 1, max(1, 128 // qlen))
        return dict(op=op, hq=hq, hk=hk, d=d, bs=bs, seqs=seqs, qlen=qlen,
                    ctx=max(qlen, _log(rng, 1, min(131072, int(300000 * small) // seqs) if qlen == 1 else 8192)),
                    sinks=rng.random() < 0.3, window=rng.choice((0, 0, 0, 1000)), lens=lens)
    seqs = _log(rng, 1, 24)
    qlen = _log(rng, 1, min(8192, 20000 // seqs))
    prefix = rng.choice((0, 0, _log(rng, 1, 8192)))
    return dict(op=op, hq=hq, hk=hk, d=d, seqs=seqs, qlen=qlen, prefix=min(prefix, 30000 // seqs),
                window=rng.choice((0, 0, 0, 777)), sinks=rng.random() < 0.3, lens=lens)


def _up(a, b):
    return -(-a // b)


def _lens(c):
    """Per sequence: keys held before the call, and new tokens.  The first
    sequence has the case's full lengths."""
    r = random.Random(c["lens"])
    n = c["seqs"]
    if c["op"] == "load":
        return [c["ctx"]] + [r.randint(0, c["ctx"]) for _ in range(n - 1)], [0] * n
    if c["op"] == "attn":
        q = [c["qlen"]] + [r.randint(1, c["qlen"]) for _ in range(n - 1)]
        total = [c["ctx"]] + [r.randint(max(q[i], c["ctx"] // 16), c["ctx"]) for i in range(1, n)]
        return [t - x for t, x in zip(total, q)], q
    before = c["ctx"] if c["op"] == "store" else c["prefix"]
    q = [c["qlen"]] + [r.randint(1, c["qlen"]) for _ in range(n - 1)]
    return [before] + [r.randint(0, before) for _ in range(n - 1)], q


def _pairs(c):
    """Query-key pairs that some head computes."""
    total = 0
    for p, q in zip(*_lens(c)):
        for lo, hi in ((p + 1, p + q),):  # query i sees p + 1 + i keys
            w = c["window"]
            if w:
                full = max(0, hi - max(lo, w) + 1)  # queries whose window is full
                part_hi = min(hi, w - 1)
                total += full * w
                if part_hi >= lo:
                    total += (lo + part_hi) * (part_hi - lo + 1) // 2
            else:
                total += (lo + hi) * (hi - lo + 1) // 2
    return total


def _row_bytes(fmt, d):
    """Bytes of one key and one value row of one kv head."""
    if fmt == "q8":
        return 2 * (d + d // 16)
    return d + d // 2 + 4 if fmt == "f8v4" else 2 * (d // 2 + d // 8)


def work(case):
    c = case
    held, new = _lens(c)
    rows = sum(held) + sum(new)
    if c["op"] in ("store", "load"):
        pages = sum(_up(a + b, c["bs"]) for a, b in zip(held, new))
        fmt = c.get("fmt", "q4")
        n = rows * c["hk"] * (_row_bytes(fmt, c["d"]) + 4 * c["d"]) + 4 * pages
        if c["op"] == "store":  # what the store itself reads and writes
            n += sum(new) * c["hk"] * (4 * c["d"] + _row_bytes(fmt, c["d"])) + 8 * (sum(new) + c["pad"])
        return dict(bytes=n, flops=0)
    t = sum(new)
    n = 4 * t * c["hq"] * c["d"] + 4 * t * c["hq"]
    keys = rows
    if c["window"]:  # keys that no query sees are not read
        keys = sum(min(a + b, b + c["window"] - 1) for a, b in zip(held, new))
    if c["op"] == "attn":
        n += keys * c["hk"] * _row_bytes("q4", c["d"]) + 4 * _up(keys, c["bs"])
    else:
        n += keys * c["hk"] * 4 * c["d"]
    return dict(bytes=n, flops=4 * c["d"] * c["hq"] * _pairs(c))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cumulative(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _half_away(v):
    """Rounding half away from zero of v >= 0."""
    r = torch.floor(v)
    return r + (v - r >= 0.5)


def _codes(x, top):
    """Codes 0 .. top, step and lowest value of rows x [..., n] in fp32."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / top).clamp_min(1e-8)
    return _half_away((x - lo) / s).clamp_(0, top).to(torch.uint8), s, lo


def _bytes_of(codes):
    """4-bit codes [..., n], two to a byte, the lower nibble first."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _quantize_q4(k, v):
    """fp32 pages [n, Hk, bs, D] to the 4-bit format: codes in the orders that the
    attention's lanes read, scales and zeros per 32 channels, token-major for
    keys and channel-major for values."""
    n, hk, bs, d = k.shape
    g = d // 32
    kc, ks, kz = _codes(k.unflatten(-1, (g, 32)), 15)
    vc, vs, vz = _codes(v.unflatten(-1, (g, 32)), 15)
    kc = _bytes_of(kc.view(n, hk, bs, g, 4, 8).transpose(3, 4).reshape(n, hk, bs, d))
    vc = _bytes_of(vc.view(n, hk, bs, g, 8, 4).transpose(3, 4).reshape(n, hk, bs, d))
    ks = torch.stack([ks, kz], 2).squeeze(-1).half()  # [n, Hk, 2, bs, G]
    vs = torch.stack([vs, vz], 2).squeeze(-1).half().transpose(-1, -2)  # [n, Hk, 2, G, bs]
    return kc, ks.contiguous(), vc, vs.contiguous()


def _quantize_q8(x):
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1, keepdim=True) / 127).clamp_min(1e-8)
    v = g / s
    return torch.copysign(_half_away(v.abs()), v).flatten(-2).to(torch.int8), s.squeeze(-1).half()


def _cache(fmt, hk, d, bs, blocks, g):
    """A cache of `blocks` pages of stored rows: keys N(0, 1) with a bias per
    channel, values N(0, 1), as bf16 rows quantised to the format."""
    bias = torch.randn((hk, 1, d), generator=g, device="cuda") * math.sqrt(2)
    parts = []
    for a in range(0, blocks, 4096):
        n = min(4096, blocks - a)
        k = torch.randn((n, hk, bs, d), generator=g, device="cuda").add_(bias).bfloat16().float()
        v = torch.randn((n, hk, bs, d), generator=g, device="cuda").bfloat16().float()
        if fmt == "q4":
            parts.append(_quantize_q4(k, v))
        elif fmt == "q8":
            kc, ks = _quantize_q8(k)
            vc, vs = _quantize_q8(v)
            parts.append((kc, ks, vc.transpose(-1, -2).contiguous(), vs.transpose(-1, -2).contiguous()))
        else:
            kc = k.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            vc, s, lo = _codes(v, 15)
            parts.append((kc, _bytes_of(vc.transpose(-1, -2)), s.squeeze(-1).half(),
                          lo.squeeze(-1).half()))
    return [torch.cat(p) for p in zip(*parts)]


def _table(pages, bs, g):
    """A block table for sequences of these page counts over a shuffled cache."""
    blocks = max(1, sum(pages))
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(pages), max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    return table.cuda(), blocks


def prepare(case, seed):
    c = case
    g = _gen(seed)
    held, new = _lens(c)
    total = [a + b for a, b in zip(held, new)]
    hk, d = c["hk"], c["d"]
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    if c["op"] == "prompt":
        t, n, hq = sum(new), sum(total), c["hq"]
        if c["prefix"]:
            q, k, v = randn(t, hq, d), randn(n, hk, d), randn(n, hk, d)
        else:  # slices of a fused projection's rows
            rows = randn(t, hq + 2 * hk, d)
            q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
        return dict(c=c, q=q, k=k, v=v, cu=_i32(_cumulative(new)), cuk=_i32(_cumulative(total)),
                    max_q=max(new), max_k=max(total),
                    sinks=torch.randn(hq, generator=g, device="cuda") * 2 if c["sinks"] else None,
                    out=torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty((t, hq), dtype=torch.float32, device="cuda"),
                    workspace=torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"))
    fmt = c.get("fmt", "q4")
    bs = c["bs"]
    table, blocks = _table([_up(x, bs) for x in total], bs, g)
    cache = _cache(fmt, hk, d, bs, blocks, g)
    rows = sum(total)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    if c["op"] == "attn":
        # the slots past a sequence's last key were never written: not a number
        length = torch.tensor(total, device="cuda")
        last = table[torch.arange(c["seqs"], device="cuda"), (length - 1) // bs].long()
        stale = torch.arange(bs, device="cuda")[None] > ((length - 1) % bs)[:, None]
        for i, m in ((1, stale.view(-1, 1, 1, bs, 1)), (3, stale.view(-1, 1, 1, 1, bs))):
            x = cache[i]
            x[last] = torch.where(m, torch.full_like(x[:1], float("nan")), x[last])
        t, hq = sum(new), c["hq"]
        return dict(c=c, cache=cache, table=table, cu=_i32(_cumulative(new)), lens=_i32(total),
                    max_q=max(new), max_k=max(total), q=randn(t, hq, d),
                    sinks=torch.randn(hq, generator=g, device="cuda") * 2 if c["sinks"] else None,
                    out=torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty((t, hq), dtype=torch.float32, device="cuda"),
                    workspace=torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"))
    state = dict(c=c, cache=cache, table=table, cuk=_i32(_cumulative(total)), status=status,
                 key=torch.empty((rows, hk, d), dtype=torch.bfloat16, device="cuda"),
                 value=torch.empty((rows, hk, d), dtype=torch.bfloat16, device="cuda"))
    if c["op"] == "store":
        t = sum(new)
        bias = torch.randn((1, hk, d), generator=g, device="cuda") * math.sqrt(2)
        pos = torch.cat([torch.arange(a, a + b) for a, b in zip(held, new)])
        seq = torch.cat([torch.full((b,), i) for i, b in enumerate(new)])
        slots = table.cpu()[seq, pos // bs].long() * bs + pos % bs
        slots = torch.cat([slots, slots.new_full((c["pad"],), -1)]).cuda()
        n = t + c["pad"]
        state.update(new_key=(torch.randn((n, hk, d), generator=g, device="cuda") + bias).bfloat16(),
                     new_value=randn(n, hk, d), slots=slots)
    return state


# ------------------------------------------------------------- plain forms

def _dequantized(c, cache, ids):
    """The fp32 K and V rows [pages * bs, Hk, D] of pages `ids`."""
    fmt, d, hk = c.get("fmt", "q4"), c["d"], c["hk"]
    n, g = ids.shape[0], d // 32
    a, b, e, f = (t[ids] for t in cache)
    bs = c["bs"]
    if fmt == "q4":
        k = _nibbles(a).view(n, hk, bs, 4, g, 8).transpose(3, 4).float()
        k = k * b[:, :, 0].float()[..., None, None] + b[:, :, 1].float()[..., None, None]
        v = _nibbles(e).view(n, hk, bs, 8, g, 4).transpose(3, 4).float()
        f = f.transpose(-1, -2).float()
        v = v * f[:, :, 0][..., None, None] + f[:, :, 1][..., None, None]
        k, v = k.reshape(n, hk, bs, d), v.reshape(n, hk, bs, d)
    elif fmt == "q8":
        k = a.float() * b.float().repeat_interleave(32, -1)
        v = (e.float() * f.float().repeat_interleave(32, -2)).transpose(-1, -2)
    else:
        k = a.view(torch.float8_e4m3fn).float()
        v = _nibbles(b).float() * e.float()[..., None, :] + f.float()[..., None, :]
        v = v.transpose(-1, -2)
    return (x.transpose(1, 2).reshape(n * bs, hk, d) for x in (k, v))


def _load(s):
    c = s["c"]
    held, new = _lens(c)
    at = 0
    for i, n in enumerate(a + b for a, b in zip(held, new)):
        for p0 in range(0, _up(n, c["bs"]), 1024):
            p1 = min(p0 + 1024, _up(n, c["bs"]))
            m = min(n, p1 * c["bs"]) - p0 * c["bs"]
            k, v = _dequantized(c, s["cache"], s["table"][i, p0:p1].long())
            s["key"][at:at + m] = k[:m]
            s["value"][at:at + m] = v[:m]
            at += m


def _store(s):
    c = s["c"]
    hk, d, bs = c["hk"], c["d"], c["bs"]
    slots = s["slots"]
    real = slots >= 0
    block, off = slots[real] // bs, slots[real] % bs
    rows = (s[x][real].float().view(-1, hk, 1, d) for x in ("new_key", "new_value"))
    kc, ks, vc, vs = _quantize_q4(*rows)
    s["cache"][0][block, :, off] = kc[:, :, 0]
    s["cache"][2][block, :, off] = vc[:, :, 0]
    s["cache"][1][block, :, :, off] = ks[:, :, :, 0]
    s["cache"][3][block, :, :, :, off] = vs[..., 0]


def _attend(q, k, v, limit, window, sinks, scale, out, lse):
    """Attention of q [n, Hq, D] over k, v [L, Hk, D] (fp32): query i sees keys up
    to limit + i, the last `window` of them.  Writes out [n, Hq, D], lse [n, Hq]."""
    n, hq, d = q.shape
    hk = k.shape[1]
    rep = hq // hk
    qh = q.view(n, hk, rep, d).permute(1, 2, 0, 3).reshape(hk, rep * n, d)
    x = torch.matmul(qh, k.permute(1, 2, 0)).mul_(scale).view(hk, rep, n, -1)
    key = torch.arange(k.shape[0], device=q.device)[None]
    last = limit + torch.arange(n, device=q.device)[:, None]
    hidden = key > last
    if window:
        hidden |= key <= last - window
    x.masked_fill_(hidden, float("-inf"))
    m = x.amax(-1, keepdim=True)
    if sinks is not None:
        m = torch.maximum(m, sinks.view(hk, rep, 1, 1))
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks.view(hk, rep, 1, 1) - m)
    o = torch.matmul(x.view(hk, rep * n, -1), v.transpose(0, 1)).view(hk, rep, n, d) / total
    out.copy_(o.permute(2, 0, 1, 3).reshape(n, hq, d))
    lse.copy_((m + torch.log(total)).squeeze(-1).permute(2, 0, 1).reshape(n, hq))


def _attn(s):
    c = s["c"]
    held, new = _lens(c)
    at = ak = 0
    for i, (p, n) in enumerate(zip(held, new)):
        if c["op"] == "prompt":
            k, v = (s[x][ak:ak + p + n].float() for x in ("k", "v"))
            ak += p + n
        else:
            k, v = _dequantized(c, s["cache"], s["table"][i, :_up(p + n, c["bs"])].long())
        step = max(1, (1 << 28) // (c["hq"] * (p + n)))
        for a in range(0, n, step):
            b = min(n, a + step)
            lo = max(0, p + a + 1 - c["window"]) if c["window"] else 0
            _attend(s["q"][at + a:at + b].float(), k[lo:p + b], v[lo:p + b], p + a - lo, c["window"],
                    s["sinks"], c["d"] ** -0.5, s["out"][at + a:at + b], s["lse"][at + a:at + b])
        at += n


def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if own:
        import paged_attention_int8_gb300 as pa
    if op in ("store", "load"):
        if own:
            if op == "store":
                pa.kv_store_q4(s["new_key"], s["new_value"], s["slots"], *s["cache"], status=s["status"])
            load = {"q8": pa.kv_load, "f8v4": pa.kv_load_f8v4, "q4": pa.kv_load_q4}[c.get("fmt", "q4")]
            load(s["key"], s["value"], s["cuk"], s["table"], *s["cache"], status=s["status"])
        else:
            if op == "store":
                _store(s)
            _load(s)
        return [s["key"], s["value"]]
    if not own:
        _attn(s)
    elif op == "attn":
        pa.paged_attention_q4(s["q"], *s["cache"], s["cu"], s["lens"], s["table"], s["max_q"],
                              s["max_k"], sinks=s["sinks"], sliding_window=c["window"], out=s["out"],
                              lse=s["lse"], workspace=s["workspace"])
    else:
        pa.prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["max_q"], cu_seqlens_k=s["cuk"],
                            max_key_len=s["max_k"], sinks=s["sinks"], sliding_window=c["window"],
                            out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------- exact

def _exact_rows(c, cache, table_row, n):
    """Keys 0 .. n - 1 of a sequence as fp64 rows [n, Hk, D], channel by channel."""
    d, hk, bs, fmt = c["d"], c["hk"], c["bs"], c.get("fmt", "q4")
    g = d // 32
    pages = table_row[:_up(n, bs)].long()
    ch = torch.arange(d, device="cuda")
    group, inner = ch // 32, ch % 32
    dense = lambda x: x.transpose(1, 2).reshape(-1, hk, d)[:n]  # noqa: E731
    if fmt == "q4":
        # the nibble of channel ch: keys in words of 8 channels, values in halves of 4
        kn = ((inner // 8) * g + group) * 8 + inner % 8
        vn = ((inner // 4) * g + group) * 4 + inner % 4

        def plane(codes, at, scale, zero):
            byte = codes[pages].to(torch.int32)[..., at // 2]
            nib = torch.where(at % 2 == 0, byte % 16, byte // 16).double()
            return dense(nib * scale.double()[..., group] + zero.double()[..., group])
        ks, vs = cache[1][pages], cache[3][pages].transpose(-1, -2)
        return plane(cache[0], kn, ks[:, :, 0], ks[:, :, 1]), plane(cache[2], vn, vs[:, :, 0], vs[:, :, 1])
    if fmt == "q8":
        k = cache[0][pages].double() * cache[1][pages].double()[..., group]
        v = cache[2][pages].double() * cache[3][pages].double()[:, :, group]
        return dense(k), dense(v.transpose(-1, -2))
    k = cache[0][pages].view(torch.float8_e4m3fn).double()
    key = torch.arange(bs, device="cuda")
    byte = cache[1][pages].to(torch.int32)[..., key // 2]
    v = torch.where(key % 2 == 0, byte % 16, byte // 16).double()
    v = v * cache[2][pages].double()[:, :, None] + cache[3][pages].double()[:, :, None]
    return dense(k), dense(v.transpose(-1, -2))


def _exact_q4(x, g):
    """Rows [n, Hk, D] through the 4-bit codes and back, fp64: the step and the code of
    the fp32 quotient, the scale and the zero rounded to fp16."""
    y = x.float().view(*x.shape[:-1], g, 32)
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    s = torch.maximum((hi - lo) / 15, torch.tensor(1e-8, device="cuda"))
    code = torch.floor(((y - lo) / s).double() + 0.5).clamp(0, 15)
    return (code * s.half().double() + lo.half().double()).flatten(-2)


def exact(case, seed):
    """In 64 bits, sequence by sequence and head by head."""
    c = case
    s = prepare(case, seed)
    held, new = _lens(c)
    d, hk = c["d"], c["hk"]
    if c["op"] in ("store", "load"):
        keys, values, at = [], [], 0
        for i, (p, n) in enumerate(zip(held, new)):
            k, v = _exact_rows(c, s["cache"], s["table"][i], p + n)
            if n:
                k = torch.cat([k[:p], _exact_q4(s["new_key"][at:at + n], d // 32)])
                v = torch.cat([v[:p], _exact_q4(s["new_value"][at:at + n], d // 32)])
            keys.append(k)
            values.append(v)
            at += n
        return [torch.cat(keys), torch.cat(values)]
    if 4 * d * c["hq"] * sum((p + n) * n for p, n in zip(held, new)) > 8e12:
        return None
    hq, rep = c["hq"], c["hq"] // hk
    outs, lses, at, ak = [], [], 0, 0
    for i, (p, n) in enumerate(zip(held, new)):
        if c["op"] == "prompt":
            k, v = s["k"][ak:ak + p + n], s["v"][ak:ak + p + n]
            ak += p + n
        else:
            k, v = _exact_rows(c, s["cache"], s["table"][i], p + n)
        out = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
        lse = torch.empty((n, hq), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 26) // (p + n))
        for h in range(hq):
            kh, vh = k[:, h // rep].double(), v[:, h // rep].double()
            for a in range(0, n, step):
                b = min(n, a + step)
                x = s["q"][at + a:at + b, h].double() @ kh.T / math.sqrt(d)
                behind = torch.arange(p + n, device="cuda")[None] - p - torch.arange(a, b, device="cuda")[:, None]
                x[behind > 0] = -math.inf
                if c["window"]:
                    x[behind <= -c["window"]] = -math.inf
                z = torch.logsumexp(x, -1)
                if s["sinks"] is not None:
                    z = torch.logaddexp(z, s["sinks"][h].double())
                lse[a:b, h] = z
                out[a:b, h] = torch.exp(x - z[:, None]) @ vh
        outs.append(out)
        lses.append(lse)
        at += n
    return [torch.cat(outs), torch.cat(lses)]
