"""Cases and plain forms of the shared-prefix serving operators.

A serving step over a batch whose requests share long prefixes runs three
operators beside the stores and the attention over the paged cache:

* ``build_block_tables``: from request lengths, the step's block table (pages
  of the persistent request table, new pages dealt from a free list, a private
  page where a request is about to write into a shared one), its slot map,
  positions and length arrays;
* ``copy_blocks``: the pages that the fork of a prefix made private, or that
  a defragmentation moves, copied inside the cache;
* ``paged_attention_shared_prefix``: attention of a batch whose groups of
  sequences share a prefix, the prefix computed once for all queries of its
  group, over either cache format.

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
        # a step of a few requests decoding together, their tables extended in place
        dict(name="tables_small", op="tables", seqs=8, rows=0, prefill=0, qlen=1, ctx=2048, bs=16,
             fork=False, pad=0, lens=1),
        # a decode step whose rows are gathered from a larger persistent request table
        dict(name="tables_decode", op="tables", seqs=256, rows=320, prefill=0, qlen=1, ctx=8192,
             bs=16, fork=False, pad=0, lens=2),
        # prefill chunks beside decodes, the token batch padded
        dict(name="tables_mixed", op="tables", seqs=132, rows=160, prefill=4, qlen=1024, ctx=16384,
             bs=32, fork=False, pad=90, lens=3),
        # a thousand samples forked off long shared prompts, each about to write its first token
        dict(name="tables_fork", op="tables", seqs=1024, rows=64, prefill=0, qlen=1, ctx=131072,
             bs=16, fork=True, pad=0, lens=4),
        # the partly filled pages of a 64-way fork made private (a padded pair list)
        dict(name="copy_fork", op="copy", fmt="q8", pairs=64, blocks=640, hk=8, d=128, bs=16,
             holes=0.2),
        # a defragmentation moving a large part of the cache
        dict(name="copy_move", op="copy", fmt="f8v4", pairs=8191, blocks=16411, hk=8, d=128, bs=16,
             holes=0.0),
        # four short samples of one prompt: latency
        dict(name="attn_tiny", op="attn", fmt="q8", hq=4, hk=2, d=64, bs=16, groups=1, seqs=4,
             prefix=100, suffix=37, qlen=1, sinks=False, lens=5),
        # a decode batch under one system prompt
        dict(name="attn_decode", op="attn", fmt="q8", hq=32, hk=8, d=128, bs=16, groups=1, seqs=64,
             prefix=8192, suffix=1024, qlen=1, sinks=False, lens=6),
        # several prompts of odd lengths, each with its own samples, with sinks
        dict(name="attn_groups", op="attn", fmt="q8", hq=64, hk=8, d=128, bs=32, groups=4, seqs=96,
             prefix=4095, suffix=511, qlen=1, sinks=True, lens=7),
        # a long document asked about by many requests
        dict(name="attn_long", op="attn", fmt="q8", hq=64, hk=8, d=128, bs=32, groups=1, seqs=128,
             prefix=32768, suffix=2048, qlen=1, sinks=False, lens=8),
        # heads of 256 channels
        dict(name="attn_d256", op="attn", fmt="q8", hq=32, hk=8, d=256, bs=16, groups=1, seqs=32,
             prefix=16384, suffix=512, qlen=1, sinks=False, lens=9),
        # up to five draft tokens a request verified together, fp8 keys and 4-bit values
        dict(name="attn_verify_f8v4", op="attn", fmt="f8v4", hq=32, hk=8, d=128, bs=16, groups=2,
             seqs=48, prefix=6001, suffix=700, qlen=5, sinks=False, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "copy", "attn", "attn", "attn"))
    lens = rng.randrange(1 << 20)
    if op == "tables":
        fork = rng.random() < 0.3
        seqs = _log(rng, 1, 1024)
        ctx = _log(rng, 16, 131072 if seqs <= 256 or fork else 16384)
        prefill = 0 if fork else min(seqs, rng.choice((0, 0, 1, 4)))
        return dict(op=op, seqs=seqs, rows=max(1, seqs // 16) if fork else seqs + rng.randrange(64),
                    prefill=prefill, qlen=_log(rng, 2, 2048) if prefill else rng.choice((1, 1, 4)),
                    ctx=ctx, bs=rng.choice((16, 32)), fork=fork, pad=rng.choice((0, 0, 7)),
                    lens=lens)
    if op == "copy":
        d = rng.choice((64, 128, 256))
        pairs = _log(rng, 1, 8191 * 128 // d // 2)
        return dict(op=op, fmt=rng.choice(("q8", "f8v4")), pairs=pairs,
                    blocks=2 * pairs + rng.randrange(1, 40), hk=rng.choice((2, 4, 8)), d=d,
                    bs=rng.choice((16, 32)) if pairs < 2000 else 16,
                    holes=rng.choice((0.0, 0.3)))
    # q heads, kv heads, channels: the framework's layouts, one q head per kv
    # head, odd and large group sizes
    hq, hk, d = rng.choice(((4, 2, 64), (32, 8, 128), (64, 8, 128), (32, 8, 256), (16, 16, 64),
                            (28, 4, 128), (32, 2, 128), (6, 2, 256)))
    qlen = rng.choice((1, 1, 1, 3, 8, 40))
    seqs = _log(rng, 1, max(1, 128 // qlen))
    groups = min(seqs, rng.choice((1, 1, 2, 5)))
    suffix = max(qlen, _log(rng, 1, 2048))
    return dict(op=op, fmt=rng.choice(("q8", "q8", "f8v4")), hq=hq, hk=hk, d=d,
                bs=rng.choice((16, 32)), groups=groups, seqs=seqs, prefix=_log(rng, 1, 32768),
                suffix=suffix, qlen=qlen, sinks=rng.random() < 0.3, lens=lens)


def _up(a, b):
    return -(-a // b)


def _table_lens(c):
    """Context, query and shared lengths and source rows of a table case."""
    r = random.Random(c["lens"])
    n = c["seqs"]
    if c["fork"]:
        # every sample continues one of the source rows, all of whose pages are shared
        row_ctx = [r.randint(c["ctx"] // 2, c["ctx"] - 1) | 1 for _ in range(c["rows"])]
        rows = [r.randrange(c["rows"]) for _ in range(n)]
        ctx = [row_ctx[i] for i in rows]
        return ctx, [1] * n, ctx, rows
    q = [c["qlen"] if i < c["prefill"] else (1 if c["prefill"] else r.randint(1, c["qlen"]))
         for i in range(n)]
    ctx = [r.randint(0, c["ctx"]) for _ in range(n)]
    rows = r.sample(range(c["rows"]), n) if c["rows"] else list(range(n))
    return ctx, q, None, rows


def _attn_lens(c):
    """Group starts, prefix lengths, and per sequence query and KV lengths."""
    r = random.Random(c["lens"])
    cuts = sorted(r.sample(range(1, c["seqs"]), c["groups"] - 1))
    starts = [0] + cuts + [c["seqs"]]
    prefix = [c["prefix"]] + [r.randint(max(1, c["prefix"] // 4), c["prefix"])
                              for _ in range(c["groups"] - 1)]
    q = [r.randint(1, c["qlen"]) for _ in range(c["seqs"])]
    lens = []
    for g in range(c["groups"]):
        for s in range(starts[g], starts[g + 1]):
            lens.append(prefix[g] + r.randint(q[s], c["suffix"]))
    return starts, prefix, q, lens


def _page_bytes(c):
    """Bytes of one page of one kv head: codes and scales of K and V."""
    if c["fmt"] == "q8":
        return 2 * c["bs"] * (c["d"] + c["d"] // 16)
    return c["bs"] * (c["d"] + c["d"] // 2 + 4)


def work(case):
    c = case
    if c["op"] == "tables":
        ctx, q, _, rows = _table_lens(c)
        pages = sum(_up(a + b, c["bs"]) for a, b in zip(ctx, q))
        new = sum(_up(a + b, c["bs"]) - _up(a, c["bs"]) for a, b in zip(ctx, q))
        # a table row is read and written only where rows move; in place, the new pages alone
        entries = (2 * pages if c["rows"] else 2 * new)
        return dict(bytes=4 * entries + 16 * (sum(q) + c["pad"]) + 28 * c["seqs"], flops=0)
    if c["op"] == "copy":
        n = c["pairs"] - int(c["pairs"] * c["holes"])
        return dict(bytes=2 * n * c["hk"] * _page_bytes(c) + 8 * c["pairs"], flops=0)
    starts, prefix, q, lens = _attn_lens(c)
    keys = sum(prefix)
    pairs = 0
    for g in range(c["groups"]):
        for s in range(starts[g], starts[g + 1]):
            keys += lens[s] - prefix[g]
            pairs += q[s] * lens[s] - q[s] * (q[s] - 1) // 2
    t = sum(q)
    return dict(bytes=keys * c["hk"] * _page_bytes(c) // c["bs"] + 4 * t * c["hq"] * c["d"]
                + 4 * t * c["hq"] + 4 * _up(keys, c["bs"]),
                flops=4 * c["d"] * c["hq"] * pairs)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cpu_gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _quantize_q8(x):
    """Rows [..., D] -> int8 codes and fp16 scales per 32 channels."""
    g = x.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1, keepdim=True) / 127).clamp_min(1e-8)
    v = g / s
    codes = torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)).clamp(-127, 127)
    return codes.flatten(-2).to(torch.int8), s.squeeze(-1).half()


def _cache(c, blocks, g):
    """A cache of `blocks` pages of stored rows: keys N(0, 1) with a bias per
    channel, values N(0, 1), as bf16 rows quantized to the case's format."""
    hk, d, bs = c["hk"], c["d"], c["bs"]
    bias = torch.randn((hk, 1, d), generator=g, device="cuda") * math.sqrt(2)
    parts = []
    for a in range(0, blocks, 4096):
        n = min(4096, blocks - a)
        k = torch.randn((n, hk, bs, d), generator=g, device="cuda").add_(bias).bfloat16().float()
        v = torch.randn((n, hk, bs, d), generator=g, device="cuda").bfloat16().float()
        if c["fmt"] == "q8":
            kc, ks = _quantize_q8(k)
            vc, vs = _quantize_q8(v)
            parts.append((kc, ks, vc.transpose(-1, -2).contiguous(),
                          vs.transpose(-1, -2).contiguous()))
        else:
            kc = k.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
            s = ((hi - lo) / 15).clamp_min(1e-8)
            idx = torch.floor((v - lo) / s + 0.5).clamp(0, 15).to(torch.uint8)
            idx = idx.transpose(-1, -2)
            parts.append((kc, (idx[..., 0::2] | (idx[..., 1::2] << 4)).contiguous(),
                          s.squeeze(-1).half(), lo.squeeze(-1).half()))
    return [torch.cat(p) for p in zip(*parts)]


def prepare(case, seed):
    c = case
    g = _gen(seed)
    if c["op"] == "tables":
        ctx, q, shared, rows = _table_lens(c)
        n_rows = c["rows"] or c["seqs"]
        # the persistent table holds each request's pages at its row
        ctx_of = [0] * n_rows
        for s, row in enumerate(rows):
            ctx_of[row] = ctx[s]
        held = [_up(x, c["bs"]) for x in ctx_of]
        stride = max(_up(a + b, c["bs"]) for a, b in zip(ctx, q)) + 3
        need = sum(_up(b, c["bs"]) + 2 for b in q)
        blocks = sum(held) + need
        perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        have = torch.tensor(held, device="cuda")
        source = torch.full((n_rows, stride), -1, dtype=torch.int32, device="cuda")
        used = torch.arange(stride, device="cuda")[None] < have[:, None]
        source[used] = perm[: sum(held)]
        free = torch.cat([perm.new_full((5,), -1), perm[sum(held):]])  # five entries already dealt
        tokens = sum(q) + c["pad"]
        return dict(c=c, ctx=_i32(ctx), q=_i32(q), shared=None if shared is None else _i32(shared),
                    rows=_i32(rows) if c["rows"] else None, source=source, free=free,
                    head=_i32([5]), blocks=blocks, tokens=tokens,
                    table=torch.full((c["seqs"], stride), -1, dtype=torch.int32, device="cuda")
                    if c["rows"] else source,
                    cu=_i32([0] * (c["seqs"] + 1)), lens=_i32([0] * c["seqs"]),
                    slots=torch.zeros(tokens, dtype=torch.int64, device="cuda"),
                    pos=torch.zeros(tokens, dtype=torch.int64, device="cuda"),
                    pairs=_i32([[0, 0]] * c["seqs"]), next=_i32([0]),
                    status=_i32([0, 0, 0, 0]))
    if c["op"] == "copy":
        cache = _cache(c, c["blocks"], g)
        perm = torch.randperm(c["blocks"], generator=g, device="cuda").to(torch.int32)
        pairs = torch.stack([perm[: c["pairs"]], perm[c["pairs"]: 2 * c["pairs"]]], 1).contiguous()
        holes = torch.randperm(c["pairs"], generator=g, device="cuda")[: int(c["pairs"] * c["holes"])]
        pairs[holes] = -1
        return dict(c=c, cache=cache, pairs=pairs, status=_i32([0, 0, 0, 0]))
    starts, prefix, q, lens = _attn_lens(c)
    bs = c["bs"]
    shared = [p // bs for p in prefix]  # whole pages that a group's rows share
    pages = [_up(x, bs) for x in lens]
    group = [g_ for g_ in range(c["groups"]) for _ in range(starts[g_], starts[g_ + 1])]
    blocks = sum(shared) + sum(n - shared[group[s]] for s, n in enumerate(pages))
    cache = _cache(c, blocks, g)
    perm = torch.randperm(blocks, generator=_cpu_gen(seed)).to(torch.int32)
    table = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32)
    at = 0
    for g_ in range(c["groups"]):
        table[starts[g_]:starts[g_ + 1], :shared[g_]] = perm[at:at + shared[g_]]
        at += shared[g_]
    for s, n in enumerate(pages):
        n0 = shared[group[s]]
        table[s, n0:n] = perm[at:at + n - n0]
        at += n - n0
    table = table.cuda()
    # the slots past a sequence's last key were never written: not a number
    length = torch.tensor(lens, device="cuda")
    last = table[torch.arange(c["seqs"], device="cuda"), (length - 1) // bs].long()
    stale = torch.arange(bs, device="cuda")[None] > ((length - 1) % bs)[:, None]  # [S, bs]
    for i in ((1, 3) if c["fmt"] == "q8" else (2, 3)):
        t = cache[i]
        m = stale.view(-1, 1, bs, 1) if c["fmt"] == "q8" and i == 1 else (
            stale.view(-1, 1, 1, bs) if c["fmt"] == "q8" else stale.view(-1, 1, bs))
        t[last] = torch.where(m, torch.full_like(t[:1], float("nan")), t[last])
    tokens = sum(q)
    cu = [0]
    for x in q:
        cu.append(cu[-1] + x)
    hq, d = c["hq"], c["d"]
    return dict(c=c, cache=cache, table=table, cu=_i32(cu), lens=_i32(lens), starts=_i32(starts),
                prefix=_i32(prefix),
                q=torch.randn((tokens, hq, d), generator=g, device="cuda").bfloat16(),
                sinks=torch.randn(hq, generator=g, device="cuda") * 2 if c["sinks"] else None,
                max_group=max(cu[starts[i + 1]] - cu[starts[i]] for i in range(c["groups"])),
                max_suffix=max(lens[s] - prefix[group[s]] for s in range(c["seqs"])),
                max_q=max(q), max_prefix=max(prefix),
                out=torch.empty((tokens, hq, d), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((tokens, hq), dtype=torch.float32, device="cuda"),
                workspace=torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------- plain forms

def _tables(s):
    c = s["c"]
    bs, n = c["bs"], c["seqs"]
    ctx, q = s["ctx"].long(), s["q"].long()
    lens = ctx + q
    cu = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(q, 0)
    held = (ctx + bs - 1) // bs
    end = (lens + bs - 1) // bs
    if s["shared"] is None:
        private = torch.zeros_like(ctx, dtype=torch.bool)
    else:
        private = (q > 0) & (ctx % bs != 0) & (s["shared"].long() > ctx // bs * bs)
    first = torch.where(private, ctx // bs, held)
    count = torch.where(q > 0, end - first, torch.zeros_like(end))
    before = torch.cumsum(count, 0) - count + s["head"].long()
    old = (s["source"] if s["rows"] is None else s["source"][s["rows"].long()]).long()
    page = torch.arange(old.shape[1], device="cuda")[None]
    fresh = s["free"].long()[(before[:, None] + page - first[:, None]).clamp(0, s["free"].numel() - 1)]
    pages = torch.where(page < first[:, None], old, fresh)
    table = torch.where(page < end[:, None], pages, s["table"].long())
    at = (ctx // bs)[:, None].clamp_max(old.shape[1] - 1)
    pair = torch.cat([old.gather(1, at), table.gather(1, at)], 1)
    s["pairs"].copy_(torch.where(private[:, None], pair, torch.full_like(pair, -1)))
    s["table"].copy_(table)
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True).clamp_max(n - 1)
    real = t < cu[n]
    pos = torch.where(real, ctx[seq] + t - cu[seq], torch.zeros_like(t))
    slot = table[seq, pos // bs] * bs + pos % bs
    s["slots"].copy_(torch.where(real, slot, torch.full_like(slot, -1)))
    s["pos"].copy_(pos)
    s["cu"].copy_(cu)
    s["lens"].copy_(lens)
    s["next"].copy_(s["head"] + count.sum())


def _copy(s):
    pairs = s["pairs"].long()
    pairs = pairs[(pairs[:, 0] >= 0) & (pairs[:, 1] >= 0)]
    s["cache"][0][pairs[:, 1]] = s["cache"][0][pairs[:, 0]]
    s["cache"][1][pairs[:, 1]] = s["cache"][1][pairs[:, 0]]
    s["cache"][2][pairs[:, 1]] = s["cache"][2][pairs[:, 0]]
    s["cache"][3][pairs[:, 1]] = s["cache"][3][pairs[:, 0]]


def _rows(c, cache, blocks):
    """The fp32 K and V rows [N, Hk, pages * bs, D] of pages `blocks` [N, pages]."""
    n, p = blocks.shape
    if c["fmt"] == "q8":
        kc, ks, vc, vs = cache
        k = kc[blocks].float() * ks[blocks].float().repeat_interleave(32, -1)
        v = vc[blocks].float() * vs[blocks].float().repeat_interleave(32, -2)
    else:
        kc, vc, vs, vz = cache
        k = kc[blocks].view(torch.float8_e4m3fn).float()
        codes = vc[blocks]
        v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        v = v * vs[blocks].float()[..., None, :] + vz[blocks].float()[..., None, :]
    k = k.transpose(1, 2).reshape(n, c["hk"], p * c["bs"], c["d"])
    v = v.permute(0, 2, 1, 4, 3).reshape(n, c["hk"], p * c["bs"], c["d"])
    return k, v


def _part(c, q, k, v, seen):
    """Attention of q [N, R, Hq, D] over k, v [N, Hk, L, D] where `seen`
    [N, 1 or R, L]: its running maximum, sum and unnormalized output."""
    n, r = q.shape[:2]
    rep = c["hq"] // c["hk"]
    # stale slots may hold anything, not-a-number too: no product takes them
    used = seen.any(1)[:, None, :, None]
    k = torch.where(used, k, torch.zeros_like(k[:1, :1, :1, :1]))
    v = torch.where(used, v, torch.zeros_like(v[:1, :1, :1, :1]))
    qh = q.view(n, r, c["hk"], rep, c["d"]).permute(0, 2, 1, 3, 4).reshape(n, c["hk"], r * rep, c["d"])
    x = torch.matmul(qh, k.transpose(-1, -2)).mul_(c["d"] ** -0.5)
    mask = seen[:, None].expand(n, 1, r, seen.shape[-1]).repeat_interleave(rep, 2)
    x = x.masked_fill_(~mask, float("-inf"))
    m = x.amax(-1)
    p = torch.exp_(x.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)[..., None]))
    back = lambda t: t.reshape(n, c["hk"], r, rep, -1).permute(0, 2, 1, 3, 4).reshape(n, r, c["hq"], -1)  # noqa: E731
    return back(m)[..., 0], back(p.sum(-1))[..., 0], back(torch.matmul(p, v))


def _attn(s):
    c = s["c"]
    bs = c["bs"]
    q = s["q"].float()
    table, cu, lens = s["table"].long(), s["cu"].long(), s["lens"].long()
    starts, prefix = s["starts"].long(), s["prefix"].long()
    # the prefix pass: every token of a group over its prefix
    g0, g1 = cu[starts[:-1]], cu[starts[1:]]
    tok = g0[:, None] + torch.arange(s["max_group"], device="cuda")[None]  # [G, R]
    ok = tok < g1[:, None]
    pages = -(-s["max_prefix"] // bs)
    k, v = _rows(c, s["cache"], table[starts[:-1], :pages].clamp_min(0))
    key = torch.arange(pages * bs, device="cuda")[None]
    seen = (key < prefix[:, None])[:, None]
    part = _part(c, q[tok.clamp_max(q.shape[0] - 1)], k, v, seen)
    mp, lp, op = (t[ok] for t in part)
    # the suffix pass: each sequence's tokens over its own keys
    seqs = torch.arange(c["seqs"], device="cuda")
    group = torch.searchsorted(starts[1:], seqs, right=True)
    ahead = prefix[group]
    pages = s["max_suffix"] // bs + 2
    col = (ahead // bs)[:, None] + torch.arange(pages, device="cuda")[None]
    blocks = table.gather(1, col.clamp_max(table.shape[1] - 1)).clamp_min(0)
    k, v = _rows(c, s["cache"], blocks)
    key = (ahead // bs * bs)[:, None] + torch.arange(pages * bs, device="cuda")[None]  # [S, L]
    tok = cu[:-1, None] + torch.arange(s["max_q"], device="cuda")[None]
    ok = tok < cu[1:, None]
    limit = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(s["max_q"], device="cuda")[None]
    seen = ((key >= ahead[:, None])[:, None] & (key[:, None] <= limit[:, :, None])
            & (key < lens[:, None])[:, None])
    part = _part(c, q[tok.clamp_max(q.shape[0] - 1)], k, v, seen)
    ms, ls, os = (t[ok] for t in part)
    # one softmax over both
    m = torch.maximum(mp, ms)
    wp, ws = torch.exp(mp - m), torch.exp(ms - m)
    total = wp * lp + ws * ls
    out = (wp[..., None] * op + ws[..., None] * os)
    if s["sinks"] is not None:
        top = torch.maximum(m, s["sinks"])
        w = torch.exp(m - top)
        total, out, m = total * w + torch.exp(s["sinks"] - top), out * w[..., None], top
    s["out"].copy_(out / total[..., None])
    s["lse"].copy_(m + torch.log(total))


def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        import paged_attention_int8_gb300 as pa
    if op == "tables":
        if own:
            pa.build_block_tables(
                s["ctx"], s["q"], s["source"], s["free"], s["blocks"], s["c"]["bs"], s["tokens"],
                source_rows=s["rows"], shared_lens=s["shared"], free_head=s["head"],
                out=(s["table"], s["cu"], s["lens"], s["slots"], s["pos"], s["pairs"], s["next"]),
                status=s["status"])
        else:
            _tables(s)
        return [s["table"], s["cu"], s["lens"], s["slots"], s["pos"], s["pairs"], s["next"]]
    if op == "copy":
        if own:
            if s["c"]["fmt"] == "q8":
                pa.copy_blocks(s["pairs"], *s["cache"], status=s["status"])
            else:
                pa.copy_blocks_f8v4(s["pairs"], *s["cache"], status=s["status"])
        else:
            _copy(s)
        # a copy moves the codes and scales as they are: whole numbers, scales as their bits
        return [t.view(torch.int16) if t.dtype == torch.float16 else t for t in s["cache"]]
    if own:
        call = pa.paged_attention_shared_prefix if s["c"]["fmt"] == "q8" \
            else pa.paged_attention_shared_prefix_f8v4
        call(s["q"], *s["cache"], s["cu"], s["lens"], s["table"], s["starts"], s["prefix"],
             s["max_q"], s["max_prefix"], s["max_suffix"], sinks=s["sinks"], out=s["out"],
             lse=s["lse"], workspace=s["workspace"])
    else:
        _attn(s)
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """Attention in 64 bits, sequence by sequence, over the dequantized pages;
    the other operators move whole numbers."""
    c = case
    if c["op"] != "attn":
        return None
    s = prepare(case, seed)
    starts, prefix, qlens, lens = _attn_lens(c)
    d, hk, bs, rep = c["d"], c["hk"], c["bs"], c["hq"] // c["hk"]

    def dense(pages, lo, hi):
        """K and V [Hk, hi - lo, D] of keys lo .. hi of a row of pages, fp64."""
        ids = pages[lo // bs: _up(hi, bs)].long()
        a, b = lo - lo // bs * bs, hi - lo // bs * bs
        if c["fmt"] == "q8":
            k = s["cache"][0][ids].double().unflatten(-1, (d // 32, 32)) \
                * s["cache"][1][ids].double()[..., None]
            v = s["cache"][2][ids].double().unflatten(-2, (d // 32, 32)) \
                * s["cache"][3][ids].double()[:, :, :, None, :]
            k, v = k.flatten(-2), v.flatten(-3, -2)
        else:
            k = s["cache"][0][ids].view(torch.float8_e4m3fn).double()
            byte = s["cache"][1][ids].to(torch.int32)
            v = torch.empty((*byte.shape[:-1], bs), dtype=torch.float64, device="cuda")
            v[..., 0::2], v[..., 1::2] = (byte % 16).double(), (byte // 16).double()
            v = v * s["cache"][2][ids].double()[:, :, None] + s["cache"][3][ids].double()[:, :, None]
        k = k.permute(1, 0, 2, 3).reshape(hk, -1, d)[:, a:b]
        v = v.permute(1, 0, 3, 2).reshape(hk, -1, d)[:, a:b]
        return k, v

    outs, lses, at = [], [], 0
    for g in range(c["groups"]):
        kp, vp = dense(s["table"][starts[g]], 0, prefix[g])
        for i in range(starts[g], starts[g + 1]):
            n = qlens[i]
            ks, vs = dense(s["table"][i], prefix[g], lens[i])
            k, v = torch.cat([kp, ks], 1), torch.cat([vp, vs], 1)
            q = s["q"][at:at + n].double().view(n, hk, rep, d).transpose(0, 1)  # [Hk, n, rep, D]
            x = torch.einsum("hnrd,hld->hnrl", q, k) / math.sqrt(d)
            for j in range(n - 1):  # the last query sees every key
                x[:, j, :, lens[i] - n + j + 1:] = -math.inf
            if s["sinks"] is not None:
                sink = s["sinks"].double().view(hk, 1, rep, 1).expand(hk, n, rep, 1)
                x = torch.cat([x, sink], -1)
                v = torch.cat([v, torch.zeros_like(v[:, :1])], 1)
            z = torch.logsumexp(x, -1)
            o = torch.einsum("hnrl,hld->hnrd", torch.exp(x - z[..., None]), v)
            outs.append(o.transpose(0, 1).reshape(n, c["hq"], d))
            lses.append(z.transpose(0, 1).reshape(n, c["hq"]))
            at += n
    return [torch.cat(outs), torch.cat(lses)]
