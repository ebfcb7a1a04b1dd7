"""Shared-prefix batches for the tests: seeded caches filled by the library's
stores, and a plain fp64 implementation of the attention over the dequantized
pages with the bounds its comparison needs."""
from __future__ import annotations

import random
from dataclasses import dataclass

import torch

from paged_attention_int8_gb300 import _lib, inputs
from tests import _harness as H


@dataclass
class Batch:
    fmt: str
    hq: int
    hk: int
    d: int
    bs: int
    prefix: list       # per group
    starts: list       # first sequence of each group, and the number of sequences
    q_lens: list
    seq_lens: list
    cache: list        # device tensors in the order of the calls
    table: torch.Tensor
    q: torch.Tensor    # [T (+ padding rows), Hq, D]
    cu: torch.Tensor
    lens: torch.Tensor
    groups: torch.Tensor
    prefixes: torch.Tensor
    sinks: torch.Tensor | None
    blocks: int

    @property
    def bounds(self):
        group = [g for g in range(len(self.prefix))
                 for _ in range(self.starts[g], self.starts[g + 1])]
        suffix = [n - self.prefix[g] for n, g in zip(self.seq_lens, group)]
        return max(self.q_lens), max(self.prefix), max(suffix)

    def call(self, **kw):
        """The call under test, its status checked; out and lse start as NaN."""
        fn = (_lib.paged_attention_shared_prefix if self.fmt == "q8"
              else _lib.paged_attention_shared_prefix_f8v4)
        bounds = kw.pop("bounds", self.bounds)
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device=self.q.device)
        ws = kw.pop("workspace", None)
        if ws is None:
            need = _lib.shared_prefix_workspace_size(
                len(self.seq_lens), self.q.shape[0], len(self.prefix), self.hq, self.hk, self.d,
                *bounds)
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=self.q.device)
            ws[:4] = 0
        fn(self.q, *self.cache, self.cu, self.lens, self.table, self.groups, self.prefixes,
           *bounds, sinks=self.sinks, out=out, lse=lse, workspace=ws, **kw)
        bits = _lib.check_status(ws)
        assert bits == 0
        return out, lse


def make(seed, device, fmt, hq, hk, d, bs, groups, sinks=None, pad_rows=0, q_scale=1.0,
         k_bias=1.0, spare=3, columns=2):
    """groups: [(prefix length, [(query length, keys past the prefix), ...]), ...]."""
    H.ensure_built()
    rnd = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    prefix = [p for p, _ in groups]
    starts, q_lens, seq_lens = [0], [], []
    for p, seqs in groups:
        for ql, own in seqs:
            assert own >= ql
            q_lens.append(ql)
            seq_lens.append(p + own)
        starts.append(len(q_lens))
    n_pages = [-(-x // bs) for x in seq_lens]
    shared = [p // bs for p in prefix]
    blocks = sum(shared) + sum(n_pages) + spare
    ids = list(range(blocks))
    rnd.shuffle(ids)
    table = torch.full((max(1, len(q_lens)), max(n_pages + [1]) + columns), -1, dtype=torch.int32)
    for i, (p, seqs) in enumerate(groups):
        common = [ids.pop() for _ in range(shared[i])]
        for s in range(starts[i], starts[i + 1]):
            row = common + [ids.pop() for _ in range(n_pages[s] - shared[i])]
            table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
    table = table[:len(q_lens)]
    # the stores write every slot some sequence owns; the others keep canaries
    slots = set()
    for s, n in enumerate(seq_lens):
        for x in range(n):
            slots.add(int(table[s, x // bs]) * bs + x % bs)
    slots = torch.tensor(sorted(slots), dtype=torch.int64)
    n = slots.numel()
    bias = torch.randn((hk, d), generator=g) * k_bias
    key = (torch.randn((n, hk, d), generator=g) + bias).bfloat16().to(device)
    value = torch.randn((n, hk, d), generator=g).bfloat16().to(device)
    make_cache = inputs.empty_cache if fmt == "q8" else inputs.empty_cache_f8v4
    cache = list(make_cache(blocks, hk, bs, d, device=device))
    if n:
        store = _lib.kv_store if fmt == "q8" else _lib.kv_store_f8v4
        store(key, value, slots.to(device), *cache)
    tokens = sum(q_lens)
    q = (torch.randn((tokens + pad_rows, hq, d), generator=g) * q_scale).bfloat16().to(device)
    cu = [0]
    for x in q_lens:
        cu.append(cu[-1] + x)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    return Batch(fmt, hq, hk, d, bs, prefix, starts, q_lens, seq_lens, cache, table.to(device), q,
                 i32(cu), i32(seq_lens), i32(starts), i32(prefix),
                 None if sinks is None else torch.tensor(sinks, dtype=torch.float32, device=device),
                 blocks)


def _rows(b, pages, lo, hi):
    """K and V [Hk, hi - lo, D] (fp64, CPU) of keys lo .. hi - 1 of a page row."""
    ids = pages[lo // b.bs: -(-hi // b.bs)].long()
    c = [t[ids.to(t.device)].cpu() for t in b.cache]
    half = lambda t: t.view(torch.float16).double()  # noqa: E731
    if b.fmt == "q8":
        k = c[0].double() * half(c[1]).repeat_interleave(32, -1)
        v = c[2].double() * half(c[3]).repeat_interleave(32, -2)
    else:
        k = c[0].view(torch.float8_e4m3fn).double()
        codes = c[1].to(torch.int64)
        v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
        v = v * half(c[2])[..., None, :] + half(c[3])[..., None, :]
    k = k.permute(1, 0, 2, 3).reshape(b.hk, -1, b.d)
    v = v.permute(1, 0, 3, 2).reshape(b.hk, -1, b.d)
    a = lo - lo // b.bs * b.bs
    return k[:, a:a + hi - lo], v[:, a:a + hi - lo]


def reference(b, scale=None):
    """Per owned token: out [T, Hq, D], lse [T, Hq], and for the bounds
    A = sum_j p_j |v_j| (shaped like out), B = max_j sum_c |q_c k_jc| * scale,
    the largest |v| and the number of keys."""
    scale = b.d ** -0.5 if scale is None else scale
    tokens = sum(b.q_lens)
    rep = b.hq // b.hk
    out = torch.zeros((tokens, b.hq, b.d), dtype=torch.float64)
    lse = torch.zeros((tokens, b.hq), dtype=torch.float64)
    A, B, N = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    Q, V = torch.zeros_like(lse), torch.zeros_like(lse)
    table = b.table.cpu()
    q = b.q.double().cpu()
    sinks = None if b.sinks is None else b.sinks.double().cpu()
    t = 0
    for g, p in enumerate(b.prefix):
        first = b.starts[g]
        for s in range(first, b.starts[g + 1]):
            kp, vp = _rows(b, table[first], 0, p)
            ks, vs = _rows(b, table[s], p, b.seq_lens[s])
            k, v = torch.cat([kp, ks], 1), torch.cat([vp, vs], 1)
            for i in range(b.q_lens[s]):
                n = b.seq_lens[s] - b.q_lens[s] + i + 1
                for h in range(b.hq):
                    kk, vv = k[h // rep, :n], v[h // rep, :n]
                    x = kk @ q[t, h] * scale
                    z = torch.logsumexp(x, 0)
                    if sinks is not None:
                        z = torch.logaddexp(z, sinks[h])
                    w = torch.exp(x - z)
                    out[t, h], lse[t, h] = w @ vv, z
                    A[t, h] = w @ vv.abs()
                    B[t, h] = (kk.abs() @ q[t, h].abs()).max() * abs(scale)
                    Q[t, h] = q[t, h].abs().sum() * abs(scale)
                    N[t, h], V[t, h] = n, vv.abs().max()
                t += 1
    return out, lse, A, B, Q, N, V


def check(b, out, lse, ref=None, scale=None, where=""):
    """out and lse against fp64, element by element.

    Score error e_s: the fp32 accumulation of D products in the tensor cores,
    each of at most D + 16 additions (with the group or part sums) off by 2^-23
    of a magnitude that B bounds; the low part of a split key and q below
    2^-14, each within 2^-25 of the other factor (counted twice).
    lse: e_s, the exponentials (2^-22 relative), the sums and the logarithm:
    e_s + 2^-18 max(1, |lse|).
    out: weights off by 2 e_s relative (numerator and denominator), P and V'
    rounded to fp16 (2^-11 each), exponentials and sums (2^-18), all against
    A; P below 2^-14 within 2^-25 of the largest |v| per key; the bf16
    rounding 2^-8 |out|."""
    r_out, r_lse, A, B, Q, N, V = reference(b, scale) if ref is None else ref
    tokens = r_out.shape[0]
    o, z = out[:tokens].double().cpu(), lse[:tokens].double().cpu()
    assert torch.isfinite(o).all() and torch.isfinite(z).all(), where
    e_s = (b.d + 16) * 2.0 ** -23 * B + 2 * 2.0 ** -25 * Q
    d_lse = (z - r_lse).abs()
    t_lse = e_s + 2.0 ** -18 * r_lse.abs().clamp_min(1)
    assert (d_lse <= t_lse).all(), f"{where}: lse {float((d_lse / t_lse).max()):.2f} of its bound"
    w = 2 * e_s + 2 * 2.0 ** -11 + 2.0 ** -18
    t_out = 2.0 ** -8 * r_out.abs() + w[..., None] * A * (1 + 2.0 ** -8) \
        + (N * V)[..., None] * 2.0 ** -25
    d_out = (o - r_out).abs()
    assert (d_out <= t_out).all(), f"{where}: out {float((d_out / t_out).max()):.2f} of its bound"
    # rows that no sequence owns are left as they were
    assert torch.isnan(out[tokens:].float()).all() and torch.isnan(lse[tokens:]).all(), where
