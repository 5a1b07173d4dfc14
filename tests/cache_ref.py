"""64-bit references of the paged latent cache's operators (dense attention of
new tokens, received weights, eviction), a maker of small inputs, and the
error bounds that the tests hold the kernels to. Shared by the GPU tests."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

D_QK, D_V = 576, 512
SCALE = 1.0 / math.sqrt(D_QK)


@dataclass
class Cache:
    q: torch.Tensor
    pages: torch.Tensor
    page_size: int
    table: torch.Tensor
    seq: torch.Tensor
    pos: torch.Tensor
    lens: list

    @property
    def S(self):
        return self.table.shape[1] * self.page_size

    def args(self):
        return self.q, self.pages, self.page_size, self.table, self.seq, self.pos

    def rows_of(self, b, s):
        """Pool rows of positions s of sequence b."""
        page = self.table[b].long()[s // self.page_size]
        page = torch.where((page >= 0) & (page < self.pages.shape[0] // self.page_size), page, 0)
        return page * self.page_size + s % self.page_size


def make(lens, chunks, heads, page_size=64, seed=0, kv_scale=1.0, extra_pages=0):
    """Sequences of `lens` cached tokens whose last chunks[b] are the query rows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = len(lens)
    used = [max(1, -(-v // page_size)) for v in lens]
    max_pages = max(used) + extra_pages
    perm = torch.randperm(sum(used) + 1, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(n, max_pages, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    seq = [b for b in range(n) for _ in range(chunks[b])]
    pos = [lens[b] - chunks[b] + j for b in range(n) for j in range(chunks[b])]
    q = torch.randn(len(seq), heads, D_QK, generator=g, device="cuda").bfloat16()
    pages = (torch.randn((sum(used) + 1) * page_size, D_QK, generator=g, device="cuda") * kv_scale).bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    return Cache(q, pages, page_size, table, torch.tensor(seq, **i32), torch.tensor(pos, **i32), list(lens))


def seen_keys(x, t, window, sinks):
    """Positions that row t sees (long tensor)."""
    b, p = int(x.seq[t]), int(x.pos[t])
    if not 0 <= b < x.table.shape[0] or p < 0:
        return torch.zeros(0, dtype=torch.long, device="cuda")
    s = torch.arange(min(p, x.S - 1) + 1, device="cuda")
    return s[(s > p - window) | (s < sinks)] if window else s


def attention(x, scale=SCALE, window=0, sinks=0):
    """(out, lse, tol_out, tol_lse) in fp64, row by row.

    Bounds: a logit is 576 exact bf16 products summed in fp32, at most 64
    roundings deep (36 steps of 16 products), so it is off by
    dx <= 64 2^-23 scale sum|q c|; exp2, log2 and the scaling add a few units
    of 2^-23 relative to the logits' size. The log of the sum moves by at most
    the largest dx. A probability is rounded to bf16 (2^-8 relative), so out is
    off by (2^-8 + 2 dx + 2^-16) sum p|c|, and by its own rounding 2^-8."""
    T, H, _ = x.q.shape
    out = torch.zeros(T, H, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for t in range(T):
        s = seen_keys(x, t, window, sinks)
        if not len(s):
            continue
        c = x.pages[x.rows_of(int(x.seq[t]), s)].double()
        q = x.q[t].double()
        z = q @ c.T * scale
        l = torch.logsumexp(z, 1)
        p = torch.exp(z - l[:, None])
        dx = 64 * 2.0 ** -23 * abs(scale) * (q.abs() @ c.abs().T).amax(1) + 8 * 2.0 ** -23 * (1 + z.abs().amax(1))
        lse[t], out[t] = l, p @ c[:, :D_V]
        tol_l[t] = dx + 4 * 2.0 ** -23 * (1 + l.abs())
        tol_o[t] = (2.0 ** -8 + 2 * dx + 2.0 ** -16)[:, None] * (p @ c[:, :D_V].abs()) + 2.0 ** -8 * out[t].abs()
    return out, lse, tol_o, tol_l


def check_attention(x, out, lse, scale=SCALE, window=0, sinks=0):
    ref_o, ref_l, tol_o, tol_l = attention(x, scale, window, sinks)
    dead = torch.isinf(ref_l)
    assert torch.equal(torch.isinf(lse), dead) and bool((lse[dead] < 0).all())
    assert bool(((lse.double() - ref_l).abs()[~dead] <= tol_l[~dead]).all()), "lse"
    assert bool(((out.double() - ref_o).abs() <= tol_o).all()), "out"
    return ref_o, ref_l


def received(x, lse, mass, scale=SCALE, window=0, sinks=0):
    """(mass after, tolerance): the weights added row by row in fp64 to `mass`.

    A weight exp(x - lse) is off by the logit's error (see attention) and a
    few units of 2^-23 of its argument; the fp32 sum over a key's rows and
    heads and the starting value rounds once per addend."""
    out = mass.double().clone()
    rel = torch.zeros((), dtype=torch.float64, device="cuda")
    adds = torch.zeros_like(out)
    T, H, _ = x.q.shape
    for t in range(T):
        s = seen_keys(x, t, window, sinks)
        if not len(s):
            continue
        b = int(x.seq[t])
        c, q = x.pages[x.rows_of(b, s)].double(), x.q[t].double()
        z = q @ c.T * scale
        l = lse[t].double()
        p = torch.where(torch.isinf(l)[:, None], 0.0, torch.exp(z - l[:, None]))
        out[b, s] += p.sum(0)
        adds[b, s] += H
        fin = l[~torch.isinf(l)]
        big = z.abs().max() + (fin.abs().max() if len(fin) else 0)
        rel = torch.maximum(rel, 64 * 2.0 ** -23 * abs(scale) * (q.abs() @ c.abs().T).max() + 8 * 2.0 ** -23 * (1 + big))
    return out, out.abs() * (rel + (adds + 1) * 2.0 ** -24)


def select(mass, seq_len, keep, sinks, recent):
    """keep_idx (list of lists) by a full sort: (-mass, position), NaN as -inf."""
    rows = []
    for b in range(mass.shape[0]):
        n = max(0, min(int(seq_len[b]), mass.shape[1]))
        if n <= keep:
            rows.append(list(range(n)))
            continue
        w = [-math.inf if math.isnan(v) else v for v in mass[b, :n].tolist()]
        middle = sorted(range(sinks, n - recent), key=lambda s: (-w[s], s))[:keep - sinks - recent]
        rows.append(sorted(list(range(sinks)) + middle + list(range(n - recent, n))))
    return rows


def compact(rows, page_size, table, keep_idx, new_len):
    """Page pool `rows` after the kept rows moved to the front."""
    out = rows.clone()
    num = rows.shape[0] // page_size
    for b in range(table.shape[0]):
        for j in range(min(int(new_len[b]), keep_idx.shape[1])):
            s = int(keep_idx[b, j])
            if s <= j or s >= table.shape[1] * page_size:
                continue
            a, z = int(table[b, s // page_size]), int(table[b, j // page_size])
            if 0 <= a < num and 0 <= z < num:
                out[z * page_size + j % page_size] = rows[a * page_size + s % page_size]
    return out
