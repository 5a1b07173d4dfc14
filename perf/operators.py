"""Operators over the paged latent cache: dense and windowed MLA attention of
newly added tokens, the attention weight each cached token has received, and
eviction of the least-attended tokens.

The caches are the framework's own: bf16 latent rows c_s of 512 + 64 columns
and e4m3 indexer keys of 128, in pages named by a block table; a query row t
belongs to sequence seq[t] and sees that sequence's keys s <= pos[t] (its last
`window` keys and the first `sinks` where window > 0).

  attn     out[t,h] = sum_s p_s c_s[0:512],  lse[t,h] = log sum_s exp(x_s),
           x_s = scale q[t,h].c_s,  p_s = exp(x_s - lse[t,h])
  mass     mass[b,s] += sum over rows t of sequence b and heads h of p_s
  select   the `keep` positions of each sequence that stay: the first `sinks`,
           the last `recent`, and the others with the largest mass (ties to
           the lower position), ascending
  compact  the kept positions' rows moved, in place, to positions 0, 1, ...

`own = False` computes them with elementary torch operations in fp32;
`own = True` calls the package's entry points on the same state.
"""
import math

import numpy as np
import torch

own = False

D_QK, D_V, D_IDX = 576, 512, 128
SCALE = 1.0 / math.sqrt(D_QK)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one request, its first generated token after a short prompt: latency
        dict(name="attn_one_short", op="attn", seqs=1, chunk=1, heads=128, lo=200, hi=200, page=64, window=0,
             sinks=0, pad=0),
        # a serving batch's decode step (64 sequences, one token each)
        dict(name="attn_decode64", op="attn", seqs=64, chunk=1, heads=128, lo=2048, hi=32768, page=64, window=0,
             sinks=0, pad=0),
        # drafted tokens checked in one step, on one of two head shards, in a batch padded by three rows
        dict(name="attn_draft", op="attn", seqs=12, chunk=7, heads=64, lo=900, hi=6001, page=128, window=0, sinks=0,
             pad=3),
        # two prompts' next chunk of 512 tokens behind an 8K context
        dict(name="attn_chunk512", op="attn", seqs=2, chunk=512, heads=128, lo=7777, hi=8704, page=64, window=0,
             sinks=0, pad=0),
        # a few sequences of the longest context
        dict(name="attn_decode_long", op="attn", seqs=3, chunk=1, heads=128, lo=98305, hi=131072, page=256, window=0,
             sinks=0, pad=0),
        # decode step that keeps a window and a few first tokens
        dict(name="window_decode64", op="attn", seqs=64, chunk=1, heads=128, lo=300, hi=16384, page=64, window=1024,
             sinks=16, pad=0),
        # a prompt's chunk through the window, on one of eight head shards
        dict(name="window_chunk1000", op="attn", seqs=1, chunk=1000, heads=16, lo=20001, hi=20001, page=64,
             window=2047, sinks=4, pad=0),
        # weights received during a decode step
        dict(name="mass_decode32", op="mass", seqs=32, chunk=1, heads=128, lo=2048, hi=32768, page=64, window=0,
             sinks=0, pad=0),
        # weights received during a prompt's last 256 tokens
        dict(name="mass_chunk256", op="mass", seqs=1, chunk=256, heads=128, lo=12289, hi=12289, page=64, window=0,
             sinks=0, pad=0),
        # which of up to 128K tokens stay, for a batch
        dict(name="select64", op="select", seqs=64, lo=4000, hi=131072, page=64, keep=8192, sinks=16, recent=512),
        # the kept rows of both caches moved together
        dict(name="compact_one", op="compact", seqs=1, lo=65001, hi=65001, page=64, keep=16384, sinks=4, recent=1024),
        dict(name="compact32", op="compact", seqs=32, lo=3000, hi=16384, page=64, keep=4099, sinks=16, recent=256),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "window", "mass", "select", "compact"])
    page = rng.choice([64, 128, 192, 256])
    if op in ("select", "compact"):
        seqs = _log_uniform(rng, 1, 64)
        hi = _log_uniform(rng, 64, min(131072, (131072 * 64 if op == "select" else 16384 * 32) // seqs))
        lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
        keep = max(2, int(hi * rng.uniform(0.03, 0.9)))
        sinks = min(rng.choice([0, 1, 4, 16, 61]), keep // 2)
        recent = min(_log_uniform(rng, 1, 2048) - 1, keep - sinks)
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, page=page, keep=keep, sinks=sinks, recent=recent)
    seqs = _log_uniform(rng, 1, 64)
    heads = rng.choice([128, 128, 64, 32, 16])
    chunk = 1 if rng.random() < 0.4 else _log_uniform(rng, 2, 512)
    hi = _log_uniform(rng, max(64, chunk), 131072)
    # no dearer than the listed chunk: rows x heads x keys and cache rows
    while seqs * chunk * heads * hi > 2 * 512 * 128 * 8192 or seqs * hi > 64 * 20000:
        if chunk > 1 and (rng.random() < 0.5 or hi <= 256):
            chunk = max(1, chunk // 2)
        elif hi > 128:
            hi = hi * 2 // 3
        else:
            seqs = max(1, seqs // 2)
        hi = max(hi, chunk)
    lo = max(chunk, int(hi * rng.uniform(0.05, 1.0)))
    window = _log_uniform(rng, 16, 4096) if op == "window" or rng.random() < 0.2 else 0
    sinks = rng.choice([0, 1, 4, 16, 100]) if window else 0
    return dict(op="attn" if op == "window" else op, seqs=seqs, chunk=chunk, heads=heads, lo=lo, hi=hi, page=page,
                window=window, sinks=sinks, pad=rng.choice([0, 0, 1, 5]) if op != "mass" else 0)


def _lengths(case):
    """Cached tokens of each sequence (the new ones among them): spread over [lo, hi], the longest first."""
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    return [hi - int((hi - lo) * ((0.6180339887 * i) % 1.0)) for i in range(n)]


# ------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    lens = _lengths(case)
    n, page = case["seqs"], case["page"]
    max_pages = -(-max(lens) // page)
    state = dict(case=case, page=page, len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "select":
        S = max_pages * page
        # accumulated weights: a long tail, and tokens that no row has looked at yet
        u = torch.rand(n, S, generator=g, device="cuda")
        state["mass"] = torch.where(u < 0.05, torch.zeros_like(u), u ** 6 * 10 + 1e-3 * u)
        state["keep_idx"] = torch.empty(n, case["keep"], dtype=torch.int32, device="cuda")
        state["new_len"] = torch.empty(n, dtype=torch.int32, device="cuda")
        return state
    used = [-(-v // page) for v in lens]
    num_pages = sum(used) + 3
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(n, max_pages, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    state["table"] = table
    state["pages"] = _normal(g, num_pages * page, D_QK)
    if case["op"] == "compact":
        keep = case["keep"]
        k = torch.randn(num_pages * page, D_IDX, generator=g, device="cuda").clamp_(-448, 448)
        state["k_pages"] = k.to(torch.float8_e4m3fn)
        S = max_pages * page
        state["mass"] = torch.rand(n, S, generator=g, device="cuda")
        score = torch.rand(n, S, generator=g, device="cuda")
        idx, new = _select(score, state["len"], keep, case["sinks"], case["recent"])
        state["keep_idx"], state["new_len"] = idx, new
        return state
    c, pad, H = case["chunk"], case["pad"], case["heads"]
    T = n * c + pad
    # sequence b's rows are its last `chunk` tokens; padding rows belong to no sequence
    seq = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    seq[:n * c] = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(c)
    pos[:n * c] = (state["len"].view(n, 1) - c + torch.arange(c, device="cuda", dtype=torch.int32)).reshape(-1)
    state["seq"], state["pos"] = seq, pos
    state["q"] = _normal(g, T, H, D_QK)
    if case["op"] == "mass":
        state["mass"] = torch.rand(n, max_pages * page, generator=g, device="cuda")
        x, _, _ = _logits(state)
        state["lse"] = _log_sum(x).reshape(T, H).contiguous()
    else:
        state["out"] = torch.empty(T, H, D_V, dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
    return state


# -------------------------------------------------------------- plain forms

def _cache_rows(state, at):
    """Pool rows of logical positions `at` [n, m]."""
    page, table = state["page"], state["table"].long()
    return table.gather(1, at // page) * page + at % page


def _logits(state):
    """(x [n, c*H, m] with -inf where a row does not see a key, keys [n, m, 576], positions [n, m]): the m
    positions are the whole cache, or the first tokens and the stretch that the rows' windows cover."""
    case = state["case"]
    n, c, H, window, sinks = (case[k] for k in ("seqs", "chunk", "heads", "window", "sinks"))
    S = state["table"].shape[1] * state["page"]
    first = (state["len"].long() - c).view(n, 1)                   # the first new token's position
    if window and sinks + window + c - 1 < S:
        lo = (first - window + 1).clamp_min(0)
        at = lo + torch.arange(window + c - 1, device="cuda")
        real = (at >= sinks) & (at < S)
        at = torch.cat([torch.arange(sinks, device="cuda").expand(n, sinks), at], 1)
        real = torch.cat([torch.ones(n, sinks, dtype=torch.bool, device="cuda"), real], 1)
        at = at.clamp_max(S - 1)
    else:
        at = torch.arange(S, device="cuda").expand(n, S)
        real = torch.ones(n, S, dtype=torch.bool, device="cuda")
    keys = state["pages"][_cache_rows(state, at)].float()
    q = state["q"][:n * c].reshape(n, c * H, D_QK).float()
    x = torch.bmm(q, keys.transpose(1, 2)).mul_(SCALE).view(n, c, H, -1)
    p = (first + torch.arange(c, device="cuda")).unsqueeze(2)       # [n, c, 1]
    seen = real.unsqueeze(1) & (at.unsqueeze(1) <= p)
    if window:
        seen &= (at.unsqueeze(1) > p - window) | (at.unsqueeze(1) < sinks)
    x.masked_fill_(~seen.unsqueeze(2), -math.inf)
    return x.view(n, c * H, -1), keys, at


def _log_sum(x):
    m = x.max(-1, keepdim=True).values
    return (x - m).exp_().sum(-1).log_() + m.squeeze(-1)


def _attn(state):
    case = state["case"]
    n, c, H = case["seqs"], case["chunk"], case["heads"]
    x, keys, _ = _logits(state)
    m = x.max(-1, keepdim=True).values
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out, lse = state["out"], state["lse"]
    out[:n * c] = (torch.bmm(p, keys[:, :, :D_V]) / total).view(n * c, H, D_V).to(torch.bfloat16)
    lse[:n * c] = (total.log() + m).view(n * c, H)
    out[n * c:] = 0
    lse[n * c:] = -math.inf
    return out, lse


def _mass(state):
    case = state["case"]
    n, c, H = case["seqs"], case["chunk"], case["heads"]
    x, _, at = _logits(state)
    p = x.sub_(state["lse"][:n * c].view(n, c * H, 1)).exp_()
    state["mass"].scatter_add_(1, at.contiguous(), p.sum(1))
    return state["mass"]


def _select(mass, length, keep, sinks, recent):
    """(positions [n, keep] ascending, -1 behind the last; how many)."""
    n, S = mass.shape
    s = torch.arange(S, device="cuda")
    length = length.long().view(n, 1)
    score = torch.where(torch.isnan(mass), torch.full_like(mass, -math.inf), mass)
    # protected positions first, then by weight, positions behind the end last
    rank = torch.where(s >= length, 2, torch.where((s < sinks) | (s >= length - recent), 0, 1))
    order = torch.sort(score, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(rank.gather(1, order), dim=1, stable=True).indices)
    new = length.clamp_max(keep)
    top = order[:, :keep]
    if top.shape[1] < keep:
        top = torch.cat([top, torch.zeros(n, keep - top.shape[1], dtype=top.dtype, device="cuda")], 1)
    j = torch.arange(keep, device="cuda")
    top = torch.sort(torch.where(j < new, top, S), dim=1).values
    return torch.where(j < new, top, -1).to(torch.int32), new.view(n).to(torch.int32)


def _compact(state):
    idx, new = state["keep_idx"].long(), state["new_len"].long().view(-1, 1)
    n, keep = idx.shape
    S = state["mass"].shape[1]
    j = torch.arange(keep, device="cuda").expand(n, keep)
    live = j < new
    to = _cache_rows(state, j.clamp_max(S - 1)).view(-1)
    src = _cache_rows(state, idx.clamp_min(0)).view(-1)
    # a position behind the last kept one writes the last kept row once more
    last = (new - 1).clamp_min(0)
    to = torch.where(live, to.view(n, keep), to.view(n, keep).gather(1, last)).view(-1)
    src = torch.where(live, src.view(n, keep), src.view(n, keep).gather(1, last)).view(-1)
    pages, keys, mass = state["pages"], state["k_pages"].view(torch.uint8), state["mass"]
    pages[to] = pages[src]
    keys[to] = keys[src]
    kept = mass.gather(1, idx.clamp_min(0))
    s = torch.arange(S, device="cuda")
    wide = kept.gather(1, s.clamp_max(keep - 1).expand(n, S))
    mass.copy_(torch.where(s < new, wide, torch.zeros_like(wide)))
    return pages, state["k_pages"], mass


# --------------------------------------------------------------------- run

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import sparse_attention_20_b200 as dsa
        if op == "attn":
            return dsa.mla_attn_paged(state["q"], state["pages"], state["page"], state["table"], state["seq"],
                                      state["pos"], SCALE, D_V, window=case["window"], sinks=case["sinks"],
                                      out=state["out"], lse=state["lse"])
        if op == "mass":
            return dsa.mla_attn_mass_paged(state["q"], state["pages"], state["page"], state["table"], state["seq"],
                                           state["pos"], state["lse"], SCALE, mass=state["mass"],
                                           window=case["window"], sinks=case["sinks"])
        if op == "select":
            return dsa.cache_evict_select(state["mass"], state["len"], case["keep"], sinks=case["sinks"],
                                          recent=case["recent"], keep_idx=state["keep_idx"],
                                          new_len=state["new_len"])
        dsa.cache_compact_paged(state["pages"], state["page"], state["table"], state["keep_idx"], state["new_len"],
                                k_pages=state["k_pages"], mass=state["mass"])
        return state["pages"], state["k_pages"], state["mass"]
    if op == "attn":
        return _attn(state)
    if op == "mass":
        return _mass(state)
    if op == "select":
        return _select(state["mass"], state["len"], case["keep"], case["sinks"], case["recent"])
    return _compact(state)


# -------------------------------------------------------------------- work

def _seen(p, window, sinks):
    """Keys that a row at position p sees."""
    if not window or p < window:
        return p + 1
    return window + min(sinks, p - window + 1)


def work(case):
    lens = _lengths(case)
    n = case["seqs"]
    if case["op"] == "select":
        return dict(bytes=4.0 * sum(v for v in lens if v > case["keep"]) + 4.0 * n * case["keep"], flops=0)
    if case["op"] == "compact":
        # kept rows read and written once (a sequence that fits, and its first tokens, stay where they are)
        moved = sum(case["keep"] - case["sinks"] for v in lens if v > case["keep"])
        zeros = sum(v - case["keep"] for v in lens if v > case["keep"])
        return dict(bytes=2.0 * moved * (2 * D_QK + D_IDX + 4) + 4.0 * n * case["keep"] + 4.0 * zeros, flops=0)
    c, H, window, sinks = case["chunk"], case["heads"], case["window"], case["sinks"]
    pairs = sum(_seen(v - c + j, window, sinks) for v in lens for j in range(c))
    # keys that some row of the sequence sees
    rows = sum(v if not window else min(v, min(window + c - 1, v) + min(sinks, max(0, v - window - c + 1)))
               for v in lens)
    T = n * c + case["pad"]
    if case["op"] == "mass":
        return dict(bytes=2.0 * D_QK * (rows + T * H) + 4.0 * T * H + 8.0 * rows, flops=2.0 * H * D_QK * pairs)
    return dict(bytes=2.0 * D_QK * (rows + T * H) + 2.0 * T * H * D_V + 4.0 * T * H,
                flops=2.0 * H * (D_QK + D_V) * pairs)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits, one sequence (and a block of rows) at a time."""
    state = prepare(case, seed)
    op, lens, page = case["op"], _lengths(case), case["page"]
    if op == "select":
        return _exact_select(case, state["mass"].double().cpu(), lens)
    table = state["table"].long()
    if op == "compact":
        # the kept rows' new places, sequence by sequence, from copies of the old contents
        pages, keys, mass = state["pages"].clone(), state["k_pages"].clone(), torch.zeros_like(state["mass"])
        old_k, new_k = state["k_pages"].view(torch.uint8), keys.view(torch.uint8)
        for b in range(case["seqs"]):
            m = int(state["new_len"][b])
            kept = state["keep_idx"][b, :m].long()
            j = torch.arange(m, device="cuda")
            src, to = table[b, kept // page] * page + kept % page, table[b, j // page] * page + j % page
            pages[to] = state["pages"][src]
            new_k[to] = old_k[src]
            mass[b, :m] = state["mass"][b, kept]
        return pages, keys, mass.double()
    H, c, window, sinks = case["heads"], case["chunk"], case["window"], case["sinks"]
    T = state["q"].shape[0]
    out = torch.zeros(T, H, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    mass = state["mass"].double() if op == "mass" else None
    for b, length in enumerate(lens):
        s = torch.arange(length, device="cuda")
        rows = state["pages"][table[b, s // page] * page + s % page].double()
        for t0 in range(0, c, 32):
            m = min(32, c - t0)
            t = b * c + t0
            p = length - c + t0 + torch.arange(m, device="cuda").view(m, 1)
            seen = s <= p
            if window:
                seen = seen & ((s > p - window) | (s < sinks))
            z = torch.einsum("thd,sd->ths", state["q"][t:t + m].double(), rows) / math.sqrt(D_QK)
            if op == "mass":
                w = torch.exp(z - state["lse"][t:t + m].double().unsqueeze(2))
                mass[b, :length] += torch.where(seen.unsqueeze(1), w, torch.zeros_like(w)).sum((0, 1))
                continue
            z = torch.where(seen.unsqueeze(1), z, torch.full_like(z, -math.inf))
            l = torch.logsumexp(z, 2)
            lse[t:t + m] = l
            out[t:t + m] = torch.einsum("ths,sd->thd", torch.exp(z - l.unsqueeze(2)), rows[:, :D_V])
    return mass if op == "mass" else (out, lse)


def _exact_select(case, mass, lens):
    keep, sinks, recent = case["keep"], case["sinks"], case["recent"]
    idx = torch.full((len(lens), keep), -1, dtype=torch.int32)
    for b, length in enumerate(lens):
        if length <= keep:
            chosen = list(range(length))
        else:
            w = mass[b, sinks:length - recent].numpy()
            middle = np.lexsort((np.arange(w.size), -w))[:keep - sinks - recent] + sinks
            chosen = sorted(list(range(sinks)) + middle.tolist() + list(range(length - recent, length)))
        idx[b, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return idx.cuda(), torch.tensor([min(v, keep) for v in lens], dtype=torch.int32, device="cuda")
