"""Eviction from the paged caches: which positions stay, the in-place move of
both caches' rows and of the weights, and the whole cycle of a serving loop."""
import math

import pytest
import torch

import sparse_attention_20_b200 as dsa
from sparse_attention_20_b200 import build as dsa_build
import cache_ref as ref
from cache_ref import D_V, SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dsa_build.build()
    dsa.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.synchronize()
    assert dsa.device_status() == 0


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _check_select(mass, lens, keep, sinks=0, recent=0):
    idx, new = dsa.cache_evict_select(mass, _i32(lens), keep, sinks=sinks, recent=recent)
    want = ref.select(mass.cpu(), lens, keep, sinks, recent)
    assert new.tolist() == [len(w) for w in want]
    for b, w in enumerate(want):
        assert idx[b].tolist() == w + [-1] * (keep - len(w)), f"sequence {b}"
    return idx, new


@pytest.mark.parametrize("max_len,lens,keep,sinks,recent", [
    (64, [64, 10, 0, 33, 32, 31], 32, 4, 8),
    (1, [1, 0], 1, 0, 0),
    (777, [777, 776, 500, 101, 100, 99], 100, 0, 0),
    (777, [777, 500], 100, 60, 40),          # nothing left to choose
    (777, [777, 500], 100, 100, 0),
    (777, [777, 500], 100, 0, 100),
    (777, [777, 500], 1, 0, 0),
    (4099, [4099, 4098, 2500], 2049, 3, 1),
    (20001, [20001, 9000, 12345], 5000, 16, 512),
    (131072, [131072, 131071, 70001], 40000, 0, 3000),
    (300000, [300000, 299999], 1000, 4, 4),
    (5, [9, -3, 5], 2, 1, 0),                # lengths outside the table
])
def test_select_is_the_full_sort(max_len, lens, keep, sinks, recent):
    g = torch.Generator(device="cuda").manual_seed(max_len + keep)
    mass = torch.rand(len(lens), max_len, generator=g, device="cuda") ** 4
    _check_select(mass, lens, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "few values", "zeros and one", "signed", "special", "descending",
                                  "close", "all nan"])
@pytest.mark.parametrize("n", [1000, 33333])
def test_select_with_ties_and_special_values(kind, n):
    g = torch.Generator(device="cuda").manual_seed(3)
    mass = torch.rand(3, n, generator=g, device="cuda")
    if kind == "equal":
        mass.fill_(0.5)
    elif kind == "few values":
        mass = (mass * 5).floor()
    elif kind == "zeros and one":
        mass = (mass > 0.999).float() * torch.where(mass > 0.9995, -0.0, 1.0)
        mass[mass == 0] = -0.0
        mass[:, ::2] += 0.0
    elif kind == "signed":
        mass -= 0.5
    elif kind == "special":
        for i, v in enumerate([math.nan, math.inf, -math.inf, -0.0, 0.0, 3e38, 1e-45]):
            mass[:, i::13] = v
    elif kind == "descending":
        mass = mass.sort(1, descending=True).values
    elif kind == "close":
        mass = 1.0 + torch.randint(0, 4, mass.shape, generator=g, device="cuda") * 2.0 ** -23
    else:
        mass.fill_(math.nan)
    for keep, sinks, recent in ((n // 2, 0, 0), (n // 3, 5, 100), (7, 2, 2)):
        _check_select(mass, [n, n - 1, n // 2 + 1], keep, sinks, recent)


@pytest.mark.parametrize("max_len,n,offset", [(5001, 3, 0), (12000, 64, 0), (70003, 2, 1), (40000, 200, 0)])
def test_select_at_every_alignment_and_cluster(max_len, n, offset):
    """Rows that start on any 4-byte boundary; few and many sequences."""
    g = torch.Generator(device="cuda").manual_seed(max_len)
    mass = torch.rand(n, max_len, generator=g, device="cuda")
    lens = [max_len - (i * 977) % (max_len // 2) for i in range(n)]
    _check_select(mass, lens, max_len // 3 + offset, 3, 50)


def test_select_captured_and_replayed():
    mass = torch.rand(4, 5000, device="cuda")
    lens = _i32([5000, 4000, 100, 3001])
    idx, new = dsa.cache_evict_select(mass, lens, 600, sinks=4, recent=32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.cache_evict_select(mass, lens, 600, sinks=4, recent=32, keep_idx=idx, new_len=new)
    for _ in range(2):
        mass.copy_(torch.rand_like(mass))
        lens.copy_(torch.randint(1, 5001, (4,)))
        g.replay()
        torch.cuda.synchronize()
        want = ref.select(mass.cpu(), lens.tolist(), 600, 4, 32)
        for b, w in enumerate(want):
            assert idx[b].tolist() == w + [-1] * (600 - len(w))


def _caches(lens, page, seed, row=576, key=128):
    x = ref.make(lens, [1] * len(lens), 1, page, seed=seed, extra_pages=1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.randint(-2 ** 15, 2 ** 15, (x.pages.shape[0], row), generator=g, device="cuda").short()
    keys = torch.randint(0, 256, (x.pages.shape[0], key), generator=g, device="cuda").to(torch.uint8)
    mass = torch.rand(len(lens), x.S, generator=g, device="cuda")
    return rows.view(torch.bfloat16), keys, x.table, mass


@pytest.mark.parametrize("lens,page,keep,sinks,recent,row,key", [
    ([200, 64, 130, 1], 64, 64, 4, 16, 576, 128),
    ([1000, 300, 999], 192, 257, 0, 0, 576, 128),
    ([1000, 300, 999], 64, 999, 0, 0, 8, 16),
    ([5000], 64, 4000, 16, 100, 576, 128),
    ([700] * 40, 128, 333, 1, 2, 24, 48),
    ([3000, 2000], 256, 1, 0, 0, 2048, 4096),
    ([30000], 64, 29999, 0, 0, 576, 128),
])
def test_compaction_moves_every_kept_row(lens, page, keep, sinks, recent, row, key):
    rows, keys, table, mass = _caches(lens, page, seed=len(lens) + keep, row=row, key=key)
    score = torch.rand(mass.shape, device="cuda")
    idx, new = dsa.cache_evict_select(score, _i32(lens), keep, sinks=sinks, recent=recent)
    want_rows = ref.compact(rows.view(torch.int16).cpu(), page, table.cpu(), idx.cpu(), new.cpu())
    want_keys = ref.compact(keys.cpu(), page, table.cpu(), idx.cpu(), new.cpu())
    want_mass = torch.zeros_like(mass)
    for b in range(len(lens)):
        m = int(new[b])
        want_mass[b, :m] = mass[b, idx[b, :m].long()]
    r2, k2 = rows.clone(), keys.clone()
    dsa.cache_compact_paged(rows, page, table, idx, new, k_pages=keys, mass=mass)
    torch.cuda.synchronize()
    assert torch.equal(rows.view(torch.int16).cpu(), want_rows)
    assert torch.equal(keys.cpu(), want_keys)
    assert torch.equal(mass, want_mass)
    # each pool alone
    dsa.cache_compact_paged(r2, page, table, idx, new)
    dsa.cache_compact_paged(k2, page, table, idx, new)
    torch.cuda.synchronize()
    assert torch.equal(r2.view(torch.int16).cpu(), want_rows) and torch.equal(k2.cpu(), want_keys)


def test_compaction_leaves_bad_entries_alone():
    rows, keys, table, mass = _caches([500, 300], 64, seed=4)
    idx, new = dsa.cache_evict_select(mass, _i32([500, 300]), 100)
    table[0, 2] = 10 ** 6          # outside the pool: rows from there, or to there, stay
    table[1, 0] = -1
    idx[0, 50] = 10 ** 6
    idx[0, 99] = -1
    new[1] = 10 ** 6               # clipped to keep
    want = ref.compact(rows.view(torch.int16).cpu(), 64, table.cpu(), idx.cpu(), new.cpu())
    dsa.cache_compact_paged(rows, 64, table, idx, new, k_pages=keys)
    torch.cuda.synchronize()
    assert torch.equal(rows.view(torch.int16).cpu(), want)


def test_compaction_captured_with_the_selection():
    lens = [900, 400]
    rows, keys, table, mass = _caches(lens, 64, seed=6)
    n = _i32(lens)
    idx, new = dsa.cache_evict_select(mass, n, 128, sinks=4, recent=32)
    before = rows.clone(), keys.clone(), mass.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.cache_evict_select(mass, n, 128, sinks=4, recent=32, keep_idx=idx, new_len=new)
        dsa.cache_compact_paged(rows, 64, table, idx, new, k_pages=keys, mass=mass)
    g.replay()
    torch.cuda.synchronize()
    want = ref.select(before[2].cpu(), lens, 128, 4, 32)
    assert idx.tolist() == want
    assert torch.equal(rows.view(torch.int16).cpu(),
                       ref.compact(before[0].view(torch.int16).cpu(), 64, table.cpu(), idx.cpu(), new.cpu()))
    assert torch.equal(mass[0, :128], before[2][0, idx[0].long()]) and bool((mass[:, 128:] == 0).all())


def test_a_bounded_cache_from_prompt_to_decode():
    """Prompt chunks, their received weights, eviction, and decode steps on the
    smaller cache, as a serving loop runs them: each step against fp64 on the
    state that the steps before left."""
    page, H, keep = 64, 128, 150
    lens = [410, 233]
    x = ref.make(lens, [210, 133], H, page, seed=31)
    keys = torch.randint(0, 120, (x.pages.shape[0], 128), device="cuda").to(torch.uint8)
    mass = torch.zeros(2, x.S, device="cuda")
    out, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V)
    ref.check_attention(x, out, lse)
    want, tol = ref.received(x, lse, mass)
    dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=mass)
    assert bool(((mass.double() - want).abs() <= tol).all())

    idx, new = dsa.cache_evict_select(mass, _i32(lens), keep, sinks=4, recent=32)
    assert idx.tolist() == ref.select(mass.cpu(), lens, keep, 4, 32)
    kept = mass.gather(1, idx.long())
    rows = ref.compact(x.pages.view(torch.int16).cpu(), page, x.table.cpu(), idx.cpu(), new.cpu())
    dsa.cache_compact_paged(x.pages, page, x.table, idx, new, k_pages=keys, mass=mass)
    torch.cuda.synchronize()
    assert torch.equal(x.pages.view(torch.int16).cpu(), rows)
    assert torch.equal(mass[:, :keep], kept) and bool((mass[:, keep:] == 0).all())

    n = new.clone()
    for step in range(3):          # one token a step: its row goes to the first free place
        g = torch.Generator(device="cuda").manual_seed(50 + step)
        for b in range(2):
            row = x.rows_of(b, n[b].long().view(1))
            x.pages[row] = torch.randn(1, ref.D_QK, generator=g, device="cuda").bfloat16()
        y = ref.Cache(torch.randn(2, H, ref.D_QK, generator=g, device="cuda").bfloat16(), x.pages, page, x.table,
                      _i32([0, 1]), n.clone(), [])
        window, sinks = (0, 0) if step < 2 else (64, 4)
        out, lse = dsa.mla_attn_paged(*y.args(), SCALE, D_V, window=window, sinks=sinks)
        ref.check_attention(y, out, lse, window=window, sinks=sinks)
        want, tol = ref.received(y, lse, mass, window=window, sinks=sinks)
        dsa.mla_attn_mass_paged(*y.args(), lse, SCALE, mass=mass, window=window, sinks=sinks)
        assert bool(((mass.double() - want).abs() <= tol).all())
        n += 1
