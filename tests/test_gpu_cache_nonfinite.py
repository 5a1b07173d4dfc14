"""Infinities and NaN in cached rows that query rows do see: dense paged
attention gives what the formulas give, wherever in a tile the key lies."""
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


def _check(x, window=0, sinks=0):
    """out and lse against the formulas in 64 bits: the same elements are no
    numbers, and the others are within cache_ref's bounds, taken over the keys
    whose rows are finite (others have a weight of 0 where anything is finite)."""
    out, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert dsa.device_status() == 0
    kinds = set()
    for t in range(x.q.shape[0]):
        s = ref.seen_keys(x, t, window, sinks)
        if not len(s):
            assert bool((out[t] == 0).all()) and bool((lse[t] == -math.inf).all())
            continue
        c, q = x.pages[x.rows_of(int(x.seq[t]), s)].double(), x.q[t].double()
        z = q @ c.T * SCALE
        l = torch.logsumexp(z, 1)
        p = torch.exp(z - l[:, None])
        o = p @ c[:, :D_V]
        # a logit of +inf: inf - inf in the softmax, hence NaN in lse, too
        assert torch.equal(torch.isnan(lse[t]), torch.isnan(l) | (l == math.inf)), t
        assert torch.equal(lse[t] == -math.inf, l == -math.inf), t
        assert torch.equal(torch.isnan(out[t]), torch.isnan(o)), t
        assert not bool(torch.isinf(out[t]).any())
        fin = torch.isfinite(c).all(1)
        cf, zf = c[fin], z[:, fin]
        dx = 64 * 2.0 ** -23 * SCALE * (q.abs() @ cf.abs().T).amax(1) + 8 * 2.0 ** -23 * (1 + zf.abs().amax(1)) \
            if bool(fin.any()) else torch.zeros_like(l)
        ok = torch.isfinite(l)
        assert bool(((lse[t].double() - l).abs() <= dx + 4 * 2.0 ** -23 * (1 + l.abs()))[ok].all()), t
        tol = (2.0 ** -8 + 2 * dx + 2.0 ** -16)[:, None] * (p[:, fin] @ cf[:, :D_V].abs()) + 2.0 ** -8 * o.abs()
        good = ~torch.isnan(o)
        assert bool(((out[t].double() - o).abs() <= tol)[good].all()), t
        kinds |= {"number" if bool(good[h].all()) else "columns" if bool(good[h].any()) else "row"
                  for h in range(x.q.shape[1])}
    return kinds


def _put(x, b, s, col, value):
    x.pages[x.rows_of(b, torch.tensor([s], device="cuda")), col] = value


@pytest.mark.parametrize("heads,lens,chunk,window,sinks,where", [
    (128, [300], 3, 0, 0, (298, 299)),            # tiles that only some rows see whole
    (128, [300], 3, 0, 0, (5, 130)),              # tiles that all do
    (16, [333, 190], 11, 0, 0, (185, 188, 5)),
    (16, [333, 190], 11, 70, 5, (3, 124, 130, 187)),
    (64, [257], 2, 100, 3, (1, 157, 158, 256)),
    (1, [400], 100, 33, 2, (0, 290, 301, 399)),
    (128, [20000], 2, 0, 0, (19998, 19999)),      # a unit cut over the clusters
    (128, [20000], 2, 0, 0, (60, 9000)),
    (16, [9001], 8, 3000, 5, (2, 5996, 5999, 8998)),
    # keys that some rows of a unit see and others do not, alone
    (16, [333, 190], 11, 0, 0, (185,)),
    (16, [333, 190], 11, 70, 5, (113, 188)),
    (64, [257], 2, 100, 3, (156, 256)),
    (1, [400], 100, 33, 2, (290, 301, 399)),
    (16, [9001], 8, 3000, 0, (5996, 8998)),
    (16, [20000], 8, 0, 0, (19995,)),
])
@pytest.mark.parametrize("col", [7, 300, 570])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_infinite_columns_of_seen_keys(heads, lens, chunk, window, sinks, where, col, value):
    """Heads whose query has the one sign meet the key with a logit of +inf (all
    NaN), those of the other with -inf: a weight of 0, and 0 times infinity in
    that column of out alone (columns from 512 on are not part of out)."""
    x = ref.make(lens, [chunk] * len(lens), heads, seed=heads + chunk)
    g = torch.Generator(device="cuda").manual_seed(col)
    sign = torch.randint(0, 2, (x.q.shape[0], heads), generator=g, device="cuda") * 2 - 1
    x.q[:, :, col] = (x.q[:, :, col].abs() + 0.25) * sign
    for b in range(len(lens)):
        for s in where:
            _put(x, b, s, col, value)
    kinds = _check(x, window, sinks)
    if heads > 1:
        assert "row" in kinds and ("columns" if col < D_V else "number") in kinds


def test_nan_of_seen_keys_and_other_infinities_beside_it():
    x = ref.make([300, 130], [3, 3], 128, seed=71)
    _put(x, 0, 299, 3, math.nan)
    _put(x, 0, 298, 100, math.inf)
    _put(x, 0, 298, 400, -math.inf)
    _put(x, 1, 128, 500, math.inf)
    x.q[:, :, 500] = -x.q[:, :, 500].abs() - 0.25
    assert _check(x) >= {"row", "columns", "number"}


@pytest.mark.parametrize("heads,lens,chunk,window", [(128, [1, 5, 130], 1, 0), (16, [200], 6, 0), (128, [9000], 1, 0),
                                                     (16, [9000, 40], 3, 0), (16, [300], 6, 20)])
@pytest.mark.parametrize("col", [100, 575])
def test_rows_all_of_whose_logits_are_minus_infinity(heads, lens, chunk, window, col):
    """lse = -inf as the formula has it, and no softmax: out is NaN, unlike that
    of a row without keys."""
    x = ref.make(lens, [chunk] * len(lens), heads, seed=72)
    x.q[:, :, col] = x.q[:, :, col].abs() + 0.25
    x.q[-1, ::2, col] *= -1                       # these heads: +inf, so lse is NaN, too
    x.pages[:, col] = -math.inf
    if x.q.shape[0] > 1:
        x.seq[0] = -1
    _check(x, window)
    # and a single finite key is the whole softmax
    if window == 0:
        for b, n in enumerate(lens):
            _put(x, b, max(0, n - chunk), col, 1.0)
        x.q[-1, ::2, col] *= -1
        _check(x)


@pytest.mark.parametrize("heads,chunk,window,sinks", [(128, 2, 0, 0), (16, 7, 0, 0), (16, 7, 60, 3)])
def test_received_weights_beside_infinite_keys(heads, chunk, window, sinks):
    """A key that is met with a logit of -inf receives nothing, and the others
    what they would without it; a logit of +inf makes a row's weights NaN, on
    the keys that it sees alone."""
    x = ref.make([333, 190], [chunk, chunk], heads, seed=73)
    x.q[:, :, 9] = -x.q[:, :, 9].abs() - 0.25
    inf_keys = [(0, 331), (0, 290), (1, 188), (1, 1)]
    for b, s in inf_keys:
        _put(x, b, s, 9, math.inf)
    _, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V, window=window, sinks=sinks)
    start = torch.rand(2, x.S, device="cuda")
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=start.clone(), window=window, sinks=sinks)
    # cache_ref.received, its bound taken over the keys whose rows are finite
    want, adds, rel = start.double(), torch.zeros(2, x.S, dtype=torch.float64, device="cuda"), 0.0
    for t in range(x.q.shape[0]):
        b, k = int(x.seq[t]), ref.seen_keys(x, t, window, sinks)
        c, q, l = x.pages[x.rows_of(b, k)].double(), x.q[t].double(), lse[t].double()
        z = q @ c.T * SCALE
        want[b, k] += torch.exp(z - l[:, None]).sum(0)
        adds[b, k] += heads
        fin = torch.isfinite(c).all(1)
        big = z[:, fin].abs().max() + l.abs().max()
        rel = max(rel, float(64 * 2.0 ** -23 * SCALE * (q.abs() @ c[fin].abs().T).max() + 8 * 2.0 ** -23 * (1 + big)))
    assert bool(((mass.double() - want).abs() <= want * (rel + (adds + 1) * 2.0 ** -24)).all())
    for b, s in inf_keys:
        assert float(mass[b, s]) == float(start[b, s])
    # one head of the last row meets one of them with +inf
    x.q[-1, 0, 9] *= -1
    _, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V, window=window, sinks=sinks)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=start.clone(), window=window, sinks=sinks)
    seen = torch.zeros(2, x.S, dtype=torch.bool, device="cuda")
    seen[1, ref.seen_keys(x, x.q.shape[0] - 1, window, sinks)] = True
    assert bool(torch.isnan(lse[-1, 0])) and torch.equal(torch.isnan(mass), seen)
