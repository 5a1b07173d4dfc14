"""Dense and windowed attention of new tokens over the paged latent cache, and
the weight each cached token receives, against 64-bit references."""
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


def _attn(x, scale=SCALE, window=0, sinks=0, **kw):
    out, lse = dsa.mla_attn_paged(*x.args(), scale, D_V, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    assert dsa.device_status() == 0
    return out, lse


CASES = [
    # lens, chunks, heads, page, window, sinks
    ([1], [1], 128, 64, 0, 0),
    ([2, 1, 3], [2, 1, 3], 128, 64, 0, 0),
    ([63, 64, 65, 127, 128, 129], [1] * 6, 128, 64, 0, 0),
    ([300, 1, 513], [5, 1, 9], 128, 128, 0, 0),
    ([257, 190], [33, 7], 64, 192, 0, 0),
    ([700], [40], 16, 64, 0, 0),
    ([130, 77], [3, 11], 48, 64, 0, 0),
    ([333], [9], 1, 256, 0, 0),
    ([200, 140], [6, 2], 5, 64, 0, 0),
    ([1000, 400, 33], [1, 4, 2], 128, 64, 100, 0),
    ([1000, 400, 33], [1, 4, 2], 128, 64, 100, 3),
    ([1000, 650], [70, 130], 16, 64, 129, 65),
    ([900], [4], 128, 128, 1, 1),
    ([900], [4], 128, 128, 1, 0),
    ([500, 200], [8, 8], 32, 64, 128, 128),
    ([500, 200], [3, 3], 128, 64, 4000, 16),     # window longer than the cache
    ([400], [3], 128, 64, 64, 1000),             # more first tokens than the cache holds
    ([1], [1], 1, 64, 0, 0),                     # a query of one row in all
    ([260, 129], [2, 3], 100, 64, 0, 0),         # 28 of a unit's 128 places unused
    ([700], [5], 127, 192, 90, 2),
    ([400, 300], [50, 45], 3, 64, 0, 0),         # 42 rows a unit, the runs' ends inside units
]


@pytest.mark.parametrize("lens,chunks,heads,page,window,sinks", CASES)
def test_attention_matches_fp64(lens, chunks, heads, page, window, sinks):
    x = ref.make(lens, chunks, heads, page, seed=len(lens) + heads)
    out, lse = _attn(x, window=window, sinks=sinks)
    ref.check_attention(x, out, lse, window=window, sinks=sinks)


@pytest.mark.parametrize("n,chunk,window", [(20000, 1, 0), (9001, 2, 0), (30011, 3, 5000)])
def test_long_rows_split_over_the_gpu(n, chunk, window):
    x = ref.make([n], [chunk], 128, seed=3)
    out, lse = _attn(x, window=window, sinks=7 if window else 0)
    ref.check_attention(x, out, lse, window=window, sinks=7 if window else 0)
    again = _attn(x, window=window, sinks=7 if window else 0)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])   # the parts join in a fixed order


def test_many_rows_of_unequal_length():
    lens = [1 + (977 * i) % 1500 for i in range(180)]
    x = ref.make(lens, [1] * 180, 128, seed=5)
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)


def test_more_rows_than_the_plan_has_threads():
    """Units of one row and of eight; runs that end anywhere; padding in between."""
    lens = [20 + (37 * i) % 300 for i in range(100)]
    x = ref.make(lens, [1 + i % 13 for i in range(100)], 128, seed=50)
    x.seq[::17] = -1
    assert x.q.shape[0] > 512
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)
    y = ref.make([900, 500, 40], [700, 333, 40], 16, seed=51)
    out, lse = _attn(y, window=200, sinks=5)
    ref.check_attention(y, out, lse, window=200, sinks=5)


@pytest.mark.parametrize("heads,lens,chunks,pads", [
    (128, [364, 370, 386], [86, 86, 86], (0, 0, 0, 5)),
    (128, [100, 120], [40, 30], (9, 70, 33)),          # before, between and behind the sequences
    (16, [300, 200], [20, 50], (40, 100, 300)),
    (128, [50], [1], (0, 700)),
    (128, [50], [1], (700, 0)),
    (64, [9], [1], (0, 3)),
])
def test_stretches_of_padding(heads, lens, chunks, pads):
    x = ref.make(lens, chunks, heads, seed=57)
    seq, pos, at = [], [], 0
    for b, c in enumerate(chunks + [0]):
        seq += [-1] * pads[b] + x.seq[at:at + c].tolist()
        pos += [-1] * pads[b] + x.pos[at:at + c].tolist()
        at += c
    g = torch.Generator(device="cuda").manual_seed(58)
    x.seq = torch.tensor(seq, dtype=torch.int32, device="cuda")
    x.pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    x.q = torch.randn(len(seq), heads, ref.D_QK, generator=g, device="cuda").bfloat16()
    out = torch.full((len(seq), heads, D_V), 5.0, dtype=torch.bfloat16, device="cuda")
    got = _attn(x, out=out)
    ref.check_attention(x, *got)
    mass = dsa.mla_attn_mass_paged(*x.args(), got[1], SCALE)
    want, tol = ref.received(x, got[1], torch.zeros_like(mass))
    assert bool(((mass.double() - want).abs() <= tol).all())


def test_only_padding():
    x = ref.make([64], [1], 128, seed=59)
    x.seq = torch.full((600,), -1, dtype=torch.int32, device="cuda")
    x.pos = torch.zeros(600, dtype=torch.int32, device="cuda")
    x.q = torch.zeros(600, 128, ref.D_QK, dtype=torch.bfloat16, device="cuda")
    out, lse = _attn(x)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    mass = torch.rand(1, x.S, device="cuda")
    start = mass.clone()
    dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=mass)
    assert torch.equal(mass, start)


@pytest.mark.parametrize("lens", [[1000] * 40, [1000] * 39 + [1500], [1000] * 39 + [6000], [64] * 74, [64] * 75])
def test_units_whole_or_cut(lens):
    """As many even units as clusters, one longer than the others, and one more."""
    x = ref.make(lens, [1] * len(lens), 128, seed=52)
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)


def test_outputs_on_any_16_byte_boundary():
    x = ref.make([500], [3], 128, seed=53)
    buf = torch.empty(3 * 128 * D_V + 8, dtype=torch.bfloat16, device="cuda")
    at = 8 if (buf.data_ptr() % 32) == 0 else 0
    out = buf[at:at + 3 * 128 * D_V].view(3, 128, D_V)
    assert out.data_ptr() % 32 == 16
    got = _attn(x, out=out)
    ref.check_attention(x, *got)


def test_workspace_may_hold_anything():
    x = ref.make([9000, 7000], [1, 1], 128, seed=54)
    ws = dsa.alloc_mla_attn_workspace(2, 128)
    want = _attn(x)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got = _attn(x, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_one_stream_after_another_kernel_of_the_library():
    """Calls back to back on one stream, each reading what the one before wrote:
    the next call's positions, then its queries from this call's output."""
    x = ref.make([3000, 2000], [1, 1], 128, seed=55)
    ws, mws = dsa.alloc_mla_attn_workspace(2, 128), dsa.alloc_mla_mass_workspace(2)
    outs, masses = [], []
    mass = torch.zeros(2, x.S, device="cuda")
    for i in range(6):
        out, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V, workspace=ws)
        dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=mass, workspace=mws)
        outs.append((out, lse, x.q.clone(), x.pos.clone()))
        masses.append(mass.clone())
        x.q[:, :, :D_V] = out
        x.pos -= 7
    torch.cuda.synchronize()
    start = torch.zeros_like(mass)
    for (out, lse, q, pos), m in zip(outs, masses):
        x.q, x.pos = q, pos
        ref.check_attention(x, out, lse)
        want, tol = ref.received(x, lse, start)
        assert bool(((m.double() - want).abs() <= tol + 2.0 ** -23 * want).all())
        start = m


def test_rows_without_keys_and_rows_beyond_the_table():
    x = ref.make([200, 100, 50], [2, 3, 1], 64, seed=6)
    x.seq[1] = -1
    x.seq[3] = 3
    x.pos[0] = -1
    x.pos[4] = 100000          # past the table: every key of the sequence
    out = torch.full((6, 64, D_V), 7.0, dtype=torch.bfloat16, device="cuda")
    got = _attn(x, out=out)
    ref.check_attention(x, *got)
    assert bool((got[0][[0, 1, 3]] == 0).all())
    # the window behind such a position holds no key: only the first tokens are left
    got = _attn(x, window=10, sinks=4)
    ref.check_attention(x, *got, window=10, sinks=4)
    got = _attn(x, window=10)
    ref.check_attention(x, *got, window=10)
    assert bool(torch.isinf(got[1][4]).all())


def test_rows_in_any_order():
    x = ref.make([300, 150, 77, 410], [9, 12, 1, 30], 16, seed=7)
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(52, generator=g).cuda()
    order = torch.cat([order, order[:5]])       # some tokens twice
    x.q, x.seq, x.pos = x.q[order].contiguous(), x.seq[order].contiguous(), x.pos[order].contiguous()
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)
    out, lse = _attn(x, window=33, sinks=2)
    ref.check_attention(x, out, lse, window=33, sinks=2)


@pytest.mark.parametrize("heads,chunk,window,sinks", [(128, 1, 0, 0), (128, 3, 70, 5), (16, 11, 0, 0),
                                                      (16, 11, 70, 5), (64, 2, 200, 0)])
@pytest.mark.parametrize("junk", [math.nan, math.inf])
def test_masked_places_may_hold_anything(heads, chunk, window, sinks, junk):
    """Every pool row that no query row of its sequence sees is NaN or infinite,
    and so are the first and last keys that only some rows see: the rows that
    do not see them stay exact."""
    x = ref.make([333, 190], [chunk, chunk], heads, seed=8)
    clean = x.pages.clone()
    used = torch.zeros(x.pages.shape[0], dtype=torch.bool, device="cuda")
    for t in range(x.q.shape[0]):
        used[x.rows_of(int(x.seq[t]), ref.seen_keys(x, t, window, sinks))] = True
    x.pages[~used] = junk
    out, lse = _attn(x, window=window, sinks=sinks)
    ref.check_attention(x, out, lse, window=window, sinks=sinks)
    # the newest token's key is seen by the last row of each sequence alone
    x.pages.copy_(clean)
    for b in range(2):
        x.pages[x.rows_of(b, torch.tensor([x.lens[b] - 1], device="cuda"))] = math.nan
    out, lse = _attn(x, window=window, sinks=sinks)
    last = x.pos == torch.tensor(x.lens, device="cuda", dtype=torch.int32)[x.seq.long()] - 1
    assert bool(torch.isnan(out[last]).all()) and bool(torch.isnan(lse[last]).all())
    if chunk > 1:
        x.pages.copy_(clean)
        ref_o, ref_l, tol_o, tol_l = ref.attention(x, SCALE, window, sinks)
        assert bool(((out.double() - ref_o).abs() <= tol_o)[~last].all())
        assert bool(((lse.double() - ref_l).abs() <= tol_l)[~last].all())


def test_bad_block_table_entries_stay_inside_the_pool():
    x = ref.make([300, 200], [1, 1], 128, seed=9)
    x.table[0, 1] = 10 ** 6
    x.table[1, 2] = -5
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)        # the reference reads page 0 there


@pytest.mark.parametrize("order", ["rising", "falling", "large"])
def test_maximum_that_moves(order):
    """Logits that rise along the keys (every tile raises the running maximum),
    fall, or reach hundreds."""
    x = ref.make([1500], [3], 128, seed=10, kv_scale=8.0 if order == "large" else 1.0)
    if order != "large":
        s = torch.arange(1500, device="cuda")
        gain = (s if order == "rising" else 1499 - s).double() / 1500
        rows = x.rows_of(0, s)
        x.pages[rows] = (x.pages[rows].double() * 0.1 + 12 * gain[:, None] * x.q[1, 5].double()).bfloat16()
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales(scale):
    x = ref.make([400], [2], 128, seed=11)
    out, lse = _attn(x, scale=scale)
    ref.check_attention(x, out, lse, scale=scale)


def test_agrees_with_sparse_attention_over_every_key():
    x = ref.make([500, 64, 200], [1, 1, 1], 128, seed=12)
    out, lse = _attn(x)
    idx = torch.arange(512, dtype=torch.int32, device="cuda").expand(3, 512).contiguous()
    idx = torch.where(idx <= x.pos[:, None], idx, -1)
    o2, l2 = dsa.sparse_mla_attn_paged(x.q, x.pages, x.page_size, x.table, x.seq, x.pos, idx, SCALE, D_V)
    torch.cuda.synchronize()
    # the sparse kernel exchanges half of each logit in fp16: its lse is within 1e-3 (tests/parity.py)
    assert bool(((lse - l2).abs() <= 1e-3 + 1e-4).all())
    # both are within 1e-2 of the exact result (rel-L2), hence 2e-2 of each other
    assert float((out.double() - o2.double()).norm() / o2.double().norm()) <= 2e-2


def test_captured_and_replayed_on_new_inputs_and_two_at_once():
    xs = [ref.make([900, 3000], [2, 2], 128, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in xs]
    graphs, outs = [], []
    for x, st in zip(xs, streams):
        ws = dsa.alloc_mla_attn_workspace(4, 128)
        _attn(x, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            o = dsa.mla_attn_paged(*x.args(), SCALE, D_V, window=700, sinks=3, workspace=ws)
        graphs.append(g)
        outs.append((o, ws))
    for rep in range(3):
        for x in xs:
            x.q.copy_(torch.randn_like(x.q, dtype=torch.float32).bfloat16())
            x.pos -= 1
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for x, (o, _) in zip(xs, outs):
            ref.check_attention(x, *o, window=700, sinks=3)


def test_another_stream_without_buffers_of_ones_own():
    x = ref.make([2000, 700], [1, 1], 128, seed=22)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [dsa.mla_attn_paged(*x.args(), SCALE, D_V, stream=st) for _ in range(4)]
    torch.cuda.synchronize()
    for o in got:
        ref.check_attention(x, *o)


def test_binding_refuses():
    x = ref.make([200], [2], 128, seed=56)
    for kw in (dict(window=2 ** 32 + 5), dict(window=8, sinks=2 ** 40)):
        with pytest.raises(ValueError, match="32 bits"):
            dsa.mla_attn_paged(*x.args(), SCALE, D_V, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        dsa.mla_attn_paged(x.q.transpose(0, 1).contiguous().transpose(0, 1), *x.args()[1:], SCALE, D_V)
    with pytest.raises(TypeError, match="bfloat16"):
        dsa.mla_attn_paged(x.q.half(), *x.args()[1:], SCALE, D_V)
    with pytest.raises(ValueError, match="whole number"):
        dsa.mla_attn_paged(x.q, x.pages[:-1].contiguous(), *x.args()[2:], SCALE, D_V)
    with pytest.raises(ValueError, match="shape"):
        dsa.mla_attn_paged(*x.args()[:4], x.seq[:1].contiguous(), x.pos, SCALE, D_V)
    with pytest.raises(ValueError, match="shape"):
        dsa.mla_attn_paged(*x.args(), SCALE, D_V, out=torch.empty(2, 64, D_V, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dsa.DSAError, match="workspace"):
        dsa.mla_attn_paged(*x.args(), SCALE, D_V, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dsa.DSAError, match="window"):
        dsa.mla_attn_paged(*x.args(), SCALE, D_V, sinks=4)
    lse = torch.zeros(2, 128, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=torch.zeros(1, 8, device="cuda"))
    with pytest.raises(ValueError, match="32 bits"):
        dsa.cache_evict_select(torch.zeros(1, 64, device="cuda"), x.seq[:1].contiguous(), 8, recent=2 ** 31)
    assert dsa.device_status() == 0


def test_pool_offsets_beyond_32_bits():
    """A pool of 2^31 + elements: the sequence's pages lie at its end."""
    page = 256
    num = (2 ** 31 // (ref.D_QK * page)) + 40
    x = ref.make([2000], [2], 128, page, seed=23)
    big = torch.zeros(num * page, ref.D_QK, dtype=torch.bfloat16, device="cuda")
    big[-x.pages.shape[0]:] = x.pages
    x.table += num - x.pages.shape[0] // page
    x.pages = big
    out, lse = _attn(x)
    ref.check_attention(x, out, lse)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE)
    want, tol = ref.received(x, lse, torch.zeros_like(mass))
    assert bool(((mass.double() - want).abs() <= tol).all())


# ------------------------------------------------------------- weights

@pytest.mark.parametrize("lens,chunks,heads,page,window,sinks", CASES)
def test_received_weights_match_fp64(lens, chunks, heads, page, window, sinks):
    x = ref.make(lens, chunks, heads, page, seed=40 + heads)
    _, lse = _attn(x, window=window, sinks=sinks)
    start = torch.rand(len(lens), x.S, device="cuda")
    mass = start.clone()
    got = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=mass, window=window, sinks=sinks)
    assert got.data_ptr() == mass.data_ptr()
    want, tol = ref.received(x, lse, start, window=window, sinks=sinks)
    assert bool(((mass.double() - want).abs() <= tol).all())
    unseen = want == start.double()
    assert torch.equal(mass[unseen], start[unseen])
    again = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=start.clone(), window=window, sinks=sinks)
    assert torch.equal(again, mass)          # one thread adds to an element, in the rows' order


def test_weights_of_rows_in_any_order_and_rows_without_keys():
    x = ref.make([300, 150, 77, 410], [9, 12, 1, 30], 16, seed=41)
    g = torch.Generator().manual_seed(2)
    order = torch.randperm(52, generator=g).cuda()
    order = torch.cat([order, order[:5]])
    x.q, x.seq, x.pos = x.q[order].contiguous(), x.seq[order].contiguous(), x.pos[order].contiguous()
    x.seq[3], x.seq[10], x.pos[20], x.pos[30] = -1, 9, -2, 100000
    _, lse = _attn(x)
    lse[7] = -math.inf
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE)
    want, tol = ref.received(x, lse, torch.zeros_like(mass))
    assert bool(((mass.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("heads,chunk,window,sinks", [(128, 2, 0, 0), (16, 5, 60, 3)])
def test_weights_ignore_what_masked_places_hold(heads, chunk, window, sinks):
    x = ref.make([333, 190], [chunk, chunk], heads, seed=42)
    used = torch.zeros(x.pages.shape[0], dtype=torch.bool, device="cuda")
    for t in range(x.q.shape[0]):
        used[x.rows_of(int(x.seq[t]), ref.seen_keys(x, t, window, sinks))] = True
    x.pages[~used] = math.nan
    _, lse = _attn(x, window=window, sinks=sinks)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, window=window, sinks=sinks)
    want, tol = ref.received(x, lse, torch.zeros_like(mass), window=window, sinks=sinks)
    assert bool(((mass.double() - want).abs() <= tol).all())


def test_weights_of_each_row_and_head_sum_to_one():
    x = ref.make([700, 20], [12, 20], 128, seed=43)
    _, lse = _attn(x)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE)
    total = mass.double().sum(1).cpu()
    # a row's 128 heads give 128: each weight is within 1e-4 relative (ref.received's bound at these sizes)
    assert abs(total[0] - 12 * 128) <= 12 * 128 * 1e-4 and abs(total[1] - 20 * 128) <= 20 * 128 * 1e-4


def test_weights_of_many_sequences_and_many_rows():
    """More sequences than the plan holds in shared memory, most without rows;
    more rows than it has threads."""
    lens = [70 + (31 * i) % 200 for i in range(1100)]
    x = ref.make(lens, [1 if i % 3 == 0 else 0 for i in range(1100)], 128, seed=45)
    _, lse = _attn(x)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE)
    want, tol = ref.received(x, lse, torch.zeros_like(mass))
    assert bool(((mass.double() - want).abs() <= tol).all())
    y = ref.make([1500, 700], [1100, 300], 8, seed=46)
    _, lse = _attn(y)
    mass = dsa.mla_attn_mass_paged(*y.args(), lse, SCALE)
    want, tol = ref.received(y, lse, torch.zeros_like(mass))
    assert bool(((mass.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("heads,window,sinks", [(128, 40, 0), (128, 40, 3), (8, 300, 300), (100, 40, 700)])
def test_weights_where_most_rows_miss_most_tiles(heads, window, sinks):
    """A long chunk behind a short window: tiles that only some rows see, parts
    of tiles that no row of a cluster's share sees."""
    x = ref.make([2600, 1400], [900, 700], heads, seed=47)
    _, lse = _attn(x, window=window, sinks=sinks)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, window=window, sinks=sinks)
    want, tol = ref.received(x, lse, torch.zeros_like(mass), window=window, sinks=sinks)
    assert bool(((mass.double() - want).abs() <= tol).all())
    again = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, window=window, sinks=sinks)
    assert torch.equal(again, mass)


def test_weights_captured_and_replayed():
    x = ref.make([900, 300], [1, 1], 128, seed=44)
    _, lse = _attn(x)
    mass = torch.zeros(2, x.S, device="cuda")
    dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=mass)
    mass.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=mass)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    one, tol = ref.received(x, lse, torch.zeros_like(mass))
    assert bool(((mass.double() - 3 * one).abs() <= 3 * tol + 3 * 2.0 ** -24 * mass).all())
