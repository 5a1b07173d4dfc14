"""Paged cache operators on more sequences than run at once: the plan of the
received weights between its own limits, and compaction in several waves."""
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


@pytest.mark.parametrize("n", [64, 65, 300, 1024, 1025])
@pytest.mark.parametrize("heads,window,sinks", [(128, 0, 0), (16, 50, 3)])
def test_received_weights_of_many_sequences(n, heads, window, sinks):
    """Planned by each CTA (64), by a kernel in shared memory (1024) and in global
    memory; every third sequence has no rows."""
    lens = [1 + (61 * i) % 400 for i in range(n)]
    x = ref.make(lens, [0 if i % 3 == 2 else min(1 + i % 2, lens[i]) for i in range(n)], heads, seed=90 + n)
    _, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V, window=window, sinks=sinks)
    start = torch.rand(n, x.S, device="cuda")
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, mass=start.clone(), window=window, sinks=sinks)
    want, tol = ref.received(x, lse, start, window=window, sinks=sinks)
    assert bool(((mass.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("n,keep", [(200, 60), (200, 1), (700, 90)])
def test_compaction_of_more_sequences_than_run_at_once(n, keep):
    lens = [1 + (37 * i) % 200 for i in range(n)]
    x = ref.make(lens, [1] * n, 1, 64, seed=91, extra_pages=1)
    g = torch.Generator(device="cuda").manual_seed(92)
    rows = torch.randint(-2 ** 15, 2 ** 15, (x.pages.shape[0], ref.D_QK), generator=g, device="cuda").short()
    keys = torch.randint(0, 256, (x.pages.shape[0], 128), generator=g, device="cuda").to(torch.uint8)
    mass = torch.rand(n, x.S, generator=g, device="cuda")
    idx, new = dsa.cache_evict_select(mass, torch.tensor(lens, dtype=torch.int32, device="cuda"), keep)
    assert new.tolist() == [min(v, keep) for v in lens]
    want_rows = ref.compact(rows.cpu(), 64, x.table.cpu(), idx.cpu(), new.cpu())
    want_keys = ref.compact(keys.cpu(), 64, x.table.cpu(), idx.cpu(), new.cpu())
    want_mass = torch.zeros_like(mass)
    for b in range(n):
        want_mass[b, :int(new[b])] = mass[b, idx[b, :int(new[b])].long()]
    rows = rows.view(torch.bfloat16)
    dsa.cache_compact_paged(rows, 64, x.table, idx, new, k_pages=keys, mass=mass)
    torch.cuda.synchronize()
    assert torch.equal(rows.view(torch.int16).cpu(), want_rows)
    assert torch.equal(keys.cpu(), want_keys)
    assert torch.equal(mass, want_mass)
