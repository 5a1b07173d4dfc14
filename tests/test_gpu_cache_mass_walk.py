"""Received weights where the walk over the steps has far to go: rows of a
sequence that lie far apart among others', many sequences, sequences without
rows."""
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


def test_steps_that_no_row_has_part_in_may_take_seconds():
    """Each sequence has one row at each end of the batch, at its first tokens and
    at its last: between the two lie some ten million steps of a cluster
    that are passed over, for longer than a wait's limit of two seconds."""
    n, T, page, pages = 74, 5120, 65536, 16
    g = torch.Generator(device="cuda").manual_seed(80)
    i32 = dict(dtype=torch.int32, device="cuda")
    S = page * pages
    seq, pos = torch.full((T,), -1, **i32), torch.zeros(T, **i32)
    seq[:n] = seq[-n:] = torch.arange(n, **i32)
    pos[:n], pos[-n:] = 5, S - 1
    x = ref.Cache(torch.randn(T, 128, ref.D_QK, generator=g, device="cuda").bfloat16(),
                  torch.randn(page, ref.D_QK, generator=g, device="cuda").bfloat16(), page,
                  torch.zeros(n, pages, **i32), seq, pos, [S] * n)
    _, lse = dsa.mla_attn_paged(*x.args(), SCALE, D_V, window=10)
    mass = dsa.mla_attn_mass_paged(*x.args(), lse, SCALE, window=10)
    torch.cuda.synchronize()
    assert dsa.device_status() == 0
    # the rows' keys: 6 and 10 places of each sequence
    got = torch.cat([mass[:, :6], mass[:, -10:]], 1).double()
    assert int((mass != 0).sum()) == n * 16
    for b in range(n):
        for t, s, at in ((b, torch.arange(6), 0), (T - n + b, torch.arange(S - 10, S), 6)):
            s = s.cuda()
            c, q = x.pages[x.rows_of(b, s)].double(), x.q[t].double()
            z, l = q @ c.T * SCALE, lse[t].double()
            want = torch.exp(z - l[:, None]).sum(0)
            # as in cache_ref.received: the logits' error, and a rounding per addend
            rel = 64 * 2.0 ** -23 * SCALE * (q.abs() @ c.abs().T).max() + \
                8 * 2.0 ** -23 * (1 + z.abs().max() + l.abs().max())
            assert bool(((got[b, at:at + len(s)] - want).abs() <= want * (rel + 129 * 2.0 ** -24)).all())
