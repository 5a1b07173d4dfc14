"""Host-side checks of the paged cache operators (no GPU): what their entry
points refuse before any launch, and what the binding refuses."""
import ctypes

import pytest
import torch

import sparse_attention_20_b200 as dsa
from sparse_attention_20_b200 import build as dsa_build

FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced: checks fail first
ODD = ctypes.c_void_p(0x10004)
SC = ctypes.c_float(0.1)


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


ATTN = dict(q=FAKE, kv=FAKE, num_pages=8, page_size=64, bt=FAKE, n_seqs=2, max_pages=4, seq=FAKE, pos=FAKE, T=3,
            Hq=128, d_qk=576, d_v=512, window=0, sinks=0, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40)

BAD_ROWS = [(dict(q=None), -1), (dict(kv=None), -1), (dict(bt=None), -1), (dict(seq=None), -1), (dict(pos=None), -1),
            (dict(lse=None), -1), (dict(q=ODD), -1), (dict(kv=ODD), -1), (dict(lse=ODD), -1), (dict(T=0), -1),
            (dict(n_seqs=0), -1), (dict(max_pages=0), -1), (dict(num_pages=0), -1), (dict(page_size=32), -2),
            (dict(page_size=0), -2), (dict(num_pages=1 << 26), -2), (dict(Hq=0), -2), (dict(Hq=129), -2),
            (dict(T=1 << 25), -2), (dict(max_pages=1 << 25), -2), (dict(d_qk=512), -2), (dict(window=-1), -1), (dict(sinks=-1), -1),
            (dict(sinks=4), -1)]


@pytest.mark.parametrize("change,code", BAD_ROWS + [(dict(out=None), -1), (dict(out=ODD), -1), (dict(d_v=576), -2),
                                                    (dict(T=1 << 20, Hq=1, max_pages=1 << 24), -2)])
def test_attention_refuses(lib, change, code):
    a = {**ATTN, **change}
    before = dsa.launch_count()
    rc = lib.dsa_mla_attn_paged(a["q"], a["kv"], a["num_pages"], a["page_size"], a["bt"], a["n_seqs"],
                                a["max_pages"], a["seq"], a["pos"], a["T"], a["Hq"], a["d_qk"], a["d_v"], SC,
                                a["window"], a["sinks"], a["out"], a["lse"], a["ws"],
                                ctypes.c_size_t(a["ws_bytes"]), None)
    assert rc == code and lib.dsa_last_error() and dsa.launch_count() == before


@pytest.mark.parametrize("change,code", BAD_ROWS + [(dict(mass=None), -1), (dict(mass=ODD), -1),
                                                    (dict(ws=None), -5), (dict(ws=ODD), -5), (dict(ws_bytes=64), -5)])
def test_weights_refuse(lib, change, code):
    a = {**ATTN, "mass": FAKE, **change}
    before = dsa.launch_count()
    rc = lib.dsa_mla_attn_mass_paged(a["q"], a["kv"], a["num_pages"], a["page_size"], a["bt"], a["n_seqs"],
                                     a["max_pages"], a["seq"], a["pos"], a["lse"], a["T"], a["Hq"], a["d_qk"], SC,
                                     a["window"], a["sinks"], a["mass"], a["ws"], ctypes.c_size_t(a["ws_bytes"]), None)
    assert rc == code and lib.dsa_last_error() and dsa.launch_count() == before


@pytest.mark.parametrize("change,code", [
    (dict(mass=None), -1), (dict(seq_len=None), -1), (dict(idx=None), -1), (dict(new_len=None), -1),
    (dict(mass=ODD), -1), (dict(n_seqs=0), -1), (dict(max_len=0), -1), (dict(keep=0), -1), (dict(sinks=-1), -1),
    (dict(recent=-1), -1), (dict(sinks=60, recent=41), -1), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), -1),
    (dict(max_len=(1 << 30) + 1), -2), (dict(keep=(1 << 30) + 1), -2)])
def test_select_refuses(lib, change, code):
    a = {**dict(mass=FAKE, max_len=1000, seq_len=FAKE, n_seqs=2, keep=100, sinks=4, recent=8, idx=FAKE,
                new_len=FAKE), **change}
    before = dsa.launch_count()
    rc = lib.dsa_cache_evict_select(a["mass"], a["max_len"], a["seq_len"], a["n_seqs"], a["keep"], a["sinks"],
                                    a["recent"], a["idx"], a["new_len"], None)
    assert rc == code and lib.dsa_last_error() and dsa.launch_count() == before


@pytest.mark.parametrize("change,code", [
    (dict(kv=None), -1), (dict(bt=None), -1), (dict(idx=None), -1), (dict(new_len=None), -1), (dict(kv=ODD), -1),
    (dict(k=ODD), -1), (dict(mass=ODD), -1), (dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(n_seqs=0), -1),
    (dict(max_pages=0), -1), (dict(keep=0), -1), (dict(num_pages=1 << 27), -2), (dict(kv_bytes=24), -2),
    (dict(kv_bytes=0), -2), (dict(kv_bytes=4112), -2), (dict(k_bytes=8), -2)])
def test_compaction_refuses(lib, change, code):
    a = {**dict(kv=FAKE, kv_bytes=1152, k=FAKE, k_bytes=128, num_pages=8, page_size=64, bt=FAKE, n_seqs=2,
                max_pages=4, idx=FAKE, keep=100, new_len=FAKE, mass=FAKE), **change}
    before = dsa.launch_count()
    rc = lib.dsa_cache_compact_paged(a["kv"], a["kv_bytes"], a["k"], a["k_bytes"], a["num_pages"], a["page_size"],
                                     a["bt"], a["n_seqs"], a["max_pages"], a["idx"], a["keep"], a["new_len"],
                                     a["mass"], None)
    assert rc == code and lib.dsa_last_error() and dsa.launch_count() == before


def test_attention_workspace(lib):
    f = lib.dsa_mla_attn_paged_workspace_size
    assert f(0, 128) == 0 and f(4, 0) == 0
    # the same for one row and for many, but for a few bytes a row
    assert f(4096, 128) - f(1, 128) <= 4096 * 64
    need = f(3, 128)
    if need:
        a = ATTN
        for ws, n in ((FAKE, need - 1), (None, need), (ODD, need)):
            assert lib.dsa_mla_attn_paged(a["q"], a["kv"], 8, 64, a["bt"], 2, 4, a["seq"], a["pos"], 3, 128, 576, 512,
                                          SC, 0, 0, a["out"], a["lse"], ws, ctypes.c_size_t(n), None) == -5


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 128, 576, dtype=torch.bfloat16)
    kv = torch.zeros(64, 576, dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.mla_attn_paged(q, kv, 64, one.view(1, 1), one, one, 0.1, 512)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.mla_attn_mass_paged(q, kv, 64, one.view(1, 1), one, one, torch.zeros(1, 128), 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.cache_evict_select(torch.zeros(1, 64), one, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.cache_compact_paged(kv, 64, one.view(1, 1), one.view(1, 1), one)
