"""Host-side checks of the decoding operators (paged attention, beam selection, forks of states and pages): every
bad argument is refused before any CUDA call, so these run without a GPU.  The addresses below are never
dereferenced."""

import ctypes
import os
import shutil

import pytest
import torch

import kda_gated_delta_03_gb300 as kda
from kda_gated_delta_03_gb300 import binding, build

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
OK, INV, UNS, WS, TOO_LARGE = (binding.KDA_OK, binding.KDA_ERR_INVALID_ARG, binding.KDA_ERR_UNSUPPORTED,
                               binding.KDA_ERR_WORKSPACE, binding.KDA_ERR_TOO_LARGE)
P, P2, ODD8, ODD2 = 0x10000, 0x20000, 0x10008, 0x10002


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def attention(lib, **over):
    a = dict(q=P, k=P, v=P, table=P, lens=P, kn=P, vn=P, B=2, Hq=8, Hkv=2, d=64, pages=10, ps=16, M=4, ks=2048, vs=2048,
             dt=1, scale=1.0, window=0, sinks=0, o=P, lse=None, ws=P, wsb=1 << 40, stream=None)
    a.update(over)
    return lib.kda_attention_decode(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(Hq=9), INV), (dict(d=0), INV), (dict(pages=-1), INV),
    (dict(ps=0), INV), (dict(M=-1), INV), (dict(window=-1), INV), (dict(sinks=-2), INV), (dict(scale=float("inf")), INV),
    (dict(dt=2), INV), (dict(d=32), UNS), (dict(d=256), UNS), (dict(q=None), INV), (dict(q=ODD8), INV), (dict(o=None), INV),
    (dict(k=None), INV), (dict(v=ODD8), INV), (dict(table=None), INV), (dict(lens=ODD2), INV), (dict(lse=ODD2), INV),
    (dict(kn=None), INV), (dict(vn=None), INV), (dict(kn=ODD8), INV), (dict(pages=0), INV), (dict(ks=2047), INV),
    (dict(ks=1024), INV), (dict(vs=2040, ks=2040), INV), (dict(M=1 << 28, ps=16), INV), (dict(B=0), OK),
])
def test_attention_refuses(lib, over, code):
    assert attention(lib, **over) == code


def test_attention_longest_table(lib):
    """A tile past the longest length still has to be a 32-bit number."""
    last = 2 ** 31 - 1024
    assert attention(lib, M=1, pages=1, ps=last, ws=None) == WS            # every other argument is accepted
    assert attention(lib, M=1, pages=1, ps=last + 1, ws=None) == INV


def test_attention_most_rows_and_heads(lib):
    """Rows past the last one, as a thread steps over them, and a row's outputs still have to be 32-bit numbers."""
    last = 2 ** 31 - 1024
    assert attention(lib, B=last, ws=None) == WS                           # every other argument is accepted
    assert attention(lib, B=last + 1, ws=None) == INV
    assert attention(lib, B=2 ** 31 - 1, ws=None) == INV
    assert attention(lib, Hq=2 ** 25 - 2, ws=None) == WS
    assert attention(lib, Hq=2 ** 25, ws=None) == INV


def test_attention_workspace(lib):
    assert lib.kda_attention_decode_workspace_size(0, 8, 2, 64, 1) == 0
    assert lib.kda_attention_decode_workspace_size(2, 9, 2, 64, 1) == 0
    need = lib.kda_attention_decode_workspace_size(2, 8, 2, 64, 1)
    assert need % 256 == 0
    if need:
        assert attention(lib, ws=None) == WS and attention(lib, wsb=need - 1) == WS and attention(lib, ws=0x10010) == WS


def select(lib, **over):
    a = dict(logits=P, stride=100, bs=P, fin=None, eos=-1, N=2, K=4, V=100, dt=1, scores=P, parent=P, token=P, fout=None,
             ws=P, wsb=1 << 40, stream=None)
    a.update(over)
    return lib.kda_beam_select(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(N=-1), INV), (dict(K=0), INV), (dict(V=0), INV), (dict(dt=9), INV), (dict(stride=99), INV), (dict(eos=100), INV),
    (dict(eos=-2), INV), (dict(fin=P), INV), (dict(K=33), UNS), (dict(K=32, V=1 << 27, stride=1 << 27), TOO_LARGE),
    (dict(N=1 << 30), TOO_LARGE), (dict(logits=None), INV), (dict(logits=0x10001), INV), (dict(bs=None), INV),
    (dict(scores=None), INV), (dict(scores=ODD2), INV), (dict(parent=None), INV), (dict(token=ODD2), INV), (dict(N=0), OK),
])
def test_select_refuses(lib, over, code):
    assert select(lib, **over) == code


def test_select_workspace(lib):
    assert lib.kda_beam_select_workspace_size(2, 33, 100, 1) == 0
    need = lib.kda_beam_select_workspace_size(2, 4, 100000, 1)
    if need:
        assert select(lib, V=100000, stride=100000, wsb=need - 1) == WS


def test_select_longest_row(lib):
    """A chunk past a row's end still has to be a 32-bit number."""
    last = 2 ** 31 - 2 ** 14
    for dt in (0, 1):
        assert 0 < lib.kda_beam_select_workspace_size(1, 1, last, dt) <= 1 << 14
        assert lib.kda_beam_select_workspace_size(1, 1, last + 1, dt) == 0
        assert lib.kda_beam_select_workspace_size(1, 1, 2 ** 31 - 1, dt) == 0
        assert select(lib, N=1, K=1, V=last, stride=last, dt=dt, ws=None) == WS       # every other argument is accepted
        assert select(lib, N=1, K=1, V=last + 1, stride=last + 1, dt=dt) == TOO_LARGE
        assert select(lib, N=1, K=1, V=2 ** 31 - 1, stride=2 ** 31 - 1, dt=dt) == TOO_LARGE


def pool(**over):
    p = dict(data=P, layer_stride=0, slot_stride=64, slot_bytes=64, layers=1, slots=10)
    p.update(over)
    return binding.Pool(**p)


BAD_POOLS = [dict(data=None), dict(data=ODD8), dict(layers=-1), dict(slots=-1), dict(slot_bytes=-16), dict(slot_bytes=40),
             dict(slot_stride=72), dict(layer_stride=8), dict(slot_stride=48), dict(slot_stride=-64)]


@pytest.mark.parametrize("bad", BAD_POOLS)
def test_pools_are_checked(lib, bad):
    arr = (binding.Pool * 2)(pool(), pool(**bad))
    assert lib.kda_copy_pages(arr, 2, P, P2, 3, None) == INV
    assert lib.kda_state_fork(arr, 2, P, P, 3, P2, None) == INV
    assert lib.kda_cache_fork(P, P, 2, P, None, 2, 4, 16, P, 10, P2, P2, P, None, None, arr, 2, P, 1 << 40, None) == INV
    assert lib.kda_cache_compact(P, 2, 4, P, 10, P2, P2, 0x30000, arr, 2, P, 1 << 40, None) == INV


def test_slots_and_rows_are_checked(lib):
    arr = (binding.Pool * 9)(*[pool() for _ in range(9)])
    assert lib.kda_copy_pages(arr, 9, P, P2, 3, None) == UNS
    assert lib.kda_copy_pages(None, 1, P, P2, 3, None) == INV
    assert lib.kda_copy_pages(arr, 1, P, None, 3, None) == INV
    assert lib.kda_copy_pages(arr, 1, ODD2, P2, 3, None) == INV
    assert lib.kda_copy_pages(arr, 1, P, P2, -1, None) == INV
    assert lib.kda_copy_pages(arr, 1, P, P2, 0, None) == OK
    assert lib.kda_state_fork(arr, 1, P, P, 8193, P2, None) == TOO_LARGE
    assert lib.kda_state_fork(arr, 1, P, P, -1, P2, None) == INV
    assert lib.kda_state_fork(arr, 1, None, P, 4, P2, None) == INV
    assert lib.kda_state_fork(arr, 1, P, P2, 4, P, None) == INV          # in place
    assert lib.kda_state_fork(arr, 1, P, P2, 4, P2, None) == INV
    assert lib.kda_state_fork(arr, 1, P, P, 0, P2, None) == OK


def fork(lib, **over):
    a = dict(table=P, lens=P, R=2, parent=P, grow=None, R2=2, M=4, ps=16, ref=P, pages=10, tout=P2, lout=P2, rout=P, cs=None,
             cd=None, pools=None, n=0, ws=P, wsb=1 << 40, stream=None)
    a.update(over)
    return lib.kda_cache_fork(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INV), (dict(R2=-1), INV), (dict(M=-1), INV), (dict(ps=0), INV), (dict(pages=-1), INV),
    (dict(M=1 << 28, ps=16), INV), (dict(R2=1 << 30), INV), (dict(parent=None), INV), (dict(grow=ODD2), INV),
    (dict(lout=None), INV), (dict(tout=None), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(ref=None), INV),
    (dict(rout=None), INV), (dict(cs=P), INV), (dict(cs=P, cd=ODD2), INV), (dict(tout=P), INV), (dict(lout=P), INV),
    (dict(n=-1), INV), (dict(ws=None), WS), (dict(wsb=100), WS), (dict(ws=0x10010), WS), (dict(R=0, R2=0), OK),
    (dict(R=8193), TOO_LARGE), (dict(R2=8193), TOO_LARGE),
])
def test_cache_fork_refuses(lib, over, code):
    assert fork(lib, **over) == code


def test_cache_fork_takes_only_pools_of_its_pages(lib):
    arr = (binding.Pool * 1)(pool(slots=11))
    assert fork(lib, pools=arr, n=1) == INV


def compact(lib, **over):
    a = dict(table=P, R=2, M=4, ref=P, pages=10, tout=P, rout=P, map=P2, pools=None, n=0, ws=P, wsb=1 << 40, stream=None)
    a.update(over)
    return lib.kda_cache_compact(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INV), (dict(M=-1), INV), (dict(pages=-1), INV), (dict(R=1 << 30), INV), (dict(table=None), INV),
    (dict(tout=ODD2), INV), (dict(ref=None), INV), (dict(rout=None), INV), (dict(map=None), INV), (dict(map=P), INV),
    (dict(ws=None), WS), (dict(wsb=64), WS), (dict(R=0, pages=0), OK),
])
def test_cache_compact_refuses(lib, over, code):
    assert compact(lib, **over) == code


def test_most_pages(lib):
    """Pages past the last one, as a thread steps over them, still have to be 32-bit numbers."""
    pages, row = 2 ** 31 - 2 ** 18, 2 ** 31 - 1024
    assert fork(lib, pages=pages, ws=None) == WS                           # every other argument is accepted
    assert fork(lib, pages=pages + 1, ws=None) == INV
    assert fork(lib, R=1, R2=1, M=row, ps=1, ws=None) == WS
    assert fork(lib, R=1, R2=1, M=row + 1, ps=1, ws=None) == INV
    assert lib.kda_cache_fork_workspace_size(2, 2, 4, pages) > 0
    assert lib.kda_cache_fork_workspace_size(2, 2, 4, pages + 1) == 0
    assert lib.kda_cache_fork_workspace_size(2, 2, row + 1, 10) == 0
    assert compact(lib, pages=pages, ws=None) == WS and compact(lib, pages=pages + 1, ws=None) == INV
    assert lib.kda_cache_compact_workspace_size(pages) > 0
    assert lib.kda_cache_compact_workspace_size(pages + 1) == 0


def test_binding_wants_cuda_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_state_fork(torch.zeros(1, 2, 8), i, i)
    with pytest.raises(ValueError):
        kda.kda_copy_pages(torch.zeros(1, 2, 8), None, i)
    with pytest.raises(ValueError):
        kda.kda_beam_select(torch.zeros(2, 8), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        kda.kda_attention_decode(torch.zeros(1, 2, 64), torch.zeros(3, 2, 4, 64), torch.zeros(3, 2, 4, 64),
                                 torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_structures_have_the_headers_sizes():
    assert ctypes.sizeof(binding.Pool) == 40
