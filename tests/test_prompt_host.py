"""Host-side checks of the prompt operators (rotary positions, cache append, attention of chunks, token log probabilities):
every bad argument is refused before any CUDA call, so these run without a GPU.  The addresses below are never
dereferenced."""

import contextlib
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
P, P2, ODD8, ODD4, ODD2, ODD1 = 0x10000, 0x20000, 0x10008, 0x10004, 0x10002, 0x10001


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def rotary(lib, **over):
    a = dict(q=P, k=P, pos=P, freq=P, T=3, Hq=8, Hkv=2, d=64, rot=64, qs=512, ks=128, dt=1, layout=0, scale=1.0, inverse=0,
             qo=P2, qos=512, ko=P2, kos=128, stream=None)
    a.update(over)
    return lib.kda_rotary(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INV), (dict(Hq=-1), INV), (dict(Hkv=-1), INV), (dict(d=0), INV), (dict(rot=-2), INV), (dict(rot=3), INV),
    (dict(rot=66), INV), (dict(dt=2), INV), (dict(layout=2), INV), (dict(layout=-1), INV), (dict(scale=float("nan")), INV),
    (dict(qs=511), INV), (dict(ks=127), INV), (dict(qos=511), INV), (dict(kos=100), INV), (dict(freq=None), INV),
    (dict(freq=ODD4), INV), (dict(pos=None), INV), (dict(pos=ODD2), INV), (dict(q=None), INV), (dict(qo=None), INV),
    (dict(ko=None), INV), (dict(q=ODD1), INV), (dict(k=ODD1), INV), (dict(qo=ODD1), INV), (dict(ko=ODD1), INV),
    (dict(q=ODD2, dt=0), INV), (dict(qo=P, qos=600), INV), (dict(ko=P, kos=600), INV), (dict(d=32, rot=32), UNS),
    (dict(d=256, Hq=1, Hkv=1, qs=512, ks=256, kos=256), UNS), (dict(Hq=1 << 24, qs=1 << 30, qos=1 << 30), INV), (dict(T=0), OK),
    (dict(k=None, Hkv=7, ks=0, Hq=0), OK),
])
def test_rotary_refuses(lib, over, code):
    assert rotary(lib, **over) == code


def append(lib, **over):
    a = dict(q=P, k=P, v=P, kp=P, vp=P, table=P, lens=P, cu=P, freq=P, B=2, T=5, Hq=8, Hkv=2, d=64, rot=64, qs=512, ks=128,
             vs=128, pages=10, ps=16, M=4, kps=2048, vps=2048, dt=1, layout=1, scale=1.0, qo=P2, qos=512, stream=None)
    a.update(over)
    return lib.kda_cache_append(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(Hq=-1), INV), (dict(Hkv=0), INV), (dict(Hkv=-2), INV), (dict(rot=65), INV),
    (dict(pages=-1), INV), (dict(ps=0), INV), (dict(M=-1), INV), (dict(M=1 << 28), INV), (dict(qs=500), INV), (dict(ks=127), INV),
    (dict(vs=127), INV), (dict(qos=511), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(v=ODD1), INV), (dict(lens=None), INV),
    (dict(cu=None), INV), (dict(cu=ODD2), INV), (dict(lens=ODD2), INV), (dict(table=None), INV), (dict(table=ODD2), INV),
    (dict(kp=None), INV), (dict(vp=ODD8), INV), (dict(pages=0), INV), (dict(kps=2040), INV), (dict(kps=2049), INV),
    (dict(vps=1024), INV), (dict(qo=None), INV), (dict(qo=P, qos=520), INV), (dict(freq=None), INV), (dict(d=32, rot=0), UNS),
    (dict(dt=7), INV), (dict(layout=5), INV), (dict(B=2 ** 31 - 1), INV), (dict(T=0), OK), (dict(B=0), OK),
])
def test_append_refuses(lib, over, code):
    assert append(lib, **over) == code


def attention(lib, **over):
    a = dict(q=P, k=P, v=P, table=P, lens=P, cu=P, B=2, T=9, Hq=8, Hkv=2, d=64, pages=10, ps=16, M=4, ks=2048, vs=2048, dt=1,
             scale=1.0, window=0, sinks=0, o=P, lse=None, ws=P, wsb=1 << 40, stream=None)
    a.update(over)
    return lib.kda_attention_prefill(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(Hq=9), INV), (dict(d=0), INV),
    (dict(pages=-1), INV), (dict(ps=0), INV), (dict(M=-1), INV), (dict(window=-1), INV), (dict(sinks=-2), INV),
    (dict(scale=float("inf")), INV), (dict(dt=2), INV), (dict(d=32), UNS), (dict(d=256), UNS), (dict(q=None), INV),
    (dict(q=ODD8), INV), (dict(o=None), INV), (dict(o=ODD8), INV), (dict(k=None), INV), (dict(v=ODD8), INV), (dict(table=None), INV),
    (dict(lens=ODD2), INV), (dict(cu=None), INV), (dict(cu=ODD2), INV), (dict(lse=ODD2), INV), (dict(pages=0), INV),
    (dict(ks=2047), INV), (dict(ks=1024), INV), (dict(vs=2040, ks=2040), INV), (dict(M=1 << 28, ps=16), INV),
    (dict(T=1 << 28), INV), (dict(B=2 ** 31 - 1), INV), (dict(Hq=2 ** 25), INV), (dict(ws=None), WS), (dict(wsb=1000), WS),
    (dict(ws=0x10010), WS), (dict(B=0), OK), (dict(T=0), OK),
])
def test_attention_refuses(lib, over, code):
    assert attention(lib, **over) == code


def test_attention_longest_table_and_workspace(lib):
    last = 2 ** 31 - 1024
    assert attention(lib, M=1, pages=1, ps=last, ws=None) == WS            # every other argument is accepted
    assert attention(lib, M=1, pages=1, ps=last + 1, ws=None) == INV
    size = lib.kda_attention_prefill_workspace_size
    assert size(0, 5, 8, 2, 64, 1) == 0 and size(2, 5, 9, 2, 64, 1) == 0 and size(2, 5, 8, 2, 32, 1) == 0 and size(2, 5, 8, 2, 64, 9) == 0
    for dt in (0, 1):
        need = size(2, 9, 8, 2, 64, dt)
        assert need > 0 and need % 256 == 0 and attention(lib, dt=dt, wsb=need - 1) == WS


def logprobs(lib, **over):
    a = dict(x=P, stride=100, tokens=P, T=3, V=100, dt=1, top=4, logp=P, lse=P, entropy=P, tl=P, tt=P, stream=None)
    a.update(over)
    return lib.kda_token_logprobs(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INV), (dict(V=0), INV), (dict(V=-3), INV), (dict(dt=3), INV), (dict(stride=99), INV), (dict(top=-1), INV),
    (dict(top=33), UNS), (dict(top=6, V=5), INV), (dict(x=None), INV), (dict(x=ODD1), INV), (dict(x=ODD2, dt=0), INV),
    (dict(tokens=None), INV), (dict(tokens=ODD2), INV), (dict(logp=None), INV), (dict(lse=ODD2), INV), (dict(entropy=ODD2), INV),
    (dict(tl=None), INV), (dict(tt=None), INV), (dict(tt=ODD2), INV), (dict(T=1 << 28), TOO_LARGE),
    (dict(V=2 ** 31 - 2 ** 14 + 1, stride=1 << 31), TOO_LARGE), (dict(T=0), OK),
])
def test_logprobs_refuses(lib, over, code):
    assert logprobs(lib, **over) == code


def backward(lib, **over):
    a = dict(x=P, stride=100, tokens=P, lse=P, entropy=P, gl=P, gh=P, T=3, V=100, dt=1, grad=P2, gstride=100, stream=None)
    a.update(over)
    return lib.kda_token_logprobs_backward(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), INV), (dict(V=0), INV), (dict(dt=3), INV), (dict(stride=99), INV), (dict(gstride=99), INV), (dict(entropy=None), INV),
    (dict(gh=None), INV), (dict(x=None), INV), (dict(x=ODD1), INV), (dict(tokens=None), INV), (dict(lse=None), INV), (dict(gl=None), INV),
    (dict(gl=ODD2), INV), (dict(gh=ODD2), INV), (dict(entropy=ODD2), INV), (dict(grad=None), INV), (dict(grad=ODD1), INV),
    (dict(grad=P, gstride=104), INV), (dict(T=1 << 28), TOO_LARGE), (dict(T=1 << 27, V=1 << 17, stride=1 << 17, gstride=1 << 17), TOO_LARGE),
    (dict(V=2 ** 31 - 2 ** 14 + 1, stride=1 << 31, gstride=1 << 31), TOO_LARGE), (dict(T=0), OK),
])
def test_backward_refuses(lib, over, code):
    assert backward(lib, **over) == code


def test_backward_refuses_more_chunks_than_a_grid_has(lib):
    assert backward(lib, T=1 << 20, V=1 << 22, stride=1 << 22, gstride=1 << 22, dt=0) == TOO_LARGE


def test_backward_takes_as_many_chunks_as_a_grid_has(lib):
    """Chunks of 4,096 bf16 and 2,048 fp32 words, wherever a row begins.  A call that is not too large is refused for its logits."""
    for dt, words, short in ((1, 4096, 7), (0, 2048, 3)):
        for V, chunks in ((9 * words - short, 9), (9 * words - short + 1, 10), (512 * words, 513), (1023 * words, 1024)):
            rows = (2 ** 31 - 1) // chunks
            assert backward(lib, T=rows, V=V, stride=V, gstride=V, dt=dt, x=None) == INV
            assert backward(lib, T=rows + 1, V=V, stride=V, gstride=V, dt=dt, x=None) == TOO_LARGE


def test_binding_wants_cuda_tensors():
    i, x = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, 64)
    pool, table = torch.zeros(3, 1, 4, 64), torch.zeros((1, 2), dtype=torch.int32)
    f = torch.zeros(4, dtype=torch.float64)
    for call in (lambda: kda.kda_rotary(x, x, i, f), lambda: kda.kda_cache_append(x, x, pool, pool, table, i[:1], i),
                 lambda: kda.kda_attention_prefill(x, pool, pool, table, i[:1], i),
                 lambda: kda.kda_token_logprobs(torch.zeros(2, 8), i),
                 lambda: kda.kda_token_logprobs_backward(torch.zeros(2, 8), i, f.float(), f.float())):
        with pytest.raises(ValueError):
            call()


@pytest.fixture
def passed(monkeypatch):
    """The binding on tensors without data (device -1), before a library that takes any call: its calls' names."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or 0

    monkeypatch.setattr(binding, "_LIB", Library())
    monkeypatch.setattr(binding, "_cuda_index", lambda name, t: t.get_device())
    monkeypatch.setattr(binding, "_elsewhere", lambda dev, stream: False)
    monkeypatch.setattr(binding, "_current_raw_stream", lambda dev: 0)
    monkeypatch.setattr(binding, "_new_workspace", lambda need, dev: torch.empty(1, dtype=torch.uint8))
    return calls


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63, -2 ** 31 - 1, -2 ** 32])
def test_numbers_beyond_32_bits_are_refused(passed, value):
    """ctypes passes the lower 32 bits of a number: a window of 2^32 would be none, 2^32 first tokens none at all."""
    i32 = dict(dtype=torch.int32)
    pages = (meta(3, 1, 4, 64), meta(3, 1, 4, 64), meta(1, 2, **i32))
    for over in (dict(window=value), dict(sinks=value), dict(window=5, sinks=value)):
        with pytest.raises(ValueError):
            kda.kda_attention_prefill(meta(2, 1, 64), *pages, meta(1, **i32), meta(2, **i32), **over)
        with pytest.raises(ValueError):
            kda.kda_attention_decode(meta(1, 1, 64), *pages, meta(1, **i32), **over)
    with pytest.raises(ValueError):
        kda.kda_token_logprobs(meta(2, 9), meta(2, **i32), top=value)
    assert not [c for c in passed if not c.endswith("_size")]
    kda.kda_attention_prefill(meta(2, 1, 64), *pages, meta(1, **i32), meta(2, **i32), window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    assert passed[-1] == "kda_attention_prefill"


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32, 2 ** 32 + 3])
def test_sizes_beyond_32_bits_are_refused(passed, n):
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    pages, table, one = (meta(3, 1, 4, 16), meta(3, 1, 4, 16)), meta(1, 2, **i32), meta(1, **i32)
    many = (meta(n, 1, 4, 16), meta(n, 1, 4, 16))
    q, two = meta(2, 1, 16), meta(2, **i32)
    for call in (lambda: kda.kda_rotary(meta(n, 1, 16), None, meta(n, **i32), None),
                 lambda: kda.kda_rotary(q, meta(2, n, 16), two, None),
                 lambda: kda.kda_cache_append(q, q, *pages, table, one, two, q=meta(2, n, 16)),
                 lambda: kda.kda_attention_prefill(meta(2, n, 16), *pages, table, one, two),
                 lambda: kda.kda_cache_append(meta(n, 1, 16), meta(n, 1, 16), *pages, table, one, two),
                 lambda: kda.kda_cache_append(q, q, *many, table, one, two),
                 lambda: kda.kda_cache_append(q, q, *pages, meta(n, 2, **i32), meta(n, **i32), meta(n + 1, **i32)),
                 lambda: kda.kda_cache_append(q, q, *pages, meta(1, n, **i32), one, two),
                 lambda: kda.kda_attention_prefill(meta(n, 1, 16), *pages, table, one, two),
                 lambda: kda.kda_attention_prefill(q, *many, table, one, two),
                 lambda: kda.kda_attention_prefill(q, *pages, meta(1, n, **i32), one, two),
                 lambda: kda.kda_token_logprobs(meta(n, 3), meta(n, **i32)),
                 lambda: kda.kda_token_logprobs(meta(1, n), one),
                 lambda: kda.kda_token_logprobs_backward(meta(n, 3), meta(n, **i32), meta(n, **f32), meta(n, **f32)),
                 lambda: kda.kda_token_logprobs_backward(meta(1, n), one, meta(1, **f32), meta(1, **f32))):
        with pytest.raises(ValueError):
            call()
    assert not passed
    kda.kda_token_logprobs_backward(meta(4, 9), meta(4, **i32), meta(4, **f32), meta(4, **f32))
    assert passed == ["kda_token_logprobs_backward"]


def test_streams_of_another_device_are_refused(monkeypatch):
    """Such a call would find itself on the tensors' device and that device's own current stream, unordered with the given one."""
    ran = []
    monkeypatch.setattr(binding, "_cuda_index", lambda name, t: 0)
    monkeypatch.setattr(binding, "_in_stream", lambda stream, call, *args, **kwargs: ran.append(call))
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())

    class Stream:
        cuda_stream = 0

        def __init__(self, device_index):
            self.device_index = device_index

    i, x = meta(2, dtype=torch.int32), meta(2, 1, 64)
    pool, table, f = meta(3, 1, 4, 64), meta(1, 2, dtype=torch.int32), meta(2, dtype=torch.float32)
    calls = [lambda s: kda.kda_rotary(x, x, i, None, stream=s), lambda s: kda.kda_cache_append(x, x, pool, pool, table, i[:1], i, stream=s),
             lambda s: kda.kda_attention_prefill(x, pool, pool, table, i[:1], i, stream=s),
             lambda s: kda.kda_token_logprobs(meta(2, 8), i, stream=s),
             lambda s: kda.kda_token_logprobs_backward(meta(2, 8), i, f, f, stream=s)]
    for call in calls:
        with pytest.raises(ValueError):
            call(Stream(1))
    assert not ran
    for call in calls:
        call(Stream(0))
    assert len(ran) == len(calls)
