"""Prompts' way through a hybrid stack as programs make it: pages handed out, chunks of keys and values rotated into them,
attention over them, decoding behind them, and the log probabilities of what came out, against attention over whole
sequences in float64 and, for the example, against its own search.

Tolerances, relative Frobenius: attention's own (3e-3 bf16, 1e-5 fp32), and what rotating brings to queries and keys: one
more rounding of each, at most 2^-8 of a value in bf16 and 1.7e-3 in the mean, which moves a score of standard deviation 1
by 2.4e-3 and an output, relative to it, by as much again with one word in sight; together 6e-3 (fp32: 2e-5)."""

import importlib.util
import math
import os

import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 6e-3, "f32": 2e-5}
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_beam_search", os.path.join(ROOT, "examples", "hybrid_beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def whole(qkv, Hq, Hkv, f, scale, window, sinks):
    """Rotated attention over one sequence's fused projection [T, Hq + 2 Hkv, d], float64."""
    x, T, n = qkv.double(), qkv.shape[0], f.shape[0]
    turn = torch.exp(1j * torch.arange(T, device=DEV).double()[:, None] * f)[:, None]
    z = torch.complex(x[:, :Hq + Hkv, :n], x[:, :Hq + Hkv, n:2 * n]) * turn
    x = x.clone()
    x[:, :Hq + Hkv, :2 * n] = torch.cat([z.real, z.imag], -1)
    q, k, v = x[:, :Hq].unflatten(1, (Hkv, Hq // Hkv)), x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    i, j = torch.arange(T, device=DEV)[:, None], torch.arange(T, device=DEV)[None, :]
    hidden = (j > i) | ((j <= i - window) & (j >= sinks) if window else j > i)
    s = (torch.einsum("thgd,jhd->hgtj", q, k) * scale).masked_fill(hidden, -float("inf"))
    return torch.einsum("hgtj,jhd->thgd", torch.softmax(s, 3), v).flatten(1, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d,rot,ps,window,sinks", [(8, 2, 128, 128, 16, 0, 0), (6, 2, 64, 32, 24, 70, 3), (4, 4, 16, 16, 7, 0, 0)])
def test_chunks_then_single_tokens(dtype, Hq, Hkv, d, rot, ps, window, sinks):
    """Five sequences in three calls of uneven chunks (none, one token, many), then four decode steps, two through the chunks'
    calls and two through the decode operator, all of it on pages that a fork call hands out; the last step in a graph."""
    i32 = dict(dtype=torch.int32, device=DEV)
    lengths = [1, 37, 300, 129, 64]
    chunks = [[1, 20, 0, 128, 64], [0, 1, 299, 1, 0], [0, 16, 1, 0, 0]]
    steps, B = 4, len(lengths)
    g = torch.Generator(device=DEV).manual_seed(d + ps)
    qkv = [torch.randn((n + steps, Hq + 2 * Hkv, d), device=DEV, generator=g).to(DT[dtype]) for n in lengths]
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) / (rot // 2))
    scale = d ** -0.5
    want = [whole(x, Hq, Hkv, f, scale, window, sinks) for x in qkv]
    M = -(-(max(lengths) + steps) // ps)
    P = sum(-(-(n + steps) // ps) for n in lengths)
    pools = [torch.full((P, Hkv, ps, d), float("nan"), dtype=DT[dtype], device=DEV) for _ in range(2)]
    table, lens, ref = torch.full((B, M), -1, **i32), torch.zeros(B, **i32), torch.zeros(P, **i32)
    same, done = torch.arange(B, **i32), [0] * B

    def split(x):
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def call(x, cu, table, lens):
        q, k, v = split(x)
        q = kda.kda_cache_append(k, v, *pools, table, lens, cu, q=q, inv_freq=f)
        return kda.kda_attention_prefill(q, *pools, table, lens, cu, scale=scale, window=window, sinks=sinks)

    def compare(o, counts):
        ref = torch.cat([w[a:a + n] for w, a, n in zip(want, done, counts)])
        assert float((o.double() - ref).norm() / ref.norm()) <= TOL[dtype]
        for b, n in enumerate(counts):
            done[b] += n

    for counts in chunks + [[1] * B] * 2:
        grow = torch.tensor(counts, **i32)
        table, lens, ref = kda.kda_cache_fork(table, lens, same, ref, ps, grow=grow)
        cu = torch.tensor([0] + counts).cumsum(0).int().to(DEV)
        compare(call(torch.cat([x[a:a + n] for x, a, n in zip(qkv, done, counts)]), cu, table, lens), counts)
    one = torch.ones(B, **i32)
    x = torch.cat([x[a:a + 1] for x, a in zip(qkv, done)])
    table, lens, ref = kda.kda_cache_fork(table, lens, same, ref, ps, grow=one)

    def step():
        q, k, v = split(x)
        q, k = kda.kda_rotary(q, k, lens - 1, f)
        return kda.kda_attention_decode(q, *pools, table, lens, scale=scale, window=window, sinks=sinks, k_new=k, v_new=v.contiguous())

    compare(step(), [1] * B)
    grown = kda.kda_cache_fork(table, lens, same, ref, ps, grow=one)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                      # captured on the old step's buffers, replayed on the new one's
        o = step()
    table.copy_(grown[0]), lens.copy_(grown[1])
    x.copy_(torch.cat([x[a:a + 1] for x, a in zip(qkv, done)]))
    graph.replay()
    compare(o, [1] * B)
    assert done == [len(q) for q in qkv] and kda.kda_get_device_error() == 0


def test_the_example_scores_its_beams_as_it_found_them(example):
    """The sum of a found sequence's log probabilities is the search's score, which is summed word by word in fp32 from logits
    that other operators made: twelve words of logits up to 20 in size, each within 1e-5 of their size."""
    model = example.HybridStack(seed=3)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 17, 40)]
    scores, sequences = example.beam_search(model, prompts, K=3, steps=12, eos=5)
    every = [p for p in prompts for _ in range(3)]
    found = [example.until(beam, 5) for beams in sequences for beam in beams]
    got, packed = example.score(model, every, found, top=4)
    total = torch.stack([got.logp[a:b].sum() for a, b in zip(packed.tolist(), packed[1:].tolist())]).view(3, 3)
    assert float((total - scores).abs().max()) <= 12 * 20 * 1e-5
    assert kda.kda_get_device_error() == 0
    assert bool((got.top_logp[:, :-1] >= got.top_logp[:, 1:]).all())
    # the words themselves in float64, through whole score matrices
    spec = importlib.util.spec_from_file_location("search_test", os.path.join(ROOT, "tests", "test_gpu_hybrid_beam_search.py"))
    plain = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(plain)
    for n in (0, 4, 8):
        p, c, at = every[n], found[n], int(packed[n]) + len(every[n]) - 1
        for i in sorted({0, len(c) // 2, len(c) - 1}):
            lp = plain.next_log_probs(model, p + c[:i])
            assert abs(float(got.logp[at + i]) - float(lp[c[i]])) <= 20 * 1e-5
            assert float((got.top_logp[at + i].double() - torch.topk(lp, 4).values).abs().max()) <= 20 * 1e-5


def test_the_example_runs(example, capsys):
    example.main()
    assert capsys.readouterr().out.count("words the likeliest") == 12
