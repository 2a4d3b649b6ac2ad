"""The decode loop of examples/hybrid_beam_search.py against a search that keeps no state: every beam's whole
sequence is run through the layers anew at each step, in float64, token by token for KDA and with a full score
matrix for attention.  And the same step captured in a CUDA graph."""

import importlib.util
import math
import os

import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_beam_search", os.path.join(ROOT, "examples", "hybrid_beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def next_log_probs(model, tokens):
    """log softmax of the logits after a sequence of tokens, float64."""
    x = model.embed[torch.tensor(tokens, device=model.device)].double()
    T, H, Hkv, d = len(tokens), model.H, model.Hkv, model.d
    for kind, w in zip(model.kinds, model.w):
        w = {n: t.double() for n, t in w.items()}
        h = model.norm(x)
        if kind == "k":
            q, k, v, beta, alpha = model.kda_inputs(w, h)
            S, o = torch.zeros((H, d, d), dtype=torch.float64, device=x.device), []
            for t in range(T):
                S = alpha[t][:, :, None] * S
                S = S + beta[t][:, None, None] * k[t][:, :, None] * (v[t] - torch.einsum("hi,hij->hj", k[t], S))[:, None, :]
                o.append(torch.einsum("hij,hi->hj", S, q[t]))
            o = torch.stack(o)
        else:
            q, k, v = model.attention_inputs(w, h)
            a = torch.einsum("thgd,shd->hgts", q.view(T, Hkv, H // Hkv, d), k) / math.sqrt(d)
            mask = torch.ones((T, T), dtype=torch.bool, device=x.device).tril()
            o = torch.einsum("hgts,shd->thgd", torch.softmax(a.masked_fill(~mask, float("-inf")), -1), v)
        x = x + o.reshape(T, H * d) @ w["o"]
    return torch.log_softmax(model.norm(x[-1]) @ model.head.double(), -1)


def search(model, prompt, K, steps, eos):
    beams = [(0.0, [], False)]
    for _ in range(steps):
        cands = []
        for b, (s, seq, done) in enumerate(beams):
            if done:
                cands.append((s, b, eos))
                continue
            lp = s + next_log_probs(model, prompt + seq)
            top = torch.topk(lp, K)
            cands += [(float(v), b, int(i)) for v, i in zip(top.values, top.indices)]
        cands.sort(key=lambda c: (-c[0], c[1], c[2]))
        beams = [(s, beams[b][1] + [t], beams[b][2] or t == eos) for s, b, t in cands[:K]]
    return beams


@pytest.mark.parametrize("K,steps,page_size,layers", [(4, 10, 4, "kaka"), (3, 9, 1, "ka"), (5, 8, 16, "ak"), (1, 12, 3, "kaak")])
def test_beam_search_matches_a_search_without_state(example, K, steps, page_size, layers):
    model = example.HybridStack(vocab=61, layers=layers, seed=K)
    g = torch.Generator().manual_seed(steps)
    prompts = [torch.randint(0, 61, (n,), generator=g).tolist() for n in (7, 1, 20)]
    with torch.no_grad():
        # a word that ends sequences early for some beams: the likeliest first word of the second prompt
        eos = int(next_log_probs(model, prompts[1]).argmax())
        scores, sequences = example.beam_search(model, prompts, K, steps, eos, page_size)
        for n, prompt in enumerate(prompts):
            want = search(model, prompt, K, steps, eos)
            for b in range(K):
                assert abs(float(scores[n, b]) - want[b][0]) <= 1e-3, (n, b)
                assert sequences[n][b] == want[b][1], (n, b)


def test_a_whole_step_in_a_cuda_graph(example):
    """Select, forks, decode and attention replayed from one capture: two replays from the same buffers give what two
    direct steps give."""
    dev, N, K, H, Hkv, d, ps, V = "cuda:0", 3, 4, 4, 2, 64, 16, 1000
    R, M, P = N * K, 12, 300
    g = torch.Generator(device=dev).manual_seed(3)
    r = lambda *s: torch.randn(s, device=dev, generator=g)
    i32 = dict(dtype=torch.int32, device=dev)

    def buffers():
        g.manual_seed(3)
        b = dict(logits=r(R, V), scores=-r(N, K).abs(), states=0.1 * r(1, R, H, d, d), k=r(1, P, Hkv, ps, d), v=r(1, P, Hkv, ps, d),
                 q=r(R, H, d), kn=r(R, Hkv, d), vn=r(R, Hkv, d), beta=torch.sigmoid(r(R, H)), alpha=torch.sigmoid(r(R, H, d)),
                 idx=torch.arange(R, **i32), ref=torch.zeros(P, **i32))
        lens = torch.tensor([40] * 4 + [16] * 4 + [99] * 4, **i32)
        b["table"], b["lens"], b["ref"] = kda.kda_cache_fork(torch.empty((0, M), **i32), torch.empty(0, **i32),
                                                             torch.full((R,), -1, **i32), b["ref"], ps, grow=lens)
        b["qn"], b["kk"] = (torch.nn.functional.normalize(r(R, H, d), dim=-1) for _ in range(2))
        return b

    one = torch.ones(R, **i32)

    def step(b):
        b["scores2"], b["parent"], b["token"], _ = kda.kda_beam_select(b["logits"], b["scores"])
        b["idx2"] = kda.kda_state_fork(b["states"], b["idx"], b["parent"])
        b["table2"], b["lens2"], b["ref"] = kda.kda_cache_fork(b["table"], b["lens"], b["parent"], b["ref"], ps, grow=one,
                                                               pools=(b["k"], b["v"]))
        b["o1"] = kda.kda_decode_step(b["qn"], b["kk"], b["q"], b["beta"], b["alpha"], b["states"][0], b["idx2"])
        b["o2"] = kda.kda_attention_decode(b["q"], b["k"][0], b["v"][0], b["table2"], b["lens2"], scale=0.1, k_new=b["kn"],
                                           v_new=b["vn"])
        # the next step's inputs
        b["scores"].copy_(b["scores2"])
        b["idx"].copy_(b["idx2"])
        b["table"].copy_(b["table2"])
        b["lens"].copy_(b["lens2"])

    direct = buffers()
    step(direct)
    step(direct)
    torch.cuda.synchronize()
    captured = buffers()
    start = {n: t.clone() for n, t in captured.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(captured)                                 # warm up: first calls ask the device for its attributes
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for n, t in start.items():
        captured[n].copy_(t)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    for n in ("scores", "parent", "token", "idx", "table", "lens", "ref", "o1", "o2", "states", "k", "v"):
        assert torch.equal(direct[n], captured[n]), n
