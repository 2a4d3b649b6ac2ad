"""A beam search over a small hybrid stack: KDA layers and full-attention layers in turn, random weights.

Shows the calls of a decode loop as a serving program makes them.  For N requests with K beams each, N * K rows:

* ``kda_cache_fork`` hands pages out to the (until then empty) rows; in the layers ``kda_prefill`` brings the prompts'
  KDA states, ``kda_cache_append`` their keys and values into the pages, ``kda_attention_prefill`` their attention;
* each step, ``kda_beam_select`` chooses the beams that go on, ``kda_state_fork`` and ``kda_cache_fork`` give them
  their states and pages, ``kda_decode_step`` and ``kda_attention_decode`` run the layers on the new tokens;
* at the end ``kda_token_logprobs`` scores the found sequences in one pass over all of them, as prompts.

Run on a GPU:  python examples/hybrid_beam_search.py
"""

import math
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kda_gated_delta_03_gb300 as kda  # noqa: E402


class HybridStack:
    """`layers` of "k" (KDA) and "a" (attention) with random weights; activations in fp32."""

    def __init__(self, vocab=211, width=96, heads=4, kv_heads=2, d=16, layers="kaka", seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=device) / math.sqrt(s[0])
        self.H, self.Hkv, self.d, self.kinds, self.device, self.vocab = heads, kv_heads, d, layers, device, vocab
        self.embed = torch.randn((vocab, width), generator=g, device=device)
        self.head = r(width, vocab) * 3
        n = heads * d
        self.w = [dict(q=r(width, n), k=r(width, n), v=r(width, n), beta=r(width, heads), alpha=r(width, n), o=r(n, width))
                  if kind == "k" else dict(q=r(width, n), k=r(width, kv_heads * d), v=r(width, kv_heads * d), o=r(n, width))
                  for kind in layers]

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)

    def kda_inputs(self, w, x):
        """q, k (unit length), v, beta, alpha of KDA for rows x [T, width]."""
        T, H, d = x.shape[0], self.H, self.d
        q, k = (torch.nn.functional.normalize((x @ w[n]).view(T, H, d), dim=-1) for n in ("q", "k"))
        beta = torch.sigmoid(x @ w["beta"])
        alpha = torch.exp(-torch.nn.functional.softplus(x @ w["alpha"]) / 8).view(T, H, d)
        return q, k, (x @ w["v"]).view(T, H, d), beta, alpha

    def attention_inputs(self, w, x):
        T = x.shape[0]
        return ((x @ w["q"]).view(T, self.H, self.d), (x @ w["k"]).view(T, self.Hkv, self.d),
                (x @ w["v"]).view(T, self.Hkv, self.d))


def run_prompts(model, prompts, K, k_pool, v_pool, table, lens, states=None):
    """Prompts through the layers, packed one after the other, prompt n in row n * K of the table (the other rows stay
    empty).  Returns the last layer's outputs and the prompts' borders; states[layer, n * K] receives their KDA states."""
    dev, (H, d) = model.device, (model.H, model.d)
    packed = torch.tensor([0] + [len(p) for p in prompts]).cumsum(0).int()
    rows = torch.cat([packed[:1], packed[1:].repeat_interleave(K)]).to(dev)  # borders of all rows, empty ones among them
    packed = packed.to(dev)
    x = model.embed[torch.tensor([t for p in prompts for t in p], device=dev)]
    ik = ia = 0
    for kind, w in zip(model.kinds, model.w):
        h = model.norm(x)
        if kind == "k":
            o, s = kda.kda_prefill(*(t.contiguous() for t in model.kda_inputs(w, h)), packed)
            if states is not None:
                states[ik, ::K] = s
            ik += 1
        else:
            q, k, v = model.attention_inputs(w, h)
            kda.kda_cache_append(k, v, k_pool[ia], v_pool[ia], table, lens, rows)
            o = kda.kda_attention_prefill(q, k_pool[ia], v_pool[ia], table, lens, rows, scale=1 / math.sqrt(d))
            ia += 1
        x = x + o.reshape(-1, H * d) @ w["o"]
    return x, packed


def score(model, prompts, continuations, page_size=4, top=1):
    """Log probabilities of each prompt's continuation, word by word, and the `top` likeliest words in their places: the
    TokenLogprobs of all sequences' tokens packed one after the other (0 for the prompts' own words), and the borders."""
    dev, n = model.device, len(prompts)
    sequences = [list(p) + list(c) for p, c in zip(prompts, continuations)]
    counts = [-(-len(s) // page_size) for s in sequences]
    i32 = dict(dtype=torch.int32, device=dev)
    k_pool = torch.zeros((model.kinds.count("a"), sum(counts), model.Hkv, page_size, model.d), device=dev)
    v_pool = torch.zeros_like(k_pool)
    table, lens, _ = kda.kda_cache_fork(torch.empty((0, max(counts)), **i32), torch.empty(0, **i32), torch.full((n,), -1, **i32),
                                        torch.zeros(sum(counts), **i32), page_size,
                                        grow=torch.tensor([len(s) for s in sequences], **i32))
    x, packed = run_prompts(model, sequences, 1, k_pool, v_pool, table, lens)
    # a position's logits are about the next word
    words = [t for p, s in zip(prompts, sequences) for t in [-1] * (len(p) - 1) + s[len(p):] + [-1]]
    return kda.kda_token_logprobs(model.norm(x) @ model.head, torch.tensor(words, **i32), top=top), packed


def beam_search(model, prompts, K, steps, eos, page_size=4, pages=None):
    """The K best continuations of each prompt: (scores [N, K], sequences: N lists of K token lists)."""
    dev, N = model.device, len(prompts)
    R, H, Hkv, d = N * K, model.H, model.Hkv, model.d
    n_kda, n_att = model.kinds.count("k"), model.kinds.count("a")
    longest = max(map(len, prompts)) + steps
    M = -(-longest // page_size)
    pages = pages or R * M
    i32 = dict(dtype=torch.int32, device=dev)
    states = torch.zeros((n_kda, R, H, d, d), device=dev)                    # one slot per row and layer
    k_pool = torch.zeros((n_att, pages, Hkv, page_size, d), device=dev)
    v_pool = torch.zeros_like(k_pool)
    state_idx = torch.arange(R, **i32)
    ref = torch.zeros(pages, **i32)

    # ---- prompts: the first row of each group gets pages for its prompt, the others stay empty ----
    lens = torch.zeros(R, **i32)
    lens[::K] = torch.tensor([len(p) for p in prompts], **i32)
    table, lens, ref = kda.kda_cache_fork(torch.empty((0, M), **i32), torch.empty(0, **i32), torch.full((R,), -1, **i32), ref,
                                          page_size, grow=lens)
    x, packed = run_prompts(model, prompts, K, k_pool, v_pool, table, lens, states)
    logits = torch.zeros((R, model.vocab), device=dev)
    logits[::K] = model.norm(x[packed[1:].long() - 1]) @ model.head

    # ---- steps ----
    scores = torch.full((N, K), float("-inf"), device=dev)
    scores[:, 0] = 0                                                         # one beam so far
    finished = torch.zeros((N, K), dtype=torch.uint8, device=dev)
    one, history = torch.ones(R, **i32), []
    for step in range(steps):
        scores, parent, token, finished = kda.kda_beam_select(logits, scores, finished=finished, eos_token=eos)
        history.append((parent, token))
        if step + 1 == steps:
            break
        state_idx = kda.kda_state_fork(states, state_idx, parent)
        table, lens, ref = kda.kda_cache_fork(table, lens, parent, ref, page_size, grow=one, pools=(k_pool, v_pool))
        x = model.embed[token.view(-1).long()]
        ik = ia = 0
        for kind, w in zip(model.kinds, model.w):
            h = model.norm(x)
            if kind == "k":
                o = kda.kda_decode_step(*(t.contiguous() for t in model.kda_inputs(w, h)), states[ik], state_idx)
                ik += 1
            else:
                q, k, v = model.attention_inputs(w, h)
                o = kda.kda_attention_decode(q, k_pool[ia], v_pool[ia], table, lens, scale=1 / math.sqrt(d), k_new=k, v_new=v)
                ia += 1
            x = x + o.reshape(R, H * d) @ w["o"]
        logits = model.norm(x) @ model.head
    errors = kda.kda_get_device_error()
    if errors:
        raise RuntimeError(f"device error bits {errors:#x}")

    # ---- follow the parents back ----
    rows, sequences = torch.arange(R), [[] for _ in range(R)]
    for parent, token in reversed(history):
        parent, token = parent.view(-1).cpu(), token.view(-1).cpu()
        for i in range(R):
            sequences[i].insert(0, int(token[rows[i]]))
        rows = parent[rows].long()
    return scores, [sequences[n * K:(n + 1) * K] for n in range(N)]


def until(beam, eos):
    """A found sequence up to its first end."""
    return beam[:beam.index(eos) + 1] if eos in beam else beam


def main():
    model = HybridStack()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (9, 1, 30)]
    scores, sequences = beam_search(model, prompts, K=4, steps=12, eos=5)
    sequences = [[until(beam, 5) for beam in beams] for beams in sequences]
    again, packed = score(model, [p for p in prompts for _ in range(4)], [beam for beams in sequences for beam in beams])
    likeliest = [x == w for x, w in zip(again.top_logp[:, 0].tolist(), again.logp.tolist())]
    packed = packed.tolist()
    for n, (s, beams) in enumerate(zip(scores.tolist(), sequences)):
        print(f"prompt of {len(prompts[n])} tokens")
        for i, (total, beam) in enumerate(zip(s, beams)):
            end = packed[4 * n + i + 1] - 1
            print(f"  {total:9.4f}  {beam}  ({sum(likeliest[end - len(beam):end])} of {len(beam)} words the likeliest)")


if __name__ == "__main__":
    main()
