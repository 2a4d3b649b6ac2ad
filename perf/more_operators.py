"""Cases and plain forms of the operators that bring prompts into a hybrid stack and score their tokens.

Four operators, each case one call of the library:

* ``attention``: attention of chunks of new tokens over a paged key-value cache (``kda_attention_prefill``).
* ``append``: a chunk's keys and values into their pages, queries and keys rotated by position on the way
  (``kda_cache_append``).
* ``rotary``: rotary positions of queries and keys outside a cache, and its gradient (``kda_rotary``).
* ``score`` and ``score_grad``: log probabilities of given tokens with entropy and top alternatives
  (``kda_token_logprobs``), and their gradient (``kda_token_logprobs_backward``).

``own`` false computes a case with elementary torch operations in 32 bits (rotation angles and long sums in 64);
``own`` true calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one user's next turn in a short chat: only the latency of the call counts
        dict(name="attention_one_turn", kind="attention", B=1, Hq=32, Hkv=8, d=128, page=16, n_min=37, n_max=37,
             past_min=200, past_max=200, window=0, sinks=0, dtype="bf16"),
        # one whole prompt of 8,192 tokens, as the prefill workload has
        dict(name="attention_prompt_8k", kind="attention", B=1, Hq=32, Hkv=8, d=128, page=64, n_min=8192, n_max=8192,
             past_min=0, past_max=0, window=0, sinks=0, dtype="bf16"),
        # a serving batch: prompts cut into chunks of at most 512 tokens, among rows that add a single one
        dict(name="attention_ragged_chunks", kind="attention", B=16, Hq=32, Hkv=8, d=128, page=16, n_min=1, n_max=512,
             past_min=100, past_max=7600, window=0, sinks=0, dtype="bf16"),
        # a few drafted tokens checked against one agent's long context
        dict(name="attention_few_over_256k", kind="attention", B=1, Hq=32, Hkv=8, d=128, page=256, n_min=13, n_max=13,
             past_min=262000, past_max=262000, window=0, sinks=0, dtype="bf16"),
        # a parity run in fp32 on sliding-window layers, with a page size that is no power of two
        dict(name="attention_f32_window", kind="attention", B=4, Hq=16, Hkv=4, d=64, page=24, n_min=50, n_max=700,
             past_min=1, past_max=2500, window=1000, sinks=4, dtype="f32"),
        # a decode step of 64 rows: one token each, queries and keys rotated by the half layout
        dict(name="append_one_token", kind="append", B=64, Hq=32, Hkv=8, d=128, page=16, n_min=1, n_max=1,
             past_min=100, past_max=16000, rot=128, layout="half", base=500000.0, factor=1.0, dtype="bf16"),
        # a packed batch of prompts, half of each head rotated with stretched positions
        dict(name="append_prompts", kind="append", B=12, Hq=32, Hkv=8, d=128, page=64, n_min=200, n_max=9000,
             past_min=0, past_max=100000, rot=64, layout="interleaved", base=10000.0, factor=8.0, dtype="bf16"),
        # a training batch of packed sequences
        dict(name="rotary_train", kind="rotary", T=16384, Hq=32, Hkv=8, d=128, rot=128, layout="half", base=10000.0,
             factor=1.0, far=16384, inverse=False, dtype="bf16"),
        # the gradient of a small fp32 model's rotation, at far positions
        dict(name="rotary_grad_f32", kind="rotary", T=1001, Hq=8, Hkv=2, d=64, rot=32, layout="interleaved",
             base=10000.0, factor=4.0, far=1 << 20, inverse=True, dtype="f32"),
        # the sampled token of a few rows, with the alternatives that an interface shows
        dict(name="score_step", kind="score", T=4, V=32001, top=5, dtype="f32"),
        # a prompt's tokens scored
        dict(name="score_prompt", kind="score", T=2048, V=131072, top=8, dtype="bf16"),
        # a policy's gradient over the same prompt: log probabilities with an entropy term
        dict(name="score_grad_prompt", kind="score_grad", T=2048, V=131072, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges, at most as much work as the largest of them."""
    kind = rng.choice(["attention", "attention", "attention", "append", "rotary", "score", "score_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("attention", "append"):
        while True:
            group, Hkv = rng.choice([1, 2, 3, 4, 5, 8, 12]), rng.choice([1, 2, 3, 4, 8, 16])
            n, past = _log(rng, 1, 8192), rng.choice([0, 1]) * _log(rng, 1, 300000)
            c = dict(kind=kind, B=_log(rng, 1, 64), Hq=group * Hkv, Hkv=Hkv, d=rng.choice([16, 64, 128, 128]),
                     page=rng.choice([1, 7, 16, 16, 24, 32, 64, 64, 100, 128, 256]),
                     n_min=max(1, n // rng.choice([1, 2, 10, 1000])), n_max=n,
                     past_min=past // rng.choice([1, 2, 10, 100]), past_max=past, dtype=dtype)
            tokens, longest = c["B"] * n, past + n
            if kind == "append":
                c.update(rot=rng.choice([0.0, 0.25, 0.5, 1.0, 1.0]), layout=rng.choice(["half", "interleaved"]),
                         base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 8.0]))
                c["rot"] = int(c["rot"] * c["d"])
                if tokens * c["Hq"] * c["d"] <= 1 << 28 and c["B"] * longest // c["page"] <= 1 << 22:
                    return c
            else:
                c.update(window=0, sinks=0)
                if rng.random() < 0.35:
                    c["window"], c["sinks"] = _log(rng, 1, 5000), rng.choice([0, 1, 4, 61])
                # the plain form lays scores and cache out densely in 32 bits: both bound what a case may cost, and so
                # do the 64-bit scores of one head
                if (tokens * longest * c["Hq"] <= 1 << 31 and c["B"] * longest * Hkv * c["d"] <= 1 << 30 and
                        tokens * longest * c["Hq"] * c["d"] <= 1 << 38 and n * longest * group <= 1 << 30):
                    return c
    if kind == "rotary":
        while True:
            group, Hkv = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 8])
            d = rng.choice([16, 64, 128, 128])
            c = dict(kind=kind, T=_log(rng, 1, 100000), Hq=group * Hkv, Hkv=Hkv, d=d,
                     rot=int(d * rng.choice([0.25, 0.5, 1.0, 1.0])), layout=rng.choice(["half", "interleaved"]),
                     base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 8.0]), far=_log(rng, 1, 1 << 22),
                     inverse=rng.random() < 0.5, dtype=dtype)
            if c["T"] * c["Hq"] * d <= 1 << 27:
                return c
    while True:
        c = dict(kind=kind, T=_log(rng, 1, 20000), V=_log(rng, 50, 260000), dtype=dtype)
        if kind == "score":
            c["top"] = rng.choice([0, 1, 2, 5, 8, 20])
        if c["T"] * c["V"] <= 1 << 28:
            return c


def _spread(lo, hi, n):
    """n lengths spread log-uniformly from lo to hi (the same ones for every seed, which orders them)."""
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    x = torch.exp(math.log(lo + 1) + u * (math.log(hi + 1) - math.log(lo + 1))) - 1
    return x.round().long().clamp(lo, hi)


def _lens(c):
    """New tokens of each row, and tokens that its cache holds already."""
    n, past = _spread(c["n_min"], c["n_max"], c["B"]), _spread(c["past_min"], c["past_max"], c["B"]).flip(0)
    if c["B"] >= 8:
        n[c["B"] // 3] = 0                                # a row that waits in this step
    return n, past


def _visible(c):
    """(query, token) pairs that see each other, and tokens of the cache that anybody sees."""
    n, past = _lens(c)
    pairs = read = 0
    for a, p in zip(n.tolist(), past.tolist()):
        if a == 0:
            continue
        pos = torch.arange(p, p + a, dtype=torch.float64) + 1
        if c["window"]:
            pairs += float(torch.minimum(pos, pos.clamp(max=c["window"]) + (pos - c["window"]).clamp(0, c["sinks"])).sum())
            first = max(0, p + 1 - c["window"])
            read += p + a - first + min(first, c["sinks"])
        else:
            pairs += float(pos.sum())
            read += p + a
    return pairs, read, int(n.sum())


def work(c):
    e = ESIZE[c["dtype"]]
    if c["kind"] == "attention":
        pairs, read, T = _visible(c)
        return {"bytes": read * c["Hkv"] * c["d"] * 2 * e + 2 * T * c["Hq"] * c["d"] * e + read / c["page"] * 4 + T * c["Hq"] * 4,
                "flops": 4.0 * pairs * c["Hq"] * c["d"]}
    if c["kind"] == "append":
        T = int(_lens(c)[0].sum())
        return {"bytes": 2.0 * T * (c["Hq"] + 2 * c["Hkv"]) * c["d"] * e + T / c["page"] * 4 + c["B"] * 8,
                "flops": 3.0 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["kind"] == "rotary":
        return {"bytes": 2.0 * c["T"] * (c["Hq"] + c["Hkv"]) * c["d"] * e + c["T"] * 4,
                "flops": 3.0 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["kind"] == "score":
        return {"bytes": c["T"] * c["V"] * e + c["T"] * (16.0 + 8 * c["top"]), "flops": 5.0 * c["T"] * c["V"]}
    return {"bytes": 2.0 * c["T"] * c["V"] * e + c["T"] * 20.0, "flops": 8.0 * c["T"] * c["V"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(shape, dtype, gen, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=gen)


def prepare(c, seed):
    cpu = torch.Generator().manual_seed(1000003 * seed + 29)
    gpu = torch.Generator(device=DEV).manual_seed(1000003 * seed + 30)
    made = {"attention": _prepare_attention, "append": _prepare_append, "rotary": _prepare_rotary,
            "score": _prepare_score, "score_grad": _prepare_score}[c["kind"]](c, cpu, gpu)
    return dict(made, case=dict(c))


def _prepare_rows(c, cpu):
    """A packed batch: block table, lengths with the new tokens, and where each row's new tokens lie."""
    B, ps = c["B"], c["page"]
    n, past = _lens(c)
    order = torch.randperm(B, generator=cpu)
    n, past = n[order], past[order]
    lens = n + past
    counts = -(-lens // ps)
    M, total = max(1, -(-(c["n_max"] + c["past_max"]) // ps)), int(counts.sum())
    perm = torch.randperm(total + 3, generator=cpu)[:total].int()
    table = torch.full((B, M), -1, dtype=torch.int32)
    table[torch.arange(M)[None, :] < counts[:, None]] = perm             # pages of a row lie anywhere in the pool
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = n.cumsum(0)
    return n, past, lens, table, cu, total + 3


def _prepare_attention(c, cpu, gpu):
    n, past, lens, table, cu, P = _prepare_rows(c, cpu)
    dt, ps, T = DT[c["dtype"]], c["page"], int(n.sum())
    k = _randn((P, c["Hkv"], ps, c["d"]), dt, gpu)
    v = _randn((P, c["Hkv"], ps, c["d"]), dt, gpu)
    # what lies in the pools past a row's end is left from earlier owners: not numbers anybody may read
    for b in range(min(4, c["B"])):
        end = int(lens[b])
        if end % ps:
            p = int(table[b, end // ps])
            k[p, :, end % ps:] = float("nan")
            v[p, :, end % ps:] = float("inf")
    return dict(q=_randn((T, c["Hq"], c["d"]), dt, gpu, 1.5), k_pages=k, v_pages=v, table=table.to(DEV),
                lens=lens.int().to(DEV), cu=cu.to(DEV), scale=c["d"] ** -0.5,
                o=torch.empty((T, c["Hq"], c["d"]), dtype=dt, device=DEV),
                lse=torch.empty((T, c["Hq"]), dtype=torch.float32, device=DEV))


def _frequencies(c):
    """Angles a position, and what stretched positions multiply the rotated part by."""
    half = c["rot"] // 2
    f = c["base"] ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    if c["factor"] > 1:                                   # far positions: slow pairs stretched, fast ones left
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f / c["factor"] * (1 - keep) + f * keep
    return f.to(DEV), (0.1 * math.log(c["factor"]) + 1.0)


def _prepare_append(c, cpu, gpu):
    n, past, lens, table, cu, P = _prepare_rows(c, cpu)
    dt, T, width = DT[c["dtype"]], int(n.sum()), c["Hq"] + 2 * c["Hkv"]
    used = int(table.max()) + 1                           # pools whose other pages nobody needs here
    live = torch.unique(torch.cat([table[b, p // c["page"]:-(-(p + a) // c["page"])] for b, (p, a) in
                                   enumerate(zip(past.tolist(), n.tolist())) if a] + [torch.zeros(0, dtype=torch.int32)]))
    small = torch.full((max(used, P),), -1, dtype=torch.int32)
    small[live.long()] = torch.randperm(live.numel(), generator=cpu).int()
    table = torch.where(table >= 0, small[table.clamp(min=0).long()], table)
    qkv = _randn((T, width, c["d"]), dt, gpu)             # the layer's projection: one tensor
    f, stretch = _frequencies(c)
    Hq, Hkv = c["Hq"], c["Hkv"]
    pool = lambda: _randn((live.numel() + 1, Hkv, c["page"], c["d"]), dt, gpu)
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], table=table.to(DEV), lens=lens.int().to(DEV),
                cu=cu.to(DEV), k_pages=pool(), v_pages=pool(), inv_freq=f, stretch=stretch,
                q_out=torch.empty((T, Hq, c["d"]), dtype=dt, device=DEV))


def _prepare_rotary(c, cpu, gpu):
    dt = DT[c["dtype"]]
    f, stretch = _frequencies(c)
    start = torch.randint(0, c["far"], (1 + c["T"] // 700,), generator=cpu)
    pos = (start.repeat_interleave(700)[: c["T"]] + torch.arange(c["T"]) % 700).int()   # packed sequences of 700 tokens
    return dict(q=_randn((c["T"], c["Hq"], c["d"]), dt, gpu), k=_randn((c["T"], c["Hkv"], c["d"]), dt, gpu),
                positions=pos.to(DEV), inv_freq=f, stretch=stretch)


def _prepare_score(c, cpu, gpu):
    T, V = c["T"], c["V"]
    logits = _randn((T, V), DT[c["dtype"]], gpu, 2.5)
    hot = torch.randint(0, V, (T, 12), generator=cpu).to(DEV)                  # a few likely words stand out
    logits.scatter_add_(1, hot, _randn((T, 12), DT[c["dtype"]], gpu, 4.0).abs())
    token = torch.where(torch.rand(T, generator=cpu) < 0.7, hot[:, 0].cpu(), torch.randint(0, V, (T,), generator=cpu)).int()
    if T >= 8:
        token[T // 3] = -1                                                     # padding: no token to score
    if V >= 200:
        banned = 7                                                             # a word that is not allowed here
        logits[:, banned] = float("-inf")
        token[token == banned] = 8
    s = dict(logits=logits, token=token.to(DEV))
    if c["kind"] == "score_grad":
        x = logits.double() if T * V <= 1 << 20 else logits.float()
        lse = torch.logsumexp(x, 1, keepdim=True)
        lp = x.sub_(lse)
        s["lse"] = lse[:, 0].float()
        s["entropy"] = -(torch.exp(lp) * lp.clamp(min=-1e30)).sum(1).float()
        s["g_logp"] = _randn((T,), torch.float32, gpu)
        s["g_entropy"] = _randn((T,), torch.float32, gpu, 0.01)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return {"attention": _attention, "append": _append, "rotary": _rotary, "score": _score,
            "score_grad": _score_grad}[s["case"]["kind"]](s)


def _attention(s):
    c = s["case"]
    if own:
        import kda_gated_delta_03_gb300 as kda
        o = kda.kda_attention_prefill(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"],
                                      scale=s["scale"], window=c["window"], sinks=c["sinks"], o=s["o"], lse=s["lse"])
        return {"o": o, "lse": s["lse"]}
    q, kp, vp, table, lens, cu = s["q"], s["k_pages"], s["v_pages"], s["table"].long(), s["lens"].long(), s["cu"].long()
    T, Hq, d = q.shape
    P, Hkv, ps, _ = kp.shape
    B, M = table.shape
    G, N, L = Hq // Hkv, c["n_max"], c["n_max"] + c["past_max"]
    i, t = torch.arange(N, device=q.device), torch.arange(L, device=q.device)
    n = cu[1:] - cu[:-1]
    real = i[None, :] < n[:, None]                                             # rows of the padded batch
    at = torch.where(real, cu[:-1, None] + i[None, :], T)
    pos = (lens - n)[:, None] + i[None, :]
    seen = (t <= pos[:, :, None]) & real[:, :, None]
    if c["window"]:
        seen = seen & ((t > pos[:, :, None] - c["window"]) | (t < c["sinks"]))
    flat = table.clamp(min=0).reshape(-1)
    held = (t < lens[:, None])[:, None, :, None]
    k = kp[flat].view(B, M, Hkv, ps, d).transpose(1, 2).reshape(B, Hkv, M * ps, d)[:, :, :L].float()
    x = q[at.clamp(max=T - 1)].view(B, N, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, d).float()
    w = torch.matmul(x, k.transpose(2, 3)).view(B, Hkv, G, N, L)
    del k
    w.mul_(s["scale"]).masked_fill_(~seen[:, None, None], float("-inf"))
    m = w.amax(4, keepdim=True)
    w = w.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = w.sum(4, keepdim=True)
    v = vp[flat].view(B, M, Hkv, ps, d).transpose(1, 2).reshape(B, Hkv, M * ps, d)[:, :, :L].float()
    v = torch.where(held, v, torch.zeros((), device=q.device))
    o = torch.matmul(w.view(B, Hkv, G * N, L), v).view(B, Hkv, G, N, d) / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.empty((T + 1, Hq, d), dtype=q.dtype, device=q.device)
    out[at] = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, d).to(q.dtype)
    lse = torch.empty((T + 1, Hq), device=q.device)
    lse[at] = (m + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(B, N, Hq)
    return {"o": out[:T], "lse": lse[:T]}


def _turned(x, angle, layout, stretch):
    """x [T, H, d], its first 2 n places rotated by angle [T, n] (64 bits), in 32 bits."""
    n = angle.shape[1]
    cos, sin = (stretch * torch.cos(angle)).float()[:, None], (stretch * torch.sin(angle)).float()[:, None]
    x = x.float()
    y = x.clone()
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :2 * n:2], x[..., 1:2 * n:2]
        y[..., :2 * n:2], y[..., 1:2 * n:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _append(s):
    c = s["case"]
    if own:
        import kda_gated_delta_03_gb300 as kda
        q = kda.kda_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], q=s["q"],
                                 inv_freq=s["inv_freq"], layout=c["layout"], rotary_scale=s["stretch"], q_out=s["q_out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    lens, cu = s["lens"].long(), s["cu"].long()
    T = s["k"].shape[0]
    token = torch.arange(T, device=lens.device)
    row = torch.searchsorted(cu[1:], token, right=True)
    pos = lens[row] - (cu[row + 1] - token)
    angle = pos.double()[:, None] * s["inv_freq"][None, :]
    page, slot = s["table"][row, pos // c["page"]].long(), pos % c["page"]
    s["k_pages"][page, :, slot] = _turned(s["k"], angle, c["layout"], s["stretch"]).to(s["k"].dtype)
    s["v_pages"][page, :, slot] = s["v"]
    s["q_out"].copy_(_turned(s["q"], angle, c["layout"], s["stretch"]))
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _rotary(s):
    c = s["case"]
    if own:
        import kda_gated_delta_03_gb300 as kda
        q, k = kda.kda_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], layout=c["layout"],
                              rotary_scale=s["stretch"], inverse=c["inverse"])
        return {"q": q, "k": k}
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :] * (-1 if c["inverse"] else 1)
    return {"q": _turned(s["q"], angle, c["layout"], s["stretch"]).to(s["q"].dtype),
            "k": _turned(s["k"], angle, c["layout"], s["stretch"]).to(s["k"].dtype)}


def _score(s):
    top = s["case"]["top"]
    if own:
        import kda_gated_delta_03_gb300 as kda
        r = kda.kda_token_logprobs(s["logits"], s["token"], top=top, entropy=True)
        return {"logp": r.logp, "lse": r.lse, "entropy": r.entropy, "top_logp": r.top_logp, "top_token": r.top_token}
    x = s["logits"].float()
    T, V = x.shape
    m = x.amax(1, keepdim=True)
    x_m = x - m
    e = torch.exp(x_m)
    # sums, and what is subtracted from them, in 64 bits: a likely word's log probability is next to zero
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    log_total = torch.log(total)
    y = s["token"].long()[:, None]
    logp = torch.where(y >= 0, x_m.gather(1, y.clamp(min=0)) - log_total, torch.zeros_like(log_total))
    inner = e.mul_(torch.where(e > 0, x_m, torch.zeros((), device=x.device)))
    entropy = log_total - inner.sum(1, keepdim=True, dtype=torch.float64) / total
    lse = m + log_total
    # the order of the values, then the lowest place among equal ones, as one whole number
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = order * (1 << 32) + ((1 << 32) - 1 - torch.arange(V, device=x.device))[None, :]
    at = (1 << 32) - 1 - (torch.topk(key, top, dim=1).values & ((1 << 32) - 1))
    return {"logp": logp[:, 0].float(), "lse": lse[:, 0].float(), "entropy": entropy[:, 0].float(),
            "top_logp": (x_m.gather(1, at) - log_total).float(), "top_token": at.int()}


def _score_grad(s):
    if own:
        import kda_gated_delta_03_gb300 as kda
        return {"g": kda.kda_token_logprobs_backward(s["logits"], s["token"], s["lse"], s["g_logp"],
                                                     entropy=s["entropy"], grad_entropy=s["g_entropy"])}
    x = s["logits"].float()
    y = s["token"].long()[:, None]
    lp = x - s["lse"][:, None]
    p = torch.exp(lp)
    real = (y >= 0).float()
    gl = s["g_logp"][:, None] * real
    g = -p * (gl + s["g_entropy"][:, None] * (torch.where(p > 0, lp, torch.zeros((), device=x.device)) + s["entropy"][:, None]))
    g.scatter_add_(1, y.clamp(min=0), gl)
    return {"g": g.to(s["logits"].dtype)}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_attention(c, s):
    T, Hq, d = s["q"].shape
    G, ps, cu = Hq // c["Hkv"], c["page"], s["cu"].tolist()
    o = torch.zeros((T, Hq, d), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    for b in range(c["B"]):
        n, end = cu[b + 1] - cu[b], int(s["lens"][b])
        if n == 0:
            continue
        pages = s["table"][b, : -(-end // ps)].long()
        for h in range(c["Hkv"]):
            K = s["k_pages"][pages, h].reshape(-1, d)[:end].double()
            W = s["v_pages"][pages, h].reshape(-1, d)[:end].double()
            for g in range(h * G, (h + 1) * G):
                a = (s["q"][cu[b]:cu[b + 1], g].double() @ K.T) * s["scale"]
                query = torch.arange(end - n, end, device=DEV)[:, None]
                key = torch.arange(end, device=DEV)[None, :]
                hidden = key > query
                if c["window"]:
                    hidden |= (query - key >= c["window"]) & (key >= c["sinks"])
                a.masked_fill_(hidden, -math.inf)
                r = torch.logsumexp(a, 1)
                lse[cu[b]:cu[b + 1], g] = r.cpu()
                o[cu[b]:cu[b + 1], g] = (torch.exp_(a.sub_(r[:, None])) @ W).cpu()
    return {"o": o, "lse": lse}


def _exact_turn(x, pos, s, c, sign=1.0):
    n = c["rot"] // 2
    if n == 0:
        return x.double()
    turn = torch.polar(torch.full((1, n), float(s["stretch"]), dtype=torch.float64, device=DEV),
                       torch.zeros((1, n), dtype=torch.float64, device=DEV))
    turn = turn * torch.exp(1j * sign * torch.outer(pos.double(), s["inv_freq"]))
    y = x.double()
    head = y[..., : 2 * n]
    pairs = head.unflatten(-1, (2, n)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (n, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    z = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
    return torch.cat([z, y[..., 2 * n:]], -1)


def exact(c, seed):
    """The computed outputs in 64 bits; nothing for what is only moved or chosen."""
    s = prepare(c, seed)
    if c["kind"] == "attention":
        return _exact_attention(c, s)
    if c["kind"] == "append":
        cu, lens = s["cu"].tolist(), s["lens"].tolist()
        where = [(b, lens[b] - cu[b + 1] + j) for b in range(c["B"]) for j in range(cu[b], cu[b + 1])]
        if not where:
            return None
        where = torch.tensor(where, device=DEV)
        row, pos = where[:, 0], where[:, 1]
        k = s["k_pages"].double()
        k[s["table"][row, pos // c["page"]].long(), :, pos % c["page"]] = _exact_turn(s["k"], pos, s, c)
        return {"q": _exact_turn(s["q"], pos, s, c), "k_pages": k, "v_pages": None}
    if c["kind"] == "rotary":
        sign = -1.0 if c["inverse"] else 1.0
        return {n: _exact_turn(s[n], s["positions"], s, c, sign) for n in ("q", "k")}
    logp = s["logits"].double()
    y = s["token"].long().clamp(min=0)[:, None]
    scored = s["token"] >= 0
    if c["kind"] == "score":
        lse = torch.logsumexp(logp, 1)
        logp -= lse[:, None]
        entropy = torch.special.entr(torch.exp(logp)).sum(1)
        best = torch.topk(logp, c["top"], 1).values
        return {"logp": torch.where(scored, logp.gather(1, y)[:, 0], 0.0), "lse": lse, "entropy": entropy,
                "top_logp": best, "top_token": None}
    logp -= s["lse"].double()[:, None]
    p = torch.exp(logp)
    g = s["g_entropy"].double()[:, None] * (torch.special.entr(p) - p * s["entropy"].double()[:, None])
    gl = torch.where(scored, s["g_logp"].double(), 0.0)[:, None]
    g -= gl * p
    return {"g": g.scatter_add_(1, y, gl)}
