"""Cases and plain forms of the decoding operators of a hybrid stack (KDA layers and full-attention layers).

Four kinds of case, each one call of the library:

* ``attention``: attention of one new token per sequence over a paged key-value cache
  (``kda_attention_decode``), with the new token's key and value written into its page by the same call.
* ``select``: a beam search's selection over beams and vocabulary (``kda_beam_select``).
* ``states``: the KDA states of the chosen beams brought into their slots (``kda_state_fork``).
* ``fork`` and ``compact``: pages of the key-value cache shared, copied, freed and handed out for a batch's
  next rows (``kda_cache_fork``), and live pages moved together at the low end of their pools
  (``kda_cache_compact``).

``own`` false computes a case with elementary torch operations in 32 bits; ``own`` true calls the library.
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
        # one user's chat a few tokens in: only the latency of the call counts
        dict(name="attention_one_short", kind="attention", B=1, Hq=32, Hkv=8, d=128, page=16, len_min=37, len_max=37,
             window=0, sinks=0, dtype="bf16"),
        # a serving batch of 64 sequences of very different lengths (log-uniform, as the packed prefill workload)
        dict(name="attention_batch_ragged", kind="attention", B=64, Hq=32, Hkv=8, d=128, page=64, len_min=128,
             len_max=16384, window=0, sinks=0, dtype="bf16"),
        # one agent's context of about a million tokens with 8 heads, as the append workload has
        dict(name="attention_one_1m", kind="attention", B=1, Hq=8, Hkv=8, d=128, page=256, len_min=1048573,
             len_max=1048573, window=0, sinks=0, dtype="bf16"),
        # a parity run in fp32 on sliding-window layers, with a page size that is no power of two and an idle slot
        dict(name="attention_f32_window", kind="attention", B=48, Hq=16, Hkv=4, d=64, page=24, len_min=1, len_max=8000,
             window=2000, sinks=4, dtype="f32"),
        # one request with four beams and a small odd vocabulary
        dict(name="select_one", kind="select", N=1, K=4, V=32001, dtype="f32", done=0),
        # 64 requests with eight beams each, some beams at their end
        dict(name="select_batch", kind="select", N=64, K=8, V=131072, dtype="bf16", done=1),
        # one request's four beams on a small model's states, kept in bf16
        dict(name="states_one", kind="states", N=1, K=4, alive=3, L=2, H=8, d=64, dtype="bf16"),
        # 512 resident fp32 states of 32 heads (the decode workload) used as 64 requests with eight beams each
        dict(name="states_batch", kind="states", N=64, K=8, alive=5, L=1, H=32, d=128, dtype="f32"),
        # one request's four beams after a step: a few pages of bookkeeping, one page copied
        dict(name="fork_one", kind="fork", N=1, K=4, alive=3, L=2, Hkv=2, d=64, page=16, len_min=500, len_max=500,
             dtype="bf16"),
        # 64 requests with four beams each on eight attention layers, after a step
        dict(name="fork_batch", kind="fork", N=64, K=4, alive=2, L=8, Hkv=8, d=128, page=16, len_min=100,
             len_max=6000, dtype="bf16"),
        # a small pool that has become sparse
        dict(name="compact_small", kind="compact", R=16, L=2, Hkv=2, d=64, page=16, pages=600, live=190, dtype="f32"),
        # a large pool brought together before its upper part is given back
        dict(name="compact_large", kind="compact", R=200, L=2, Hkv=8, d=128, page=16, pages=16384, live=8192,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges, at most as much work as the largest of them."""
    kind = rng.choice(["attention", "attention", "attention", "select", "select", "states", "fork", "compact"])
    if kind == "attention":
        while True:
            group, Hkv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 24]), rng.choice([1, 2, 3, 4, 8, 16])
            d = rng.choice([16, 64, 128, 128])
            dtype = rng.choice(["bf16", "bf16", "f32"])
            hi = _log(rng, 2, 400000)
            c = dict(kind=kind, B=_log(rng, 1, 400), Hq=group * Hkv, Hkv=Hkv, d=d,
                     page=rng.choice([1, 7, 16, 16, 24, 32, 64, 64, 100, 128, 256]),
                     len_min=max(1, hi // rng.choice([1, 2, 10, 100])), len_max=hi, window=0, sinks=0, dtype=dtype)
            if rng.random() < 0.35:
                c["window"], c["sinks"] = _log(rng, 1, 5000), rng.choice([0, 1, 4, 61])
            # the plain form lays the cache out densely in 32 bits: both bound what a case may cost
            if c["B"] * hi * Hkv * d <= 1 << 30 and c["B"] * hi * c["Hq"] <= 1 << 28:
                return c
    if kind == "select":
        while True:
            c = dict(kind=kind, N=_log(rng, 1, 200), K=rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), V=_log(rng, 50, 260000),
                     dtype=rng.choice(["bf16", "f32"]), done=rng.choice([0, 1]))
            if c["N"] * c["K"] * c["V"] <= 64 * 8 * 131072:
                return c
    if kind == "states":
        while True:
            K = rng.choice([2, 3, 4, 5, 8])
            c = dict(kind=kind, N=_log(rng, 1, 200), K=K, alive=rng.randint(1, K), L=rng.choice([1, 2, 3]),
                     H=rng.choice([1, 2, 8, 15, 32]), d=rng.choice([16, 64, 128]), dtype=rng.choice(["bf16", "f32"]))
            if c["N"] * K * c["L"] * c["H"] * c["d"] ** 2 * ESIZE[c["dtype"]] <= 1 << 30:
                return c
    if kind == "fork":
        while True:
            K, hi = rng.choice([1, 2, 3, 4, 8]), _log(rng, 20, 30000)
            c = dict(kind=kind, N=_log(rng, 1, 128), K=K, alive=rng.randint(1, K), L=rng.choice([1, 2, 8]),
                     Hkv=rng.choice([1, 2, 3, 8]), d=rng.choice([16, 64, 128]), page=rng.choice([1, 7, 16, 24, 64, 256]),
                     len_min=max(1, hi // rng.choice([1, 3, 30])), len_max=hi, dtype=rng.choice(["bf16", "f32"]))
            if _fork_pages(c) * c["L"] * 2 * _page_bytes(c) <= 4 << 30 and _fork_pages(c) <= 1 << 20:
                return c
    while True:
        pages = _log(rng, 40, 60000)
        c = dict(kind=kind, R=_log(rng, 1, 300), L=rng.choice([1, 2, 4]), Hkv=rng.choice([1, 2, 3, 8]),
                 d=rng.choice([16, 64, 128]), page=rng.choice([1, 7, 16, 24, 64]), pages=pages,
                 live=max(1, int(pages * rng.uniform(0.05, 0.95))), dtype=rng.choice(["bf16", "f32"]))
        if pages * c["L"] * 2 * _page_bytes(c) <= 2 << 30:
            return c


def _page_bytes(c):
    return c["Hkv"] * c["page"] * c["d"] * ESIZE[c["dtype"]]


def _fork_pages(c):
    """Pages of a fork case's pools: every beam's own pages at full length, and some to spare."""
    per_row = c["len_max"] // c["page"] + 2
    return c["N"] * c["K"] * per_row + 64


def _lens(c, n):
    """n lengths spread log-uniformly over the case's range (the same ones for every seed, which orders them)."""
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    lens = torch.exp(math.log(c["len_min"]) + u * (math.log(c["len_max"]) - math.log(c["len_min"]))).round().long()
    return lens.clamp(c["len_min"], c["len_max"])


def _attention_lens(c):
    lens = _lens(c, c["B"])
    if c["B"] >= 8:
        lens[c["B"] // 2] = 0                             # an idle slot of the batch
    return lens


def work(c):
    kind = c["kind"]
    if kind == "attention":
        e, lens = ESIZE[c["dtype"]], _attention_lens(c)
        vis = int((lens.clamp(max=c["window"] + c["sinks"]) if c["window"] else lens).sum())
        return {"bytes": vis * c["Hkv"] * c["d"] * 2 * e + c["B"] * (2 * c["Hq"] + 4 * c["Hkv"]) * c["d"] * e +
                vis / c["page"] * 4, "flops": 4.0 * vis * c["Hq"] * c["d"]}
    if kind == "select":
        n = c["N"] * c["K"]
        live = n * (1 - 0.2 * c["done"]) * c["V"]
        return {"bytes": live * ESIZE[c["dtype"]] + n * 18, "flops": 4.0 * live}
    if kind == "states":
        copies = c["N"] * (c["K"] - c["alive"])
        return {"bytes": 2.0 * copies * c["L"] * c["H"] * c["d"] ** 2 * ESIZE[c["dtype"]] + c["N"] * c["K"] * 12,
                "flops": 0}
    if kind == "fork":
        lens = _lens(c, c["N"])
        copies = (c["K"] - c["alive"]) * int((lens % c["page"] != 0).sum())      # a length at a page's end needs none
        return {"bytes": 2.0 * copies * 2 * c["L"] * _page_bytes(c) + c["K"] * int(lens.sum()) / c["page"] * 8 +
                c["N"] * c["K"] * 16 + _fork_pages(c) * 8, "flops": 0}
    moves = c["live"] * (1 - c["live"] / c["pages"])
    return {"bytes": 2.0 * moves * 2 * c["L"] * _page_bytes(c) + c["live"] * 8 + c["pages"] * 12, "flops": 0}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(shape, dtype, gen, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=gen)


def _bits(t):
    """The stored bits of a tensor as whole numbers: what is moved has to arrive unchanged."""
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def prepare(c, seed):
    cpu = torch.Generator().manual_seed(1000003 * seed + 17)
    gpu = torch.Generator(device=DEV).manual_seed(1000003 * seed + 18)
    return dict({"attention": _prepare_attention, "select": _prepare_select, "states": _prepare_states,
                 "fork": _prepare_fork, "compact": _prepare_compact}[c["kind"]](c, cpu, gpu), case=dict(c))


def _prepare_attention(c, cpu, gpu):
    B, Hq, Hkv, d, ps, dt = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], DT[c["dtype"]]
    lens = _attention_lens(c)[torch.randperm(B, generator=cpu)]
    M = max(1, -(-c["len_max"] // ps))
    counts = -(-lens // ps)
    total = int(counts.sum())
    P = total + 3
    perm = torch.randperm(P, generator=cpu)[:total].int()
    table = torch.full((B, M), -1, dtype=torch.int32)
    col = torch.arange(M)[None, :].expand(B, M)
    table[col < counts[:, None]] = perm                   # pages of a row lie anywhere in the pool
    s = dict(q=_randn((B, Hq, d), dt, gpu, 1.5), k_pages=_randn((P, Hkv, ps, d), dt, gpu),
             v_pages=_randn((P, Hkv, ps, d), dt, gpu), k_new=_randn((B, Hkv, d), dt, gpu),
             v_new=_randn((B, Hkv, d), dt, gpu), table=table.to(DEV), lens=lens.int().to(DEV), scale=d ** -0.5,
             o=torch.empty((B, Hq, d), dtype=dt, device=DEV))
    s["k_bits"], s["v_bits"] = _bits(s["k_pages"]), _bits(s["v_pages"])
    # what lies in the pools past a row's end is left from earlier owners: not numbers anybody may read
    used = (torch.arange(M * ps)[None, :] < lens[:, None]).view(B, M, ps)
    tail = (used.any(2) & ~used.all(2)).nonzero()
    for b, m in tail.tolist()[:4]:
        p, n = int(table[b, m]), int(lens[b]) - m * ps
        s["k_pages"][p, :, n:] = float("nan")
        s["v_pages"][p, :, n:] = float("inf")
    if own:
        import kda_gated_delta_03_gb300 as kda
        n = kda.kda_attention_decode_workspace_size(B, Hq, Hkv, d, dt)
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return s


def _prepare_select(c, cpu, gpu):
    N, K, V = c["N"], c["K"], c["V"]
    logits = _randn((N * K, V), DT[c["dtype"]], gpu, 2.5)
    hot = torch.randint(0, V, (N * K, 12), generator=cpu).to(DEV)              # a few likely words stand out
    logits.scatter_add_(1, hot, _randn((N * K, 12), DT[c["dtype"]], gpu, 4.0).abs())
    if V >= 200:
        logits[:, 3] = float("-inf")                                           # a word that is not allowed here
    scores = (-30.0 * torch.rand((N, K), generator=cpu)).sort(1, descending=True).values
    done = (torch.rand((N, K), generator=cpu) < 0.2) if c["done"] else torch.zeros((N, K), dtype=torch.bool)
    s = dict(logits=logits, scores=scores.to(DEV), done=done.to(torch.uint8).to(DEV), eos=min(2, V - 1),
             scores_out=torch.empty((N, K), device=DEV), parent=torch.empty((N, K), dtype=torch.int32, device=DEV),
             token=torch.empty((N, K), dtype=torch.int32, device=DEV),
             done_out=torch.empty((N, K), dtype=torch.uint8, device=DEV))
    if own:
        import kda_gated_delta_03_gb300 as kda
        n = kda.kda_beam_select_workspace_size(N, K, V, DT[c["dtype"]])
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return s


def _parents(N, K, alive, gen):
    """Parents (row numbers) of every row: in each group of K rows, `alive` of them go on, the others are dropped."""
    keep = torch.rand((N, K), generator=gen).argsort(1)[:, :alive]
    extra = torch.randint(0, alive, (N, K - alive), generator=gen)
    order = torch.rand((N, K), generator=gen).argsort(1)
    chosen = torch.cat([keep, keep.gather(1, extra)], 1).gather(1, order)
    return (chosen + torch.arange(N)[:, None] * K).reshape(-1).int()


def _prepare_states(c, cpu, gpu):
    B = c["N"] * c["K"]
    S = B + 2
    pool = _randn((c["L"], S, c["H"], c["d"], c["d"]), DT[c["dtype"]], gpu, 0.02)
    return dict(pool=pool, bits=_bits(pool),
                idx=torch.randperm(S, generator=cpu)[:B].int().to(DEV),
                parent=_parents(c["N"], c["K"], c["alive"], cpu).to(DEV),
                idx_out=torch.empty(B, dtype=torch.int32, device=DEV))


def _prepare_fork(c, cpu, gpu):
    N, K, ps = c["N"], c["K"], c["page"]
    R, P = N * K, _fork_pages(c)
    M = c["len_max"] // ps + 2
    lens = _lens(c, N)[torch.randperm(N, generator=cpu)].repeat_interleave(K)
    prompt = (lens // 2) // ps                                                 # pages that a group's beams share
    counts = -(-lens // ps)
    perm = torch.randperm(P, generator=cpu)
    col = torch.arange(M)[None, :]
    first = (torch.arange(R) // K * K)
    ids = perm[: R * M].view(R, M) if P >= R * M else perm[(torch.arange(R * M) % P)].view(R, M)
    table = torch.where(col < prompt[:, None], ids[first], ids)
    table = torch.where(col < counts[:, None], table, torch.full_like(table, -1)).int()
    ref = torch.bincount(table[table >= 0].long(), minlength=P).int()
    k = _randn((c["L"], P, c["Hkv"], ps, c["d"]), DT[c["dtype"]], gpu)
    v = _randn((c["L"], P, c["Hkv"], ps, c["d"]), DT[c["dtype"]], gpu)
    s = dict(table=table.to(DEV), lens=lens.int().to(DEV), ref=ref.to(DEV), k=k, v=v, k_bits=_bits(k), v_bits=_bits(v),
             parent=_parents(N, K, c["alive"], cpu).to(DEV), grow=torch.ones(R, dtype=torch.int32, device=DEV),
             table_out=torch.empty((R, M), dtype=torch.int32, device=DEV),
             lens_out=torch.empty(R, dtype=torch.int32, device=DEV), ref_out=torch.empty(P, dtype=torch.int32, device=DEV))
    if own:
        import kda_gated_delta_03_gb300 as kda
        n = kda.kda_cache_fork_workspace_size(R, R, M, P)
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return s


def _prepare_compact(c, cpu, gpu):
    R, P, live, ps = c["R"], c["pages"], c["live"], c["page"]
    ids = torch.randperm(P, generator=cpu)[:live].int()
    M = -(-live // R)
    table = torch.full((R * M,), -1, dtype=torch.int32)
    table[:live] = ids
    ref = torch.zeros(P, dtype=torch.int32)
    ref[ids.long()] = torch.randint(1, 5, (live,), generator=cpu).int()        # other tables may hold a page too
    k = _randn((c["L"], P, c["Hkv"], ps, c["d"]), DT[c["dtype"]], gpu)
    v = _randn((c["L"], P, c["Hkv"], ps, c["d"]), DT[c["dtype"]], gpu)
    s = dict(table=table.view(R, M).to(DEV), ref=ref.to(DEV), k=k, v=v, k_bits=_bits(k), v_bits=_bits(v),
             table_out=torch.empty((R, M), dtype=torch.int32, device=DEV),
             ref_out=torch.empty(P, dtype=torch.int32, device=DEV), page_map=torch.empty(P, dtype=torch.int32, device=DEV))
    if own:
        import kda_gated_delta_03_gb300 as kda
        n = kda.kda_cache_compact_workspace_size(P)
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    return {"attention": _attention, "select": _select, "states": _states, "fork": _fork,
            "compact": _compact}[s["case"]["kind"]](s)


def _attention(s):
    c = s["case"]
    if own:
        import kda_gated_delta_03_gb300 as kda
        o = kda.kda_attention_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], scale=s["scale"],
                                     window=c["window"], sinks=c["sinks"], k_new=s["k_new"], v_new=s["v_new"],
                                     o=s["o"], workspace=s["workspace"])
    else:
        o = _attention_plain(s, c)
    return {"o": o, "k_pages": s["k_bits"], "v_pages": s["v_bits"]}


def _attention_plain(s, c):
    q, kp, vp, table, lens = s["q"], s["k_pages"], s["v_pages"], s["table"].long(), s["lens"].long()
    B, Hq, d = q.shape
    P, Hkv, ps, _ = kp.shape
    M, G = table.shape[1], Hq // Hkv
    # the new token's key and value into the last place of each row that has one
    rows = torch.arange(B, device=q.device)
    at = (lens - 1).clamp(min=0)
    page, slot, has = table[rows, at // ps].clamp(min=0), at % ps, (lens > 0)[:, None, None]
    kp[page, :, slot] = torch.where(has, s["k_new"], kp[page, :, slot])
    vp[page, :, slot] = torch.where(has, s["v_new"], vp[page, :, slot])
    t = torch.arange(M * ps, device=q.device)
    seen = t[None, :] < lens[:, None]
    if c["window"]:
        seen = seen & ((t[None, :] >= lens[:, None] - c["window"]) | (t[None, :] < c["sinks"]))
    flat = table.clamp(min=0).reshape(-1)
    k = kp[flat].view(B, M, Hkv, ps, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * ps, d).float()
    w = torch.matmul(q.float().view(B, Hkv, G, d), k.transpose(2, 3)) * s["scale"]
    del k
    seen = seen[:, None, None, :]
    w = torch.where(seen, w, torch.full((), float("-inf"), device=q.device))
    m = w.amax(3, keepdim=True)
    w = torch.exp(w - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = w.sum(3, keepdim=True)
    v = vp[flat].view(B, M, Hkv, ps, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * ps, d).float()
    v = torch.where(seen[:, :, 0, :, None], v, torch.zeros((), device=q.device))
    o = torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, Hq, d).to(q.dtype)


def _select(s):
    if own:
        import kda_gated_delta_03_gb300 as kda
        scores, parent, token, done = kda.kda_beam_select(
            s["logits"], s["scores"], finished=s["done"], eos_token=s["eos"], scores_out=s["scores_out"],
            parent=s["parent"], token=s["token"], finished_out=s["done_out"], workspace=s["workspace"])
        return {"scores": scores, "parent": parent, "token": token, "done": done}
    N, K = s["scores"].shape
    V = s["logits"].shape[1]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    score = s["scores"].view(N * K, 1) + (x - lse)
    done = s["done"].view(N * K, 1) != 0
    is_eos = torch.arange(V, device=x.device)[None, :] == s["eos"]
    kept = torch.where(is_eos, s["scores"].view(N * K, 1), torch.full((), float("-inf"), device=x.device))
    score = torch.where(done, kept, score)
    score = torch.where(torch.isnan(score), torch.full((), float("-inf"), device=x.device), score) + 0.0
    # the order of the values, then the lowest place among equal ones, as one whole number
    bits = score.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long().view(N, K * V)
    key = order * (1 << 32) + ((1 << 32) - 1 - torch.arange(K * V, device=x.device))[None, :]
    at = (1 << 32) - 1 - (torch.topk(key, K, dim=1).values & ((1 << 32) - 1))
    beam, token = at // V, at % V
    parent = beam + torch.arange(N, device=x.device)[:, None] * K
    out = (s["done"].gather(1, beam) != 0) | (token == s["eos"])
    return {"scores": score.view(N, K * V).gather(1, at), "parent": parent.int(), "token": token.int(),
            "done": out.to(torch.uint8)}


def _states(s):
    if own:
        import kda_gated_delta_03_gb300 as kda
        idx = kda.kda_state_fork(s["pool"], s["idx"], s["parent"], state_idx_out=s["idx_out"])
        return {"idx": idx, "pool": s["bits"]}
    idx, parent, pool = s["idx"].long(), s["parent"].long(), s["pool"]
    B = idx.shape[0]
    row = torch.arange(B, device=idx.device)
    first = torch.full((B,), B, device=idx.device).scatter_reduce(0, parent, row, "amin")
    keeps = first[parent] == row                                   # a parent's first child stays where the parent is
    free = idx[(first == B).nonzero()[:, 0]]                       # slots of the rows that nobody continues
    out = torch.where(keeps, idx[parent], free[(torch.cumsum(~keeps, 0) - 1).clamp(0, max(free.numel() - 1, 0))]
                      if free.numel() else idx[parent])
    src, dst = idx[parent][~keeps], out[~keeps]
    pool[:, dst] = pool[:, src]
    s["idx_out"].copy_(out)
    return {"idx": s["idx_out"], "pool": s["bits"]}


def _fork(s):
    ps = s["case"]["page"]
    if own:
        import kda_gated_delta_03_gb300 as kda
        kda.kda_cache_fork(s["table"], s["lens"], s["parent"], s["ref"], ps, grow=s["grow"], pools=(s["k"], s["v"]),
                           block_table_out=s["table_out"], seq_lens_out=s["lens_out"], ref_count_out=s["ref_out"],
                           workspace=s["workspace"])
        return {"table": s["table_out"], "lens": s["lens_out"], "ref": s["ref_out"], "k": s["k_bits"],
                "v": s["v_bits"]}
    table, lens, parent, ref = s["table"].long(), s["lens"].long(), s["parent"].long(), s["ref"].long()
    R, M = table.shape
    P = ref.shape[0]
    row = torch.arange(R, device=table.device)
    col = torch.arange(M, device=table.device)[None, :]
    first = torch.full((R,), R, device=table.device).scatter_reduce(0, parent, row, "amin")
    old, tail = lens[parent], lens[parent] % ps
    new = old + s["grow"].long()
    copies = (tail > 0) & (first[parent] != row)                   # this row's last page is another row's already
    shared = torch.where(copies, old // ps, -(-old // ps))         # pages taken over as they are
    need = -(-new // ps)
    out = torch.where(col < shared[:, None], table[parent], torch.full((), -1, device=table.device))
    held = col < (-(-lens // ps))[:, None]
    ref = ref - torch.bincount(table[held], minlength=P) + torch.bincount(out[out >= 0], minlength=P)
    fresh = (col >= shared[:, None]) & (col < need[:, None])
    pages = (ref == 0).nonzero()[:, 0][: int(fresh.sum())]
    out[fresh] = pages
    ref[pages] = 1
    src = table[parent[copies], old[copies] // ps]
    dst = out[copies, old[copies] // ps]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    s["table_out"].copy_(out)
    s["lens_out"].copy_(new)
    s["ref_out"].copy_(ref)
    return {"table": s["table_out"], "lens": s["lens_out"], "ref": s["ref_out"], "k": s["k_bits"],
            "v": s["v_bits"]}


def _compact(s):
    if own:
        import kda_gated_delta_03_gb300 as kda
        kda.kda_cache_compact(s["table"], s["ref"], pools=(s["k"], s["v"]), block_table_out=s["table_out"],
                              ref_count_out=s["ref_out"], page_map=s["page_map"], workspace=s["workspace"])
    else:
        ref = s["ref"]
        P = ref.shape[0]
        page = torch.arange(P, device=ref.device)
        live = ref > 0
        n = live.sum()
        moved = (live & (page >= n)).nonzero()[:, 0]
        holes = (~live & (page < n)).nonzero()[:, 0]
        where = torch.where(live, page, torch.full((), -1, device=ref.device))
        where[moved] = holes
        s["k"][:, holes] = s["k"][:, moved]
        s["v"][:, holes] = s["v"][:, moved]
        s["ref_out"].zero_()
        s["ref_out"][where[live]] = ref[live]
        s["page_map"].copy_(where)
        t = s["table"].long()
        s["table_out"].copy_(torch.where(t >= 0, where[t.clamp(min=0)], torch.full((), -1, device=ref.device)))
    return {"table": s["table_out"], "ref": s["ref_out"], "map": s["page_map"], "k": s["k_bits"], "v": s["v_bits"]}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(c, seed):
    """The computed outputs in 64 bits; nothing for what is only moved or chosen."""
    if c["kind"] == "attention":
        s = prepare(c, seed)
        o = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64)
        for b in range(c["B"]):
            n = int(s["lens"][b])
            if n == 0:
                continue
            pages = s["table"][b, : -(-n // c["page"])].long()
            for h in range(c["Hkv"]):
                K = s["k_pages"][pages, h].reshape(-1, c["d"])[:n].double()
                W = s["v_pages"][pages, h].reshape(-1, c["d"])[:n].double()
                K[n - 1], W[n - 1] = s["k_new"][b, h].double(), s["v_new"][b, h].double()
                if c["window"] and n > c["window"] + c["sinks"]:
                    keep = list(range(c["sinks"])) + list(range(n - c["window"], n))
                    keep = torch.tensor(keep, device=K.device)
                    K, W = K[keep], W[keep]
                g = c["Hq"] // c["Hkv"]
                a = (s["q"][b, h * g:(h + 1) * g].double() @ K.T) * s["scale"]
                o[b, h * g:(h + 1) * g] = (torch.softmax(a, 1) @ W).cpu()
        return {"o": o, "k_pages": None, "v_pages": None}
    if c["kind"] == "select":
        s = prepare(c, seed)
        logp = torch.log_softmax(s["logits"].double(), 1).view(c["N"], c["K"], c["V"])
        logp = s["scores"].double()[:, :, None] + logp
        for n, b in (s["done"] != 0).nonzero().tolist():
            logp[n, b] = float("-inf")
            logp[n, b, s["eos"]] = s["scores"][n, b].double()
        return {"scores": torch.topk(logp.view(c["N"], -1), c["K"], 1).values, "parent": None, "token": None,
                "done": None}
    return None
