"""kda_attention_prefill against softmax attention in float64, over the chunk sizes, contexts, masks and page layouts where
a paged, split kernel can go wrong.

Tolerances, relative Frobenius: the bf16 output is rounded once (at most 2^-8 of a value, 2^-8 / sqrt(12) * 1.44 = 1.7e-3 in
the mean over a binade) and the weights before it once each (the same, divided by the square root of the weights' number
and at most as much again for a row of one: 2.4e-3 together), so 3e-3; the fp32 path sums up to 10,000 terms of
random sign in fp32 (2^-24 a step, growing with the square root: below 1e-5).  A single row of d values may be twice as
far off."""

import math

import numpy as np
import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 3e-3, "f32": 1e-5}
DEV = "cuda:0"


def make(rows, Hq, Hkv, d, ps, dtype, seed, extra_pages=3, max_pages=None, qstd=1.5, interleaved=False, behind=0):
    """rows: (new tokens, tokens in the cache before them) of each sequence; `behind` tokens after the last one."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, dt = len(rows), DT[dtype]
    lens = [n + past for n, past in rows]
    counts = [-(-n // ps) for n in lens]
    M = max_pages if max_pages is not None else max([1] + counts)
    P = sum(counts) + extra_pages
    perm = rng.permutation(P)
    table = np.full((B, M), -1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    if interleaved:                                    # keys and values of a page next to each other
        pool = torch.randn((P, 2, Hkv, ps, d), device=DEV, generator=g).to(dt)
        k, v = pool[:, 0], pool[:, 1]
    else:
        k = torch.randn((P, Hkv, ps, d), device=DEV, generator=g).to(dt)
        v = torch.randn((P, Hkv, ps, d), device=DEV, generator=g).to(dt)
    used = np.zeros((P, ps), bool)
    for b, n in enumerate(lens):
        for j in range(counts[b]):
            used[table[b, j], :min(ps, n - j * ps)] = True
    stale = torch.from_numpy(~used).to(DEV)[:, None, :, None]
    k.masked_fill_(stale, float("nan"))                # what earlier owners left is never used
    v.masked_fill_(stale, float("inf"))
    cu = np.concatenate([[0], np.cumsum([n for n, _ in rows])]).astype(np.int32)
    q = (qstd * torch.randn((int(cu[-1]) + behind, Hq, d), device=DEV, generator=g)).to(dt)
    return dict(q=q, k_pages=k, v_pages=v, block_table=torch.from_numpy(table).to(DEV),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=torch.from_numpy(cu).to(DEV))


def reference(t, rows, ps, scale, window=0, sinks=0):
    """o, lse in float64, sequence by sequence."""
    T, Hq, d = t["q"].shape
    Hkv = t["k_pages"].shape[1]
    o = torch.zeros((T, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -float("inf"), dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, past) in enumerate(rows):
        if n:
            end = n + past
            pages = t["block_table"][b, :-(-end // ps)].long()
            i, j = torch.arange(past, end, device=DEV)[:, None], torch.arange(end, device=DEV)[None, :]
            hidden = j > i
            if window:
                hidden = hidden | ((j <= i - window) & (j >= sinks))
            k = t["k_pages"][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :end].double()
            v = t["v_pages"][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :end].double()
            q = t["q"][at:at + n].double().view(n, Hkv, Hq // Hkv, d)
            s = torch.einsum("thgd,hjd->hgtj", q, k) * scale
            s.masked_fill_(hidden, -float("inf"))
            o[at:at + n] = torch.einsum("hgtj,hjd->thgd", torch.softmax(s, 3), v).reshape(n, Hq, d)
            lse[at:at + n] = torch.logsumexp(s, 3).permute(2, 0, 1).reshape(n, Hq)
        at += n
    return o, lse


def rel(x, ref):
    return float((x.double() - ref).norm() / ref.norm().clamp(min=1e-300))


def check(rows, Hq, Hkv, d, ps, dtype, seed=0, window=0, sinks=0, scale=None, **kw):
    t = make(rows, Hq, Hkv, d, ps, dtype, seed, **kw)
    scale = d ** -0.5 if scale is None else scale
    ref, ref_lse = reference(t, rows, ps, scale, window, sinks)
    T, behind = int(t["cu_seqlens"][-1]), kw.get("behind", 0)
    lse = torch.full((T + behind, Hq), 7.0, device=DEV)
    o = torch.full_like(t["q"], 7.0)
    got = kda.kda_attention_prefill(**t, scale=scale, window=window, sinks=sinks, o=o, lse=lse)
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    assert got.data_ptr() == o.data_ptr() and bool(torch.isfinite(o).all())
    assert bool((o[T:] == 7).all()) and bool((lse[T:] == 7).all())        # tokens of no sequence
    o, ref, lse, ref_lse = o[:T], ref[:T], lse[:T], ref_lse[:T]
    assert rel(o, ref) <= TOL[dtype], rel(o, ref)
    per = (o.double() - ref).norm(dim=2) / ref.norm(dim=2)                # no row hides behind the others
    # A score is a sum of d products in fp32: off by sqrt(d) roundings of its size, which its weight is off by then.  With
    # delta for that, o = sum p v moves by sum p delta (v - o), at most 2 delta |v|: for the scores of 200 and more that
    # peaked rows have (lse is the largest) this is above what the sums themselves lose.
    delta = math.sqrt(d) * 2.0 ** -24 * float(ref_lse[torch.isfinite(ref_lse)].abs().max())
    assert float(per.max()) <= 2 * TOL[dtype] + 2 * delta, (per.max(), int(per.argmax()) // Hq, int(per.argmax()) % Hq)
    assert float((lse.double() - ref_lse).abs().max()) <= 1e-4
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_lengths_around_tiles_and_pages(dtype, d):
    check([(1, 0), (0, 5), (2, 0), (15, 1), (16, 0), (17, 47), (63, 1), (64, 64), (65, 63), (127, 0), (1, 127), (128, 1),
           (1, 128), (129, 300), (3, 509), (200, 55), (257, 0), (0, 0)], 8, 2, d, 16, dtype, seed=d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (6, 3), (3, 1), (32, 8), (5, 1), (16, 2), (9, 1), (12, 1), (17, 1), (40, 1),
                                   (130, 1), (300, 1)])
def test_head_layouts(dtype, heads):
    check([(70, 10), (1, 128), (5, 0), (33, 270)], *heads, 64, 32, dtype, seed=heads[0])
    check([(130, 130), (3, 30)], *heads, 128, 16, dtype, seed=heads[1] + 50)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ps", [1, 3, 7, 16, 24, 48, 64, 100, 128, 131, 256, 1000])
def test_page_sizes(dtype, ps):
    check([(1, 0), (99, 200), (40, 600), (201, 800)], 4, 2, 64, ps, dtype, seed=ps)
    check([(140, 23)], 2, 2, 128, ps, dtype, seed=ps + 1)


@pytest.mark.parametrize("ps", [2, 5, 9, 65, 66, 67, 71, 77, 90, 94, 127, 134, 201, 469])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_of_few_divisors(d, ps):
    """Tiles of less than 128 tokens, in one box or several."""
    check([(1, 0), (99, 200), (40, 600), (256, 801)], 4, 2, d, ps, "bf16", seed=ps)
    check([(99, 200), (300, 701), (1, 5000)], 2, 2, d, ps, "bf16", seed=ps + 1, window=150, sinks=70)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (64, 64), (100, 4), (300, 70), (2000, 4), (129, 500),
                                          (2 ** 31 - 1, 0), (7, 2 ** 31 - 1)])
def test_window_and_sinks(dtype, window, sinks):
    check([(1, 0), (4, 0), (63, 70), (64, 0), (65, 400), (130, 0), (400, 1), (0, 9), (500, 1000)], 8, 2, 64, 24, dtype,
          seed=(window + sinks) % 1000, window=window, sinks=sinks)
    check([(70, 2930), (1, 776)], 8, 1, 128, 64, dtype, seed=window % 1000, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [([(3, 60000)], 8, 2, 128, 64), ([(1, 30000), (3, 0), (0, 0), (50, 9000)], 32, 4, 128, 16),
                                  ([(7, 40000)], 3, 1, 16, 256), ([(9, 9000)] * 3, 8, 8, 64, 100),
                                  ([(n % 3, n) for n in range(1, 200)] + [(300, 5000)], 8, 2, 128, 16),
                                  ([(1, 100)] * 700, 8, 2, 64, 16), ([(1500, 0), (1200, 700)], 8, 2, 128, 64)],
                         ids=["one_long", "long_and_short", "one_kv_head", "several_long", "many_short", "single_tokens",
                              "prompts"])
def test_work_split_over_the_gpu(dtype, case):
    check(*case, dtype, seed=len(case[0]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_behind_the_last_sequence_and_a_wider_table(dtype):
    check([(37, 0), (0, 4), (250, 1)], 8, 2, 128, 16, dtype, max_pages=40, extra_pages=0, behind=9)
    check([(5, 0)], 4, 2, 64, 16, dtype, behind=300)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pools_with_keys_and_values_interleaved(dtype):
    check([(300, 0), (17, 33), (64, 64)], 8, 4, 64, 16, dtype, interleaved=True)
    check([(300, 5)], 8, 4, 128, 64, dtype, interleaved=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qstd", [0.0, 40.0])
def test_flat_and_peaked_softmax(dtype, qstd):
    check([(1, 0), (333, 0), (200, 1800)], 8, 2, 64, 32, dtype, seed=9, qstd=qstd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.25, 0.0, 1e-30, -3.0])
def test_scales_of_either_sign_and_zero(dtype, scale):
    for window in (0, 50):
        check([(1, 0), (77, 0), (30, 270), (200, 4800)], 8, 2, 64, 16, dtype, 31, scale=scale, window=window, sinks=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("others", [1, 500])
def test_many_keys_of_one_score(dtype, d, others):
    """A few keys of score 0 (one, or more than three tiles of them, behind whose maximum the reference then stays) and thousands
    that share another one, whose weight is next to half a step of bf16 from its rounding, so that nearly all of a row's
    weights have one and the same error.  Values of 1 give outputs of 1, the sums' own roundings left: 4,016 terms of one size, one
    after the other, at most 2^-24 of what is summed so far each, 4,016 / 2 * 2^-24 = 1.2e-4 together in fp32, which is far less
    than half a step of bf16 below 1 (2^-9).  With values a and b in the mean and weights A and B of the
    two scores, o = (A a + B b) / (A + B) moves by AB / (A + B)^2 <= 1/4 times the difference of the two scores' errors (at most
    2^-8 each in bf16, 2^-24 in fp32) times |a - b|.  Forty sequences of eight heads, on the same pages, so that a CTA goes through
    whole rows; alone, too, where rows are cut into pieces."""
    n, B, half = 16, 40, (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
    i32 = dict(dtype=torch.int32, device=DEV)
    for seed, (exponent, part) in enumerate([(e, x) for e in (-6, -1, 0, 2, 7) for x in (1.0038, 1.0040, 1.5)]):
        t = make([(n, 4000)], 16, 8, d, 64, dtype, seed)
        pages = t["block_table"][0].long()
        size = math.log(2.0 ** exponent * part)
        high = float(torch.tensor(size).to(DT[dtype]))
        t["k_pages"][pages] = 0
        for at, x in ((0, high), (1, size - high)):    # a score to 16 bits, also in bf16
            score = torch.full((pages.numel() * 64,), x, device=DEV)
            score[:others] = 0
            t["k_pages"][pages, :, :, at] = score.view(-1, 1, 64).to(DT[dtype])
        t["q"].zero_()
        t["q"][..., :2] = 1
        ref, ref_lse = reference(t, [(n, 4000)], 64, 1.0)
        v = t["v_pages"][pages].double().transpose(0, 1).reshape(8, -1, d)
        apart = (v[:, :others].mean(1) - v[:, others:4000].mean(1)).abs().repeat_interleave(2, 0)
        # (the last 16 tokens, which not every row sees, move the mean by less than 0.1)
        bound = half * ref.abs() + half / 2 * (apart + 0.1) + 1.2e-4 * v.nan_to_num(0, 0, 0).abs().max()
        many = dict(t, q=t["q"].repeat(B, 1, 1), block_table=t["block_table"].repeat(B, 1), seq_lens=t["seq_lens"].repeat(B),
                    cu_seqlens=torch.arange(0, n * B + 1, n, **i32))
        for call in (t, many):
            lse = torch.empty(call["q"].shape[:2], device=DEV)
            o = kda.kda_attention_prefill(**call, lse=lse).double().view(-1, n, 16, d)
            assert bool(((o - ref).abs() <= bound).all()), (exponent, part, float(((o - ref).abs() / bound).max()))
            assert float((lse.double().view(-1, n, 16) - ref_lse).abs().max()) <= 1e-4
        t["v_pages"][pages] = 1
        for call in (t, many):
            o = kda.kda_attention_prefill(**call)
            assert float((o - 1).abs().max()) <= (0 if dtype == "bf16" else 1.2e-4), (exponent, part, float((o - 1).abs().max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rising_and_falling_scores(dtype):
    """Keys that grow along the sequence (the maximum moves in every tile) and that shrink."""
    for sign in (1, -1):
        t = make([(300, 1500)], 4, 2, 64, 16, dtype, 3)
        pages = t["block_table"][0].long()
        ramp = torch.linspace(0.1, 8, pages.numel() * 16, device=DEV).view(-1, 1, 16, 1)
        k = t["k_pages"][pages].nan_to_num(0).abs() * sign
        t["k_pages"][pages] = (k * ramp).to(k.dtype)
        t["q"].abs_()
        ref, _ = reference(t, [(300, 1500)], 16, 0.125)
        o = kda.kda_attention_prefill(**t, scale=0.125)
        assert rel(o, ref) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_page_offsets_beyond_32_bits(dtype):
    """Pages that lie more than 2^31 elements into their pool."""
    ps, Hkv, d, rows = 256, 8, 128, [(100, 600), (300, 0)]
    P = (1 << 31) // (ps * Hkv * d) + 12
    t = make(rows, 16, Hkv, d, ps, dtype, 5)
    n = t["k_pages"].shape[0]
    k = torch.empty((P, Hkv, ps, d), dtype=DT[dtype], device=DEV)
    v = torch.empty((P, Hkv, ps, d), dtype=DT[dtype], device=DEV)
    k[P - n:], v[P - n:] = t["k_pages"], t["v_pages"]
    ref, _ = reference(t, rows, ps, d ** -0.5)
    t.update(k_pages=k, v_pages=v, block_table=torch.where(t["block_table"] >= 0, t["block_table"] + (P - n), t["block_table"]))
    o = kda.kda_attention_prefill(**t, scale=d ** -0.5)
    assert rel(o, ref) <= TOL[dtype] and kda.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_calls_give_the_same_bits(dtype):
    t = make([(40, 9000), (1, 0), (450, 0), (0, 0), (3, 30000)], 32, 8, 128, 64, dtype, 3)
    a = kda.kda_attention_prefill(**t, scale=0.1)
    b = kda.kda_attention_prefill(**t, scale=0.1)
    i = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(a.view(i), b.view(i))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_masked_is_not_used_whatever_it_holds(dtype, d, bad):
    """A later token's key and value, and ones before the window, that are not finite: tokens that do not see them are
    right, those that do see them say so."""
    rows, at, window = [(200, 90), (30, 10)], 170, 60
    for where in ("k_pages", "v_pages"):
        t = make(rows, 4, 2, d, 16, dtype, 4)
        t[where][int(t["block_table"][0, at // 16]), 0, at % 16] = bad
        for w in (0, window):
            clean = dict(t, **{where: t[where].nan_to_num(0, 0, 0)})
            ref, ref_lse = reference(clean, rows, 16, 0.1, w)
            lse = torch.empty(t["q"].shape[:2], device=DEV)
            o = kda.kda_attention_prefill(**t, scale=0.1, window=w, lse=lse)
            pos = torch.arange(90, 290, device=DEV)
            sees = (pos >= at) & ((pos - at < w) if w else pos >= 0)
            fine = torch.ones((230, 4), dtype=torch.bool, device=DEV)
            fine[:200, :2] = ~sees[:, None]
            assert bool(torch.isfinite(o[fine]).all()) and rel(o[fine], ref[fine]) <= TOL[dtype]
            assert float((lse[fine].double() - ref_lse[fine]).abs().max()) <= 1e-4
            if where == "v_pages":
                assert not bool(torch.isfinite(o[~fine]).any())
            elif bad != bad:
                assert bool(torch.isnan(o[~fine]).all()) and bool(torch.isnan(lse[~fine]).all())


@pytest.mark.parametrize("d,ps", [(64, 96), (128, 96), (128, 16), (64, 100), (16, 16), (64, 67), (128, 71), (128, 134)])
@pytest.mark.parametrize("window,sinks", [(500, 0), (300, 130), (0, 0)])
def test_values_that_are_not_finite_in_every_partly_seen_tile(d, ps, window, sinks):
    """256 rows of one token each, and in every tile that some of them see in part, and in two pages in three elsewhere among the first
    tokens, a value that is not finite: rows that see none of them are right, the others say so."""
    n, past = 256, 701
    t = make([(n, past)], 2, 2, d, ps, "bf16", d + ps)
    pos = torch.arange(past, past + n, device=DEV)
    seen = lambda j: (pos >= j) & ((pos - j < window) | torch.tensor(j < sinks, device=DEV) if window else pos >= 0)
    part = [j for j in range(past + n) if 0 < int(seen(j).sum()) < n]          # tokens that some rows see and others not
    bad = part[5::50] if window else part[5::60]
    clean = t["v_pages"].clone()
    for i, j in enumerate(bad):
        t["v_pages"][int(t["block_table"][0, j // ps]), i % 2, j % ps, i % d] = (math.nan, math.inf, -math.inf)[i % 3]
    assert len(bad) >= (5 if window == 0 else 9)
    ref, ref_lse = reference(dict(t, v_pages=clean), [(n, past)], ps, 0.1, window, sinks)
    lse = torch.empty((n, 2), device=DEV)
    o = kda.kda_attention_prefill(**t, scale=0.1, window=window, sinks=sinks, lse=lse)
    assert kda.kda_get_device_error() == 0
    hit = torch.zeros((n, 2, d), dtype=torch.bool, device=DEV)
    for i, j in enumerate(bad):
        hit[:, i % 2, i % d] |= seen(j)
    assert bool(hit.any()) and not bool(hit.all())
    assert bool(torch.isfinite(o[~hit]).all()) and not bool(torch.isfinite(o[hit]).any())
    assert float((o[~hit].double() - ref[~hit]).norm() / ref[~hit].norm()) <= TOL["bf16"]
    assert float((lse.double() - ref_lse).abs().max()) <= 1e-4


def test_a_row_whose_scores_are_all_minus_infinity():
    for dtype in ("bf16", "f32"):
        t = make([(40, 0)], 2, 1, 64, 16, dtype, 11)
        t["k_pages"].fill_(float("-inf"))
        t["v_pages"].fill_(1.0)
        t["q"].fill_(1.0)
        lse = torch.empty((40, 2), device=DEV)
        o = kda.kda_attention_prefill(**t, lse=lse)
        assert not o.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_tables_and_lengths_are_reported_not_faulted(dtype):
    rows = [(50, 150), (64, 0), (20, 70)]
    t = make(rows, 8, 2, 64, 16, dtype, 8)
    ref, _ = reference(t, rows, 16, 0.1)
    cap = 16 * t["block_table"].shape[1]
    for length in (cap + 1, -1, 2 ** 31 - 1, -2 ** 31):
        lens = t["seq_lens"].clone()
        lens[2] = length
        o = kda.kda_attention_prefill(**dict(t, seq_lens=lens), scale=0.1)
        assert kda.kda_get_device_error() == 0x20 and kda.kda_get_device_error() == 0
        assert rel(o[:114], ref[:114]) <= TOL[dtype] and not o[114:].any()
    lens = t["seq_lens"].clone()
    lens[1] = 60                                       # 64 new tokens: the first four lie before position 0
    o = kda.kda_attention_prefill(**dict(t, seq_lens=lens), scale=0.1)
    assert kda.kda_get_device_error() == 0x20
    assert not o[50:54].any() and bool(torch.isfinite(o).all())
    assert rel(o[114:], ref[114:]) <= TOL[dtype]
    for page in (-1, t["k_pages"].shape[0], 1 << 30, -2 ** 31):
        table = t["block_table"].clone()
        table[0, 3] = page                             # reads as zeros
        o = kda.kda_attention_prefill(**dict(t, block_table=table), scale=0.1)
        assert kda.kda_get_device_error() == 0x20
        k, v = (torch.cat([t[n], torch.zeros_like(t[n][:1])]) for n in ("k_pages", "v_pages"))
        table[0, 3] = k.shape[0] - 1
        want, _ = reference(dict(t, k_pages=k, v_pages=v, block_table=table), rows, 16, 0.1)
        assert rel(o, want) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 7), (64, 64), (16, 16), (128, 200)])
@pytest.mark.parametrize("window,sinks", [(40, 0), (100, 3), (129, 20), (1, 0)])
def test_pages_behind_every_window_may_be_any_number(dtype, d, ps, window, sinks):
    """A server that has given such pages back leaves -1 or a stale number in the table: nothing is reported, and the results are
    those of the full table.  One page that some token sees is reported."""
    rows = [(1, 700), (30, 555), (300, 900), (0, 400), (64, 0)]
    t = make(rows, 4, 2, d, ps, dtype, window + ps)
    want_lse, lse = (torch.empty(t["q"].shape[:2], device=DEV) for _ in range(2))
    want = kda.kda_attention_prefill(**t, scale=0.1, window=window, sinks=sinks, lse=want_lse)
    assert kda.kda_get_device_error() == 0
    for number in (-1, t["k_pages"].shape[0], -2 ** 31, 2 ** 31 - 1):
        table = t["block_table"].clone()
        for b, (n, past) in enumerate(rows):
            first = max(0, past + 1 - window) if n else n + past               # of the first new token's window
            for i in range(-(-(n + past) // ps)):
                if i * ps >= sinks and (i + 1) * ps <= first:
                    table[b, i] = number
        assert int((table[2] == number).sum()) >= (901 - window - sinks) // ps - 2
        o = kda.kda_attention_prefill(**dict(t, block_table=table), scale=0.1, window=window, sinks=sinks, lse=lse)
        assert kda.kda_get_device_error() == 0
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
        seen = max(0, 900 + 1 - window) // ps                                  # holds the first token of the third row's window
        table[2, seen] = number
        kda.kda_attention_prefill(**dict(t, block_table=table), scale=0.1, window=window, sinks=sinks)
        assert kda.kda_get_device_error() == 0x20


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_borders_are_reported_not_faulted(dtype):
    rows = [(50, 150), (64, 0), (20, 70)]
    t = make(rows, 8, 2, 64, 16, dtype, 8)
    ref, _ = reference(t, rows, 16, 0.1)
    for b, x in ((3, 135), (3, 2 ** 31 - 1), (3, 113), (3, -5)):
        cu = t["cu_seqlens"].clone()
        cu[b] = x
        o = kda.kda_attention_prefill(**dict(t, cu_seqlens=cu), scale=0.1, o=torch.zeros_like(t["q"]))
        assert kda.kda_get_device_error() & 0x1
        assert rel(o[:114], ref[:114]) <= TOL[dtype] and not o[114:].any()
    cu = t["cu_seqlens"].clone()
    cu[0] = 3
    kda.kda_attention_prefill(**dict(t, cu_seqlens=cu), scale=0.1)
    assert kda.kda_get_device_error() & 0x1


def test_no_pages_and_no_tokens():
    for dtype in ("bf16", "f32"):
        t = make([(5, 0)], 4, 2, 64, 16, dtype, 1)
        i32 = dict(dtype=torch.int32, device=DEV)
        empty = dict(block_table=torch.empty((1, 0), **i32), seq_lens=torch.zeros(1, **i32))
        o = kda.kda_attention_prefill(**dict(t, **empty), scale=0.1)
        assert not o.any() and kda.kda_get_device_error() == 0x20
        o = kda.kda_attention_prefill(**dict(t, q=t["q"][:0], cu_seqlens=torch.zeros(2, **i32)))
        assert o.shape == (0, 4, 64)
        o = kda.kda_attention_prefill(t["q"], t["k_pages"], t["v_pages"], torch.empty((0, 3), **i32), torch.empty(0, **i32),
                                      torch.zeros(1, **i32), o=torch.full_like(t["q"], 3.0))
        assert bool((o == 3).all()) and kda.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_streams_and_graphs(dtype):
    """On a side stream with its own workspace, and captured: replayed with other lengths and other values; two captured
    calls that share a workspace."""
    rows = [(60, 5000), (77, 0)]
    t = make(rows, 8, 2, 128, 16, dtype, 6)
    i = torch.int16 if dtype == "bf16" else torch.int32
    want = kda.kda_attention_prefill(**t, scale=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kda.kda_attention_prefill(**t, scale=0.1, stream=side)
    side.synchronize()
    assert torch.equal(got.view(i), want.view(i))
    ws = torch.empty(kda.kda_attention_prefill_workspace_size(2, 137, 8, 2, 128, DT[dtype]), dtype=torch.uint8, device=DEV)
    o, o2 = torch.empty_like(t["q"]), torch.empty_like(t["q"])
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_attention_prefill(**t, scale=0.1, o=o, workspace=ws)
    with torch.cuda.graph(second):
        kda.kda_attention_prefill(**t, scale=0.2, o=o2, workspace=ws)
    for lens in ([5060, 77], [60, 77], [3000, 77]):
        t["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay(), second.replay(), graph.replay()
        ref, _ = reference(t, [(60, lens[0] - 60), (77, 0)], 16, 0.1)
        assert rel(o, ref) <= TOL[dtype]
        ref, _ = reference(t, [(60, lens[0] - 60), (77, 0)], 16, 0.2)
        assert rel(o2, ref) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_is_the_decode_steps(dtype):
    rows = [(1, n) for n in (0, 5, 300, 2000)]
    t = make(rows, 8, 2, 128, 16, dtype, 17)
    a = kda.kda_attention_prefill(**t, scale=0.1, window=900, sinks=2)
    cu = t.pop("cu_seqlens")
    assert cu.tolist() == [0, 1, 2, 3, 4]
    b = kda.kda_attention_decode(**t, scale=0.1, window=900, sinks=2)
    assert rel(a, b.double()) <= 2 * TOL[dtype]


def test_argument_checks():
    t = make([(40, 3), (5, 0)], 4, 2, 64, 16, "bf16", 12)
    call = lambda **over: kda.kda_attention_prefill(**{**t, **over})
    for error, over in [(TypeError, dict(q=t["q"].float())), (TypeError, dict(seq_lens=t["seq_lens"].long())),
                        (TypeError, dict(q=t["q"].half())), (ValueError, dict(q=t["q"].cpu())),
                        (ValueError, dict(q=t["q"][0])), (ValueError, dict(block_table=t["block_table"][:1])),
                        (ValueError, dict(cu_seqlens=t["cu_seqlens"][:2])), (ValueError, dict(k_pages=t["k_pages"][0])),
                        (ValueError, dict(q=t["q"].transpose(0, 1).contiguous().transpose(0, 1))),
                        (ValueError, dict(k_pages=t["k_pages"].transpose(1, 2).contiguous().transpose(1, 2))),
                        (ValueError, dict(v_pages=t["v_pages"][:-1])), (kda.KdaError, dict(window=-1)),
                        (kda.KdaError, dict(scale=math.nan)), (kda.KdaError, dict(sinks=-1)),
                        (kda.KdaError, dict(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)))]:
        with pytest.raises(error):
            call(**over)
    u = make([(40, 0)], 4, 2, 32, 16, "bf16", 13)
    with pytest.raises(kda.KdaError):                  # no kernel for this head size
        kda.kda_attention_prefill(**u)
    assert kda.kda_get_device_error() == 0
