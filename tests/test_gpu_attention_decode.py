"""kda_attention_decode against softmax attention in float64, over the sizes, masks and page layouts where
a paged, split kernel can go wrong.

Tolerances, relative Frobenius: the bf16 output is rounded once (at most 2^-9 of each value, 1.7e-3 in the
mean over a binade's values) and everything before it keeps 16 bits or more, so 3e-3; the fp32 path sums up to
70,000 terms of random sign in fp32 (2^-24 a step, growing with the square root: below 2e-5)."""

import numpy as np
import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 3e-3, "f32": 2e-5}
DEV = "cuda:0"


def make(lens, Hq, Hkv, d, ps, dtype, seed, extra_pages=3, max_pages=None, qstd=1.5, interleaved=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, dt = len(lens), DT[dtype]
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
    r = lambda *s: torch.randn(s, device=DEV, generator=g).to(dt)
    return dict(q=(qstd * r(B, Hq, d)).to(dt), k_pages=k, v_pages=v, block_table=torch.from_numpy(table).to(DEV),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV)), (r(B, Hkv, d), r(B, Hkv, d))


def reference(t, lens, ps, scale, window, sinks, new=None):
    """o, lse in float64, row by row."""
    B, Hq, d = t["q"].shape
    Hkv = t["k_pages"].shape[1]
    o = torch.zeros((B, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -float("inf"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = t["block_table"][b, :-(-n // ps)].long()
        pos = torch.arange(n, device=DEV)
        seen = (pos >= n - window) | (pos < sinks) if window else pos >= 0
        k = t["k_pages"][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].double()
        v = t["v_pages"][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].double()
        if new is not None:
            k[:, n - 1], v[:, n - 1] = new[0][b].double(), new[1][b].double()
        k, v = k[:, seen], v[:, seen]
        s = torch.einsum("hgd,htd->hgt", t["q"][b].double().view(Hkv, Hq // Hkv, d), k) * scale
        o[b] = torch.einsum("hgt,htd->hgd", torch.softmax(s, 2), v).reshape(Hq, d)
        lse[b] = torch.logsumexp(s, 2).reshape(Hq)
    return o, lse


def rel(x, ref):
    return float((x.double() - ref).norm() / ref.norm().clamp(min=1e-300))


def check(lens, Hq, Hkv, d, ps, dtype, seed=0, window=0, sinks=0, append=True, **kw):
    t, new = make(lens, Hq, Hkv, d, ps, dtype, seed, **kw)
    scale = d ** -0.5
    ref, ref_lse = reference(t, lens, ps, scale, window, sinks, new if append else None)
    want = t["k_pages"].clone(), t["v_pages"].clone()
    if append:
        for b, n in enumerate(lens):
            if n:
                p, at = int(t["block_table"][b, (n - 1) // ps]), (n - 1) % ps
                want[0][p, :, at], want[1][p, :, at] = new[0][b], new[1][b]
    lse = torch.empty((len(lens), Hq), device=DEV)
    o = kda.kda_attention_decode(**t, scale=scale, window=window, sinks=sinks, lse=lse,
                                 **(dict(k_new=new[0], v_new=new[1]) if append else {}))
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    assert o.dtype == DT[dtype] and bool(torch.isfinite(o).all())
    assert rel(o, ref) <= TOL[dtype], rel(o, ref)
    for b, n in enumerate(lens):                       # no row hides behind the others
        if n:
            assert rel(o[b], ref[b]) <= 2 * TOL[dtype], (b, n, rel(o[b], ref[b]))
            assert float((lse[b].double() - ref_lse[b]).abs().max()) <= 1e-4
        else:
            assert not o[b].any() and bool(torch.isneginf(lse[b]).all())
    for got, exp in zip((t["k_pages"], t["v_pages"]), want):
        i = torch.int16 if got.element_size() == 2 else torch.int32
        assert torch.equal(got.contiguous().view(i), exp.contiguous().view(i))
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_lengths_around_tiles_and_pages(dtype, d):
    check([1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 511, 513, 1000], 8, 2, d, 16, dtype, seed=d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (6, 3), (3, 1), (32, 8), (5, 1), (16, 2), (9, 1), (12, 1), (32, 2),
                                   (17, 1), (48, 2), (32, 1), (40, 1)])
def test_head_layouts(dtype, heads):
    check([70, 129, 5, 300], *heads, 64, 32, dtype, seed=heads[0])
    check([260, 33], *heads, 128, 16, dtype, seed=heads[1] + 50)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ps", [1, 3, 7, 16, 24, 48, 64, 100, 128, 256, 1000])
def test_page_sizes(dtype, ps):
    check([1, 99, 640, 1001], 4, 2, 64, ps, dtype, seed=ps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (64, 64), (100, 4), (300, 70), (2000, 4), (129, 500)])
def test_window_and_sinks(dtype, window, sinks):
    check([1, 4, 63, 64, 65, 130, 400, 0, 1500], 8, 2, 64, 24, dtype, seed=window + sinks, window=window, sinks=sinks)
    check([3000, 777], 8, 1, 128, 64, dtype, seed=window, window=window, sinks=sinks, append=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [([70001], 8, 8, 128, 64), ([40000, 3, 0, 17000], 32, 4, 128, 16), ([65537], 3, 1, 16, 256),
                                  ([20000] * 3, 8, 8, 64, 100), ([31, 32, 33] * 100 + [5000], 8, 2, 128, 16)],
                         ids=["one_long", "long_and_short", "one_kv_head", "several_long", "many_short"])
def test_lengths_split_over_the_gpu(dtype, case):
    check(*case, dtype, seed=len(case[0]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("tiles", [1, 4, 5, 8, 9])
def test_rows_that_the_table_keeps_short(dtype, d, tiles):
    """Units done whole and in shares: tables that hold up to 4, 8 and more tiles, few rows and many."""
    most = tiles * {128: 64, 64: 128, 16: 256}[d] // (1 if dtype == "bf16" else 2)
    check([most], 8, 2, d, 16, dtype, seed=tiles)
    check([0, most, 1, most - 1], 4, 4, d, 32, dtype, seed=tiles + 1)
    check([most if b % 3 == 0 else b % 5 for b in range(70)], 2, 2, d, 16, dtype, seed=tiles + 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [450, 700, 1500])
def test_more_rows_than_the_gpu_holds_ctas(dtype, B):
    check([(b * 7) % 41 for b in range(B)], 2, 1, 64, 8, dtype, seed=B, max_pages=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(40, 0), (20, 5), (1, 100)])
def test_rows_that_the_window_keeps_short(dtype, window, sinks):
    check([5000, 30, 0, 1000, 41, 1], 8, 2, 128, 16, dtype, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_a_new_token_and_with_a_wider_table(dtype):
    check([37, 0, 250], 8, 2, 128, 16, dtype, append=False, max_pages=40, extra_pages=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pools_with_keys_and_values_interleaved(dtype):
    check([300, 17, 64], 8, 4, 64, 16, dtype, interleaved=True)
    check([300, 17, 64], 8, 4, 128, 64, dtype, interleaved=True, append=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qstd", [0.0, 40.0])
def test_flat_and_peaked_softmax(dtype, qstd):
    """All scores equal, and scores of hundreds (one token takes nearly everything)."""
    check([1, 333, 2000], 8, 2, 64, 32, dtype, seed=9, qstd=qstd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.25, 0.0, 1e-30, -3.0])
def test_scales_of_either_sign_and_zero(dtype, scale):
    lens = [1, 77, 300, 5000]
    t, _ = make(lens, 8, 2, 64, 16, dtype, 31)
    for window in (0, 50):
        ref, ref_lse = reference(t, lens, 16, scale, window, 3)
        lse = torch.empty((4, 8), device=DEV)
        o = kda.kda_attention_decode(**t, scale=scale, window=window, sinks=3, lse=lse)
        assert rel(o, ref) <= TOL[dtype] and float((lse.double() - ref_lse).abs().max()) <= 1e-4


def test_values_keep_their_precision_under_many_equal_weights():
    """A bf16 row whose values nearly cancel: the weights must not be rounded to bf16 before the sum.  With flat
    weights w rounded at random, the error against the exact mean would be 2^-9 / sqrt(3) of |v| / sqrt(n) per
    output, which is 1.1e-3 of the outputs themselves, on top of the output's own rounding (1.7e-3)."""
    t, _ = make([4096] * 8, 8, 1, 128, 64, "bf16", 21, qstd=0.2)
    ref, _ = reference(t, [4096] * 8, 64, 128 ** -0.5, 0, 0)
    o = kda.kda_attention_decode(**t, scale=128 ** -0.5)
    rounded = rel(ref.to(torch.bfloat16), ref)
    assert rel(o, ref) <= 1.1 * rounded


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_page_offsets_beyond_32_bits(dtype):
    """Pages that lie more than 2^31 elements into their pool."""
    ps, Hkv, d, lens = 256, 8, 128, [700, 300]
    P = (1 << 31) // (ps * Hkv * d) + 12
    t, new = make(lens, 16, Hkv, d, ps, dtype, 5)
    k = torch.empty((P, Hkv, ps, d), dtype=DT[dtype], device=DEV)
    v = torch.empty((P, Hkv, ps, d), dtype=DT[dtype], device=DEV)
    n = t["k_pages"].shape[0]
    k[P - n:], v[P - n:] = t["k_pages"], t["v_pages"]
    table = torch.where(t["block_table"] >= 0, t["block_table"] + (P - n), t["block_table"])
    ref, _ = reference(t, lens, ps, d ** -0.5, 0, 0, new)
    o = kda.kda_attention_decode(t["q"], k, v, table, t["seq_lens"], scale=d ** -0.5, k_new=new[0], v_new=new[1])
    assert rel(o, ref) <= TOL[dtype]
    p = int(table[0, 2])
    assert torch.equal(k[p, :, 699 - 512], new[0][0]) and torch.equal(v[p, :, 699 - 512], new[1][0])
    assert kda.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_calls_give_the_same_bits(dtype):
    t, _ = make([9000, 1, 450, 0, 30000], 32, 8, 128, 64, dtype, 3)
    a = kda.kda_attention_decode(**t, scale=0.1)
    b = kda.kda_attention_decode(**t, scale=0.1)
    i = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(a.view(i), b.view(i))


def test_not_a_number_in_a_visible_place_is_not_hidden():
    t, _ = make([100, 100], 4, 2, 64, 16, "bf16", 4)
    t["v_pages"][int(t["block_table"][0, 1]), 0, 3] = float("nan")
    o = kda.kda_attention_decode(**t, scale=0.1)
    assert bool(torch.isnan(o[0, :2]).all()) and bool(torch.isfinite(o[0, 2:]).all()) and bool(torch.isfinite(o[1]).all())


def test_runs_on_the_given_stream():
    t, _ = make([5000, 77], 8, 2, 128, 16, "bf16", 6)
    want = kda.kda_attention_decode(**t, scale=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(max(1, kda.kda_attention_decode_workspace_size(2, 8, 2, 128)), dtype=torch.uint8, device=DEV)
    got = torch.empty_like(want)
    kda.kda_attention_decode(**t, scale=0.1, o=got, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_tables_are_reported_not_faulted(dtype):
    """A length that the table cannot hold counts as 0 and a page outside the pool as page 0: all reads stay in
    bounds, the other rows are right, and the error word says so."""
    lens = [200, 64, 90]
    t, _ = make(lens, 8, 2, 64, 16, dtype, 8)
    ref, _ = reference(t, lens, 16, 0.1, 0, 0)
    bad = dict(t, seq_lens=torch.tensor([200, 64, 16 * t["block_table"].shape[1] + 1], dtype=torch.int32, device=DEV))
    o = kda.kda_attention_decode(**bad, scale=0.1)
    assert kda.kda_get_device_error() == 0x20 and kda.kda_get_device_error() == 0
    assert rel(o[:2], ref[:2]) <= TOL[dtype] and not o[2].any()
    for page in (-1, t["k_pages"].shape[0], 1 << 30):
        table = t["block_table"].clone()
        table[1, 2] = page
        o = kda.kda_attention_decode(**dict(t, block_table=table), scale=0.1)
        assert kda.kda_get_device_error() == 0x20
        assert rel(o[0], ref[0]) <= TOL[dtype] and rel(o[2], ref[2]) <= 2 * TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [-1, 9, 1 << 30])
def test_a_new_token_without_a_page_is_reported(dtype, page):
    """A new token that begins a page which the table does not name: nobody reads that page, but what is not stored has
    to be told.  The outputs are right, the pools unchanged but for the other row's token."""
    lens = [33, 48]
    t, new = make(lens, 4, 2, 64, 16, dtype, 41)
    ref, _ = reference(t, lens, 16, 0.1, 0, 0, new)
    want = t["k_pages"].clone(), t["v_pages"].clone()
    p = int(t["block_table"][1, 2])
    want[0][p, :, 15], want[1][p, :, 15] = new[0][1], new[1][1]
    t["block_table"][0, 2] = page
    assert t["k_pages"].shape[0] == 9
    o = kda.kda_attention_decode(**t, scale=0.1, k_new=new[0], v_new=new[1])
    assert kda.kda_get_device_error() == 0x20 and kda.kda_get_device_error() == 0
    assert rel(o, ref) <= TOL[dtype]
    i = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(t["k_pages"].view(i), want[0].view(i)) and torch.equal(t["v_pages"].view(i), want[1].view(i))


def test_a_row_whose_scores_are_all_minus_infinity():
    """Keys of -inf against a positive query: every weight is exp(-inf), the row counts as empty."""
    t, _ = make([40], 2, 1, 64, 16, "f32", 11)
    t["k_pages"].fill_(float("-inf"))
    t["q"].fill_(1.0)
    lse = torch.empty((1, 2), device=DEV)
    o = kda.kda_attention_decode(**t, lse=lse)
    assert not o.any() and bool(torch.isneginf(lse).all())


def test_argument_checks():
    t, new = make([40, 3], 4, 2, 64, 16, "bf16", 12)
    call = lambda **over: kda.kda_attention_decode(**{**t, **over})
    with pytest.raises(TypeError):
        call(q=t["q"].float())
    with pytest.raises(TypeError):
        call(seq_lens=t["seq_lens"].long())
    with pytest.raises(ValueError):
        call(q=t["q"].cpu())
    with pytest.raises(ValueError):
        call(block_table=t["block_table"][:1])
    with pytest.raises(ValueError):
        call(k_new=new[0])
    with pytest.raises(ValueError):
        call(k_pages=t["k_pages"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        call(q=t["q"].transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(kda.KdaError):
        call(window=-1)
    with pytest.raises(kda.KdaError):
        call(scale=float("nan"))
    if kda.kda_attention_decode_workspace_size(2, 4, 2, 64) > 16:
        with pytest.raises(kda.KdaError):
            call(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    u, _ = make([40], 4, 2, 32, 16, "bf16", 13)
    with pytest.raises(kda.KdaError):                  # no kernel for this head size
        kda.kda_attention_decode(**u)
    assert kda.kda_get_device_error() == 0
