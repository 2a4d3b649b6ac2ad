"""kda_token_logprobs and its gradient against log_softmax in float64.

Tolerances.  A float32 difference x - m is off by 2^-24 of itself, its exponential by that times the difference and 2^-22
of the instruction, a sum of V positive terms by a few 2^-24 more: 2e-6 of each sum at the differences (up to 30) that carry
weight, and so of a log probability and an entropy, next to zero as well; 2e-6 times the size of m for lse.  A gradient's
entry has p (that, and lse's own rounding, 2^-24 |lse|, times p) and one rounding to its type."""

import math

import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"
REL = 4e-6


def reference(logits, tokens, top):
    x = logits.double()
    lse = torch.logsumexp(x, 1)
    m = x.amax(1, keepdim=True)
    lp = (x - m) - torch.log1p((torch.exp(x - m).sum(1, keepdim=True) - 1).clamp(min=0))
    y = tokens.long()
    logp = torch.where(y >= 0, lp.gather(1, y.clamp(min=0)[:, None])[:, 0], torch.zeros((), dtype=torch.float64, device=DEV))
    p = torch.exp(lp)
    entropy = -torch.where(p > 0, p * lp, torch.zeros((), dtype=torch.float64, device=DEV)).sum(1)
    order = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :top]
    return logp, lse, entropy, lp.gather(1, order), order.int()


def near(got, want, floor=0.0):
    got = got.double()
    assert bool((torch.isneginf(got) == torch.isneginf(want)).all())
    fine = torch.isfinite(want)
    assert bool(torch.isfinite(got[fine]).all())
    off = (got[fine] - want[fine]).abs() / want[fine].abs().clamp(min=1e-30 + floor)
    assert off.numel() == 0 or float(off.max()) <= REL, float(off.max())


def check(logits, tokens, top, entropy=True):
    r = kda.kda_token_logprobs(logits, tokens, top=top, entropy=entropy)
    logp, lse, H, best, word = reference(logits, tokens, top)
    # log1p's argument in the reference is a difference of 64-bit numbers near 1: 1e-16 of 1e-8 and more
    near(r.logp, logp, 1e-8)
    near(r.lse, lse, 1.0)
    near(r.top_logp, best, 1e-8)
    assert torch.equal(r.top_token, word)
    if entropy:
        near(r.entropy, H, 1e-7)
    else:
        assert r.entropy is None
    assert kda.kda_get_device_error() == 0
    return r


def make(T, V, dtype, seed=0, std=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = (std * torch.randn((T, V), device=DEV, generator=g)).to(DT[dtype])
    tokens = torch.randint(0, V, (T,), device=DEV, generator=g).int()
    return logits, tokens


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (2, 50), (9, 1000), (700, 33), (3, 4095), (3, 4097), (2, 8191), (2, 8193),
                                 (4, 32001), (1, 65536), (20, 50257), (400, 9001), (1, 262147), (3, 131072), (330, 16385)])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_sizes(dtype, T, V, top):
    logits, tokens = make(T, V, dtype, seed=T + V)
    if T > 2:
        tokens[1] = -1
    check(logits, tokens, min(top, V), entropy=top != 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two_values", "steps", "few_allowed", "first_part_masked",
                                  "negative_zeros"])
def test_rows_in_any_order(dtype, kind):
    """Ties, and rows that bring a new best word all along."""
    T, V = 5, 60001
    j = torch.arange(V, device=DEV).float()
    row = {"equal": torch.zeros(V, device=DEV) - 3, "rising": j / 1000 - 40, "falling": 20 - j / 1000, "two_values": (j % 17 == 3).float(),
           "steps": torch.floor(j / 5000), "few_allowed": torch.where(j % 20011 == 20010, j / 1e5, -math.inf),
           "first_part_masked": torch.where(j < 20000, -math.inf, torch.sin(j)),
           "negative_zeros": torch.where(j % 2 == 0, -0.0, 0.0)}[kind]
    logits = row.to(DT[dtype]).expand(T, V).contiguous()
    tokens = torch.tensor([0, 1, V - 1, 20010, -1], dtype=torch.int32, device=DEV)
    for top in (1, 4, 20, 32):
        check(logits, tokens, top)
    many = logits[:1].expand(400, V).contiguous()
    check(many, tokens[3:4].expand(400).contiguous(), 20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [0.0, 3.0, 12.0, 18.0, 60.0, 200.0])
def test_a_likely_word_keeps_its_small_probability_gap(dtype, gap):
    """-log p and the entropy next to zero, wherever the word lies."""
    V = 40000
    for at in (0, 5, 9999, 20000, 39999):
        logits, _ = make(2, V, dtype, seed=at, std=0.5)
        logits[:, at] = logits.float().amax() + gap
        tokens = torch.tensor([at, (at + 1) % V], dtype=torch.int32, device=DEV)
        logp, lse, H, best, _ = reference(logits, tokens, 2)
        r = kda.kda_token_logprobs(logits, tokens, top=2, entropy=True)
        x = logits.double()
        rest = torch.exp(x - x[:, at:at + 1])
        rest[:, at] = 0
        exact = -torch.log1p(rest.sum(1))
        near(r.logp[:1], exact[:1])
        near(r.top_logp[:, 0], exact)
        xm = x - x[:, at:at + 1]
        xm[:, at] = 0
        h = torch.log1p(rest.sum(1)) - (rest * xm).sum(1) / (1 + rest.sum(1))
        near(r.entropy, h, 1e-35)
        near(r.logp[1:], (xm[1, (at + 1) % V] + exact[1])[None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_with_nothing_allowed_and_with_values_that_are_not_finite(dtype):
    logits, tokens = make(6, 9000, dtype)
    logits[1] = -math.inf
    logits[2, 8500] = math.nan
    logits[3, 77] = math.inf
    logits[4, :8999] = -math.inf
    tokens[1], tokens[4] = 5, 8999
    r = kda.kda_token_logprobs(logits, tokens, top=3, entropy=True)
    for t in (0, 5):
        one = kda.kda_token_logprobs(logits[t:t + 1], tokens[t:t + 1], top=3, entropy=True)
        assert all(torch.equal(a[t:t + 1], b) for a, b in zip(r, one))
    assert r.lse[1] == -math.inf and r.logp[1] == -math.inf and r.entropy[1] == 0
    assert r.top_token[1].tolist() == [0, 1, 2] and bool(torch.isneginf(r.top_logp[1]).all())
    for t in (2, 3):
        assert bool(torch.isnan(torch.stack([r.lse[t], r.logp[t], r.entropy[t]])).all()) and bool(torch.isnan(r.top_logp[t]).all())
    assert r.top_token[3, 0] == 77 and 8500 not in r.top_token[2].tolist()
    assert r.logp[4] == 0 and r.entropy[4] == 0 and r.top_token[4].tolist() == [8999, 0, 1]
    one = torch.zeros(6, device=DEV)
    g = kda.kda_token_logprobs_backward(logits, tokens, r.lse, one + 1, entropy=r.entropy, grad_entropy=one + 1)
    assert not g[1].any() and not g[4].any()
    assert kda.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_of_the_types_lowest_value(dtype):
    """Words masked by the lowest finite value, and a row of nothing else, which is a flat one."""
    low = torch.finfo(DT[dtype]).min
    logits, tokens = make(4, 20000, dtype)
    logits[0, 100:] = low
    logits[1, :19990] = low
    logits[2] = low
    logits[3, ::2], logits[3, 1::2] = low, -math.inf
    tokens[:] = torch.tensor([5, 19995, 7, 8], dtype=torch.int32)
    r = kda.kda_token_logprobs(logits, tokens, top=4, entropy=True)
    logp, _, H, best, word = reference(logits, tokens, 4)
    near(r.logp, logp)
    near(r.entropy, H)
    near(r.top_logp, best)
    assert torch.equal(r.top_token, word) and r.top_token[2].tolist() == [0, 1, 2, 3]
    assert float(r.lse[2]) == float(torch.tensor(low, dtype=torch.float32))
    nans = logits.clone()
    nans[0, 3], nans[0, 50] = math.nan, math.nan
    nans[0, 100:] = -math.inf
    nans[0, 8:100] = -math.inf
    r = kda.kda_token_logprobs(nans, tokens, top=12)
    assert r.top_token[0].tolist()[7:] == [3, 8, 9, 10, 11] and sorted(r.top_token[0].tolist()[:7]) == [0, 1, 2, 4, 5, 6, 7]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_outside_are_reported(dtype):
    logits, tokens = make(4, 100, dtype)
    tokens[1], tokens[2], tokens[3] = 100, -2, -2 ** 31
    r = kda.kda_token_logprobs(logits, tokens)
    assert kda.kda_get_device_error() == 0x100 and r.logp[1:].tolist() == [0, 0, 0] and r.logp[0] != 0
    g = kda.kda_token_logprobs_backward(logits, tokens, r.lse, torch.ones(4, device=DEV))
    assert not g[1:].any() and g[0].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,stride", [(1000, 1003), (777, 777), (8200, 8201), (5, 9), (9001, 9008)])
def test_strides_and_places(dtype, V, stride):
    base, tokens = make(7, stride + 3, dtype, seed=V)
    big = torch.zeros(7 * stride + 20, dtype=DT[dtype], device=DEV)
    for shift in (0, 1, 3):
        logits = big[shift:shift + 7 * stride].view(7, stride)[:, :V]
        logits.copy_(base[:, :V])
        y = tokens % V
        a, b = check(logits, y, min(3, V)), kda.kda_token_logprobs(logits.contiguous(), y, top=min(3, V), entropy=True)
        assert all(torch.allclose(u, v, rtol=1e-6, atol=1e-6) for u, v in zip(a, b))
        g = torch.randn(7, device=DEV)
        want = kda.kda_token_logprobs_backward(logits.contiguous(), y, a.lse, g, entropy=a.entropy, grad_entropy=g)
        before = big.clone()
        got = kda.kda_token_logprobs_backward(logits, y, a.lse, g, entropy=a.entropy, grad_entropy=g, grad=logits)
        assert got.data_ptr() == logits.data_ptr() and torch.equal(got, want)
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[shift:shift + 7 * stride].view(7, stride)[:, :V] = False
        assert torch.equal(big[keep], before[keep])                           # what lies between the rows


def gradient(logits, tokens, gl, gh):
    x = logits.double().detach().requires_grad_()
    lp = torch.log_softmax(x, 1)
    logp = lp.gather(1, tokens.long().clamp(min=0)[:, None])[:, 0] * (tokens >= 0)
    loss = (logp * gl.double()).sum()
    if gh is not None:
        loss = loss - ((torch.exp(lp) * lp).sum(1) * gh.double()).sum()
    return torch.autograd.grad(loss, x)[0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (5, 7), (300, 65), (3, 4097), (7, 32001), (2, 131072)])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient_against_the_formulas(dtype, T, V, entropy):
    logits, tokens = make(T, V, dtype, seed=V)
    if T > 2:
        tokens[1] = -1
    gl, gh = torch.randn(T, device=DEV), torch.randn(T, device=DEV) if entropy else None
    r = kda.kda_token_logprobs(logits, tokens, entropy=True)
    g = kda.kda_token_logprobs_backward(logits, tokens, r.lse, gl, entropy=r.entropy if entropy else None, grad_entropy=gh)
    want = gradient(logits, tokens, gl, gh)
    assert g.dtype == DT[dtype]
    p = torch.softmax(logits.double(), 1)
    # p's relative error times what it is multiplied by, and the rounding to the type
    size = p * (gl.abs()[:, None] + (gh.abs()[:, None] * (30 + 1) if entropy else 0)) + (gl.abs()[:, None] if dtype == "f32" else 0) * 1e-3
    bound = 4e-6 * size + torch.finfo(DT[dtype]).eps / 2 * want.abs() + 1e-30
    assert bool(((g.double() - want).abs() <= bound).all()), float(((g.double() - want).abs() / bound).max())


def test_gradient_against_differences():
    logits, tokens = make(3, 40, "f32", seed=2)
    gl, gh = torch.tensor([1.0, -0.5, 0.3], device=DEV), torch.tensor([0.2, 0.7, -1.0], device=DEV)
    r = kda.kda_token_logprobs(logits, tokens, entropy=True)
    g = kda.kda_token_logprobs_backward(logits, tokens, r.lse, gl, entropy=r.entropy, grad_entropy=gh)
    step = 2.0 ** -6
    for j in (0, 13, 39, int(tokens[0])):
        up, down = logits.clone(), logits.clone()
        up[:, j] += step
        down[:, j] -= step
        a, b = (kda.kda_token_logprobs(x, tokens, entropy=True) for x in (up, down))
        diff = ((a.logp - b.logp) * gl + (a.entropy - b.entropy) * gh) / (2 * step)
        # third derivatives of both are below 6: 6 / 6 * step^2 * 2 = 5e-4 and the outputs' own 2e-6 * 10 / step = 1.3e-3
        assert float((g[:, j] - diff).abs().max()) <= 2e-3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 1000, 40001])
def test_gradient_of_rows_far_from_zero(dtype, V):
    """Logits so large that lse in fp32 is off by a part of a word's probability, or by all of it: rows masked by the type's lowest
    value and nothing else, or by a large number, and rows far from zero.  Differences of the logits are exact (or, between two
    of a size, the logits' own), so p is as near as that of any row: its sum's and exponentials' roundings, 4e-6 of it."""
    low = torch.finfo(DT[dtype]).min
    j = torch.arange(V, device=DEV).float()
    rows = [torch.full((V,), low, device=DEV), torch.where(j % 3 == 0, low, -math.inf), torch.full((V,), -1e9, device=DEV),
            torch.where(j % 5 == 0, 1e6 + 8 * torch.sin(j), -1e9), -3e4 + 4 * torch.cos(j), 1500 + 3 * torch.sin(3 * j), -1025 - j % 7,
            1023 + 0 * j, torch.sin(j)]
    logits = torch.stack(rows).to(DT[dtype])
    T = logits.shape[0]
    tokens = ((torch.arange(T, device=DEV) * 3) % V).int()
    tokens[2] = -1
    g = torch.Generator(device=DEV).manual_seed(V)
    gl, gh = (torch.randn(T, device=DEV, generator=g) for _ in range(2))
    r = kda.kda_token_logprobs(logits, tokens, entropy=True)
    p = torch.softmax(logits.double(), 1)
    lse = torch.logsumexp(logits.double(), 1).abs()
    scored = (tokens >= 0)[:, None]
    given = torch.zeros_like(p).scatter_(1, tokens.long().clamp(min=0)[:, None], 1.0) * scored
    entr = torch.special.entr(p)
    for entropy in (False, True):
        want = gl.double()[:, None] * (given - p * scored)
        size = p * gl.abs()[:, None] + (gl.abs()[:, None] * 1e-3 if dtype == "f32" else 0)
        if entropy:
            want = want + gh.double()[:, None] * (entr - p * entr.sum(1, keepdim=True))
            size = size + p * gh.abs()[:, None] * (30 + 1)
        # within 1,024 of zero p has lse's rounding, too
        rounding = torch.where(lse <= 1024.01, lse * 2.0 ** -24, 0.0)[:, None]
        bound = (4e-6 + rounding) * size + torch.finfo(DT[dtype]).eps / 2 * want.abs() + 1e-30
        extra = dict(entropy=r.entropy, grad_entropy=gh) if entropy else {}
        for place in (None, logits.clone()):           # the last one in the logits' place
            got = kda.kda_token_logprobs_backward(logits if place is None else place, tokens, r.lse, gl, grad=place, **extra)
            off = ((got.double() - want).abs() / bound).amax(1)
            assert bool((off <= 1).all()), off.tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_streams_and_graphs(dtype):
    logits, tokens = make(6, 50257, dtype)
    a = kda.kda_token_logprobs(logits, tokens, top=9, entropy=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = kda.kda_token_logprobs(logits, tokens, top=9, entropy=True, stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = kda.kda_token_logprobs(logits, tokens, top=9, entropy=True)
        g = kda.kda_token_logprobs_backward(logits, tokens, c.lse, c.logp)
    other, _ = make(6, 50257, dtype, seed=5)
    logits.copy_(other)
    graph.replay()
    d = kda.kda_token_logprobs(logits, tokens, top=9, entropy=True)
    assert all(torch.equal(u, v) for u, v in zip(c, d))
    assert torch.equal(g, kda.kda_token_logprobs_backward(logits, tokens, d.lse, d.logp))


def test_a_matrix_beyond_32_bit_offsets():
    T, V = 17000, 131072
    logits = torch.zeros((T, V), dtype=torch.bfloat16, device=DEV)
    logits[-1], tokens = make(1, V, "bf16")[0][0], torch.full((T,), 9, dtype=torch.int32, device=DEV)
    r = kda.kda_token_logprobs(logits, tokens, top=4)
    want = reference(logits[-1:], tokens[-1:], 4)
    near(r.logp[-1:], want[0])
    assert torch.equal(r.top_token[-1:], want[4]) and abs(float(r.logp[0]) + math.log(V)) < 1e-4
    g = kda.kda_token_logprobs_backward(logits, tokens, r.lse, torch.ones(T, device=DEV), grad=logits)
    want = gradient(make(1, V, "bf16")[0], tokens[-1:], torch.ones(1, device=DEV), None)
    assert float((g[-1:].double() - want).norm() / want.norm()) < 3e-3


def test_argument_checks():
    logits, tokens = make(3, 100, "bf16")
    f = torch.zeros(3, device=DEV)
    call = kda.kda_token_logprobs
    for error, args, kw in [(TypeError, (logits.half(), tokens), {}), (TypeError, (logits, tokens.long()), {}),
                            (ValueError, (logits[0], tokens), {}), (ValueError, (logits.t(), tokens), {}),
                            (ValueError, (logits.cpu(), tokens), {}), (ValueError, (logits, tokens[:2]), {}),
                            (kda.KdaError, (logits, tokens), dict(top=33)), (kda.KdaError, (logits[:, :4], tokens), dict(top=5)),
                            (kda.KdaError, (logits, tokens), dict(top=-1))]:
        with pytest.raises(error):
            call(*args, **kw)
    back = kda.kda_token_logprobs_backward
    for error, over in [(ValueError, dict(entropy=f)), (ValueError, dict(grad_entropy=f)), (TypeError, dict(grad=logits.float())),
                        (ValueError, dict(grad=logits[:, :50])), (ValueError, dict(grad=logits.t().contiguous().t()))]:
        with pytest.raises(error):
            back(logits, tokens, f, f, **over)
    empty = call(logits[:0], tokens[:0], top=2, entropy=True)
    assert empty.logp.shape == (0,) and empty.top_token.shape == (0, 2)
    assert back(logits[:0], tokens[:0], f[:0], f[:0]).shape == (0, 100)
    assert kda.kda_get_device_error() == 0
