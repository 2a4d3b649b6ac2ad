"""kda_beam_select against a float64 selection, with ties, masks and rows that offer nothing.

Random scores of these sizes lie far enough apart (about 1e-3 between neighbours, float32 resolves 2e-6) for
the choice itself to be compared; scores agree to 1e-5 of their size (float32, a sum of up to 262,144 terms)."""

import numpy as np
import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NINF = -float("inf")


def reference(logits, bs, finished=None, eos=-1):
    """(scores, parent, token, finished) by the definition, the sum in float64 and the score's three additions in
    float32 as the definition has them, lowest place first among equals."""
    N, K = bs.shape
    x = logits.double().cpu().numpy().reshape(N, K, -1)
    V = x.shape[2]
    with np.errstate(all="ignore"):
        m = x.max(2, keepdims=True)
        lse = m.astype(np.float32) + np.log(np.exp(x - m).sum(2, keepdims=True)).astype(np.float32)
        s = (bs.cpu().numpy()[:, :, None] + (x.astype(np.float32) - lse)).astype(np.float64)
    if finished is not None:
        f = finished.cpu().numpy() != 0
        for n, b in zip(*np.nonzero(f)):
            s[n, b] = NINF
            s[n, b, eos] = float(bs[n, b])
    s[np.isnan(s)] = NINF
    flat = s.reshape(N, K * V)
    at = np.stack([np.lexsort((np.arange(K * V), -flat[n]))[:K] for n in range(N)])
    parent = at // V + np.arange(N)[:, None] * K
    token = at % V
    done = np.zeros((N, K), bool) if finished is None else np.take_along_axis(f, at // V, 1)
    if eos >= 0:
        done = done | (token == eos)
    return np.take_along_axis(flat, at, 1), parent, token, done


def check(logits, bs, finished=None, eos=-1, **kw):
    ref = reference(logits, bs, finished, eos)
    s, parent, token, done = kda.kda_beam_select(logits, bs, finished=finished, eos_token=eos, **kw)
    torch.cuda.synchronize()
    s, parent, token = s.cpu().numpy(), parent.cpu().numpy(), token.cpu().numpy()
    fin = np.isfinite(ref[0])
    assert np.array_equal(fin, np.isfinite(s)) and np.array_equal(s[~fin], ref[0][~fin])
    assert np.abs(s[fin] - ref[0][fin]).max(initial=0) <= 1e-5 * max(1.0, np.abs(ref[0][fin]).max(initial=0))
    assert np.array_equal(parent, ref[1]) and np.array_equal(token, ref[2])
    if done is not None:
        assert np.array_equal(done.cpu().numpy() != 0, ref[3])
    assert kda.kda_get_device_error() == 0
    return s, parent, token


def inputs(N, K, V, dtype, seed, std=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = std * torch.randn((N * K, V), device=DEV, generator=g)
    bs = -20 * torch.rand((N, K), device=DEV, generator=g)
    return logits.to(DT[dtype]), bs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (1, 1, 7), (2, 4, 3), (3, 2, 255), (1, 4, 4096), (5, 3, 4097), (2, 8, 8192),
                                   (2, 5, 8193), (3, 4, 32001), (7, 8, 50000), (1, 16, 131072), (2, 32, 20000),
                                   (1, 3, 262144), (40, 2, 1000)])
def test_sizes(dtype, N, K, V):
    check(*inputs(N, K, V, dtype, N * 1000 + K))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_further_apart_than_the_vocabulary(dtype):
    wide, bs = inputs(3, 4, 5003, dtype, 5)
    wide[:, 4990:] = 100.0                             # padding past the vocabulary: not to be read
    check(wide[:, :4990], bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_finished_beams_and_a_forbidden_word(dtype):
    logits, bs = inputs(6, 4, 9001, dtype, 6)
    logits[:, 17] = NINF
    fin = (torch.rand((6, 4), device=DEV) < 0.4).to(torch.uint8)
    fin[0] = 1
    check(logits, bs, fin, 2)
    check(logits, bs, torch.zeros_like(fin), 9000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_only_the_first_beam_lives(dtype):
    """The start of a search: every beam but the first has no score yet."""
    logits, bs = inputs(4, 8, 30000, dtype, 7)
    bs[:, 1:] = NINF
    _, parent, _ = check(logits, bs)
    assert np.array_equal(parent % 8, np.zeros((4, 8)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_offer_nothing(dtype):
    """NaN, +inf and all-masked rows, beams without a score, fewer words than beams, and nothing at all."""
    logits, bs = inputs(4, 4, 12345, dtype, 8)
    logits[0, 77] = float("nan")
    logits[1, 12000] = float("inf")
    logits[2] = NINF
    logits[5, 3:] = NINF
    bs[1, 0], bs[1, 2], bs[1, 3] = NINF, float("nan"), NINF
    bs[2] = NINF
    logits[12:16] = NINF
    check(logits, bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", [-1e4, -1e10, -3e38, "lowest", NINF])
def test_words_masked_by_a_large_negative_number(dtype, fill):
    """A grammar leaves a few words, the others hold the mask's value: whole parts of the row, and whole rows."""
    logits, bs = inputs(4, 4, 60000, dtype, 20)
    fill = float(torch.finfo(DT[dtype]).min) if fill == "lowest" else fill
    keep = torch.zeros(60000, dtype=torch.bool, device=DEV)
    keep[[5, 31000, 31001, 45678, 59999]] = True
    logits = torch.where(keep, logits, torch.full_like(logits, fill))
    check(logits, bs)
    logits[1:7] = fill                                 # rows without a word left
    _, parent, token = check(logits, bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", [-200.0, -1e4, -1e10, "lowest"])
@pytest.mark.parametrize("N,K", [(320, 1), (40, 8), (2, 4)])
def test_weak_words_behind_masked_ones_and_strong_ones(dtype, fill, N, K):
    """What a thread has met so far may be masks alone when others have already met the best words: the weak words
    that it meets then are no candidates, but belong to the sum as they are."""
    V, chunk = 40000, 8192 if dtype == "bf16" else 4096
    logits, bs = inputs(N, K, V, dtype, 30)
    fill = float(torch.finfo(DT[dtype]).min) if fill == "lowest" else fill
    g = torch.Generator(device=DEV).manual_seed(31)
    few = torch.rand(V, device=DEV, generator=g) < 0.002
    check(torch.where(few, logits, torch.full_like(logits, fill)), bs)
    strong, weak = torch.zeros(V, dtype=torch.bool, device=DEV), torch.zeros(V, dtype=torch.bool, device=DEV)
    strong[torch.arange(chunk + 5, 2 * chunk - 60, 150, device=DEV)] = True
    weak[torch.arange(2 * chunk + 70, V, 331, device=DEV)] = True
    high, low = logits.abs() + 9, -logits.abs() - 1
    check(torch.where(strong, high, torch.where(weak, low, torch.full_like(logits, fill))), bs)
    if fill != float(torch.finfo(DT[dtype]).min):      # a mask that is added leaves the masked words different
        check(torch.where(strong, high, torch.where(weak, low, logits + fill)), bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_in_order(dtype):
    """Rising and falling rows: every chunk of the one holds larger logits than all before it."""
    ramp = torch.linspace(-20, 20, 100000, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    noise = 1e-3 * torch.rand((8, 100000), device=DEV, generator=g)
    logits = (torch.stack([ramp, ramp.flip(0)] * 4) + noise).to(DT[dtype])
    bs = -3.0 * torch.arange(8, device=DEV, dtype=torch.float32).view(2, 4) / 7
    check(logits, bs)
    check(100 * logits, bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [-20.0, -1e4])
def test_rising_rows_cost_a_few_reads_more(dtype, first):
    """Rows whose every word is larger than those before it (behind a masked first stretch, too) overflow the lists that
    a part keeps.  A search with a bound on its passes (ten, each some ten reads of the row at most) stays within a
    hundred times the same rows in random order; one that drops a list's length of words a pass does not."""
    N, K, V = 40, 8, 400000
    row = torch.linspace(-20, 20, V, device=DEV)
    row[:V // 40] = first
    order = torch.randperm(V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    bs = -50.0 * torch.arange(K, device=DEV, dtype=torch.float32).repeat(N, 1)
    times = []
    for r in (row, row[order]):
        r = r.to(DT[dtype])
        logits = r.repeat(N * K, 1)
        best = torch.sort(r.float(), descending=True, stable=True).indices[:K].tolist()
        took = []
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            _, parent, token, _ = kda.kda_beam_select(logits, bs)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        assert token.tolist() == [best] * N and parent.tolist() == [[n * K] * K for n in range(N)]
        times.append(min(took))
    assert times[0] <= 100 * times[1], times


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2, 2500, 40001])
def test_ties_go_to_the_lowest_place(dtype, V):
    """Equal logits within a row and equal rows: the same arithmetic gives the same score wherever it stands."""
    g = torch.Generator(device=DEV).manual_seed(V)
    row = torch.randint(-2, 3, (V,), device=DEV, generator=g).float()
    logits = row.repeat(8, 1).to(DT[dtype])
    bs = torch.full((2, 4), -3.0, device=DEV)
    s, parent, token, _ = kda.kda_beam_select(logits, bs)
    top = torch.nonzero(row == row.max())[:, 0].tolist()
    places = [(b, v) for b in range(4) for v in top][:4]
    if len(places) < 4:                                # V = 2 may hold one word of the best value a beam
        places = sorted(((b, v) for b in range(4) for v in range(V)), key=lambda c: (-float(row[c[1]]), c))[:4]
    for n in range(2):
        assert [(int(p) - 4 * n, int(t)) for p, t in zip(parent[n], token[n])] == places
    assert bool((s[:, 0] == s[:, 3]).all()) or len(top) < 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 9000, 70001])
def test_scores_that_round_together(dtype, V):
    """Beside a beam score of -2^27, whose neighbours are 16 away, every word of a beam (x - lse between -12 and
    -4) rounds to the same score, whatever its logit: the choice is by place, and the words with the largest
    logits have no claim to it."""
    logits, _ = inputs(2, 4, V, dtype, 10, std=0.1)
    bs = torch.full((2, 4), -2.0 ** 27, device=DEV)
    bs[1, 0] = -2.0 ** 28
    s, parent, token, _ = kda.kda_beam_select(logits, bs)
    assert parent.tolist() == [[0] * 4, [5] * 4] and token.tolist() == [[0, 1, 2, 3]] * 2
    lse = torch.logsumexp(logits.double(), 1)
    want = (bs.double().view(8) + (logits.double().mean(1) - lse)).float()       # the same for the row's other words
    assert bool((s[0] == want[0]).all()) and bool((s[1] == want[5]).all())


def test_scores_that_round_together_in_part():
    """Scores that collapse to a few values, compared with the same float32 arithmetic by torch."""
    logits, _ = inputs(3, 4, 20011, "f32", 11, std=2.0)
    bs = torch.full((3, 4), -2.0 ** 22, device=DEV) + torch.arange(4, device=DEV)[None, :]
    lse = torch.logsumexp(logits.double(), 1, keepdim=True).float()
    s = (bs.view(12, 1) + (logits - lse)).view(3, -1)
    got, parent, token, _ = kda.kda_beam_select(logits, bs)
    # lse differs by a rounding at most, which moves a score to its neighbour only where x - lse sits at a tie of
    # the rounding: the values are compared exactly, the places by their own scores
    for n in range(3):
        want = torch.sort(s[n], descending=True, stable=True)
        place = (parent[n].long() - 4 * n) * 20011 + token[n].long()
        assert len(set(place.tolist())) == 4
        assert float((got[n] - want.values[:4]).abs().max()) <= 0.5
        for a, b in zip(range(3), range(1, 4)):
            assert got[n, a] > got[n, b] or (got[n, a] == got[n, b] and place[a] < place[b])


def known_sums(N, K, V, dtype):
    """Logits of -20 behind one of 50 in the third place, beside which no sum of V others up to 9 shows in float32 (V e^-41
    is below 2^-26): a row's log-sum is 50, and every score is known to the bit."""
    logits = torch.full((N * K, V), -20.0, dtype=DT[dtype], device=DEV)
    logits[:, 2] = 50.0
    return logits


def check_exactly(logits, bs):
    """Scores, parents and tokens of rows whose log-sum is 50, the lowest place first among equal scores."""
    N, K = bs.shape
    V = logits.shape[1]
    s = (bs.view(N * K, 1) + (logits.float() - 50.0)).view(N, K * V)
    best = torch.sort(s, dim=1, descending=True, stable=True)
    score, parent, token, _ = kda.kda_beam_select(logits, bs)
    rows = torch.arange(N, device=DEV)[:, None] * K
    assert torch.equal(score, best.values[:, :K])
    wrong = ((parent - rows) * V + token != best.indices[:, :K]).any(1).nonzero()[:, 0].tolist()
    assert not wrong, (len(wrong), N)


# float32 logits from 7.25 up, 2^-21 apart, bf16 ones from 4 up, 2^-5 apart; the beam scores' neighbours lie further apart
NEIGHBOURS = {"f32": (7.25, 2.0 ** -21, (-30.0, -300.0)), "bf16": (4.0, 2.0 ** -5, (-2.0 ** 18, -2.0 ** 19, -1.3e5))}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_logits_beside_their_upper_neighbour(dtype):
    """Two words at some logit x, and later two at the next larger one.  Where the four score the same, the two lower
    places win, although a list of the largest logits names but one of them."""
    start, step, scores = NEIGHBOURS[dtype]
    for beam in scores:
        logits, bs = known_sums(64, 3, 2048, dtype), torch.full((64, 3), NINF, device=DEV)
        bs[:, 0] = beam
        x = start + step * torch.arange(64, device=DEV)
        logits[::3, 5] = logits[::3, 6] = x.to(DT[dtype])
        logits[::3, 1000] = logits[::3, 1001] = (x + step).to(DT[dtype])
        check_exactly(logits, bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 4, 16, 32])
@pytest.mark.parametrize("V", [300, 9000, 70001])
def test_neighbouring_logits_that_round_together(dtype, K, V):
    """Few values, many words of each, a few of which share a score: places and scores to the bit."""
    rng = np.random.default_rng(V + K)
    start, step, scores = NEIGHBOURS[dtype]
    for beam in scores:
        N = 24
        logits, bs = known_sums(N, K, V, dtype), torch.full((N, K), NINF, device=DEV)
        bs[:, 0] = beam * torch.from_numpy(rng.uniform(1, 2, N)).float().to(DEV)
        if K > 2:
            bs[:, 1] = bs[:, 0]
        for r in range(N * K):
            words = torch.from_numpy(3 + rng.permutation(V - 3)[:3 * K]).to(DEV)
            values = start + step * torch.from_numpy(rng.integers(0, 32, 3 * K)).to(DEV)
            logits[r, words] = values.to(DT[dtype])
        check_exactly(logits, bs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_of_both_signs_are_one_value(dtype):
    logits = torch.full((2, 5000), -5.0, device=DEV)
    logits[:, 4000], logits[:, 70], logits[:, 71] = 0.0, -0.0, 0.0
    s, parent, token, _ = kda.kda_beam_select(logits.to(DT[dtype]), torch.tensor([[-1.0, -1.0]], device=DEV))
    assert parent.tolist() == [[0, 0]] and token.tolist() == [[70, 71]]


def test_in_place_and_reproducible():
    logits, bs = inputs(9, 6, 33333, "bf16", 12)
    fin = (torch.rand((9, 6), device=DEV) < 0.3).to(torch.uint8)
    a = kda.kda_beam_select(logits, bs, finished=fin, eos_token=1)
    b2, f2 = bs.clone(), fin.clone()
    b = kda.kda_beam_select(logits, b2, finished=f2, eos_token=1, scores_out=b2, finished_out=f2)
    assert b[0] is b2 and all(torch.equal(x, y) for x, y in zip(a, b))


def test_argument_checks():
    logits, bs = inputs(2, 4, 100, "f32", 13)
    with pytest.raises(TypeError):
        kda.kda_beam_select(logits.half(), bs)
    with pytest.raises(TypeError):
        kda.kda_beam_select(logits, bs.double())
    with pytest.raises(ValueError):
        kda.kda_beam_select(logits[:7], bs)
    with pytest.raises(ValueError):
        kda.kda_beam_select(logits.t().contiguous().t(), bs)
    with pytest.raises(kda.KdaError):
        kda.kda_beam_select(logits, bs, eos_token=100)
    with pytest.raises(kda.KdaError):                  # finished beams need a word to go on with
        kda.kda_beam_select(logits, bs, finished=torch.zeros((2, 4), dtype=torch.uint8, device=DEV))
    with pytest.raises(kda.KdaError):                  # 33 beams
        kda.kda_beam_select(torch.zeros((33, 10), device=DEV), torch.zeros((1, 33), device=DEV))
