"""kda_rotary and kda_cache_append against a rotation in complex float64.

Tolerances: an output a cos - b sin is off by two or three roundings to float32 of products of a, b with a sine that is itself
off by 2^-32 of a turn and 2 units of its last place: 6e-7 of |a| + |b|, and then rounded once to its type."""

import math
from fractions import Fraction

import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


def frequencies(rot, base=10000.0):
    return base ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) / max(rot // 2, 1))


def turned(x, positions, inv_freq, layout, scale=1.0, sign=1.0):
    n = inv_freq.shape[0]
    y = x.double().clone()
    if n == 0:
        return y
    angle = positions.double()[:, None] * inv_freq
    turn = scale * torch.exp(1j * sign * torch.remainder(angle, 2 * math.pi))[:, None]
    if layout == "half":
        z = torch.complex(y[..., :n], y[..., n:2 * n]) * turn
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:2 * n:2], y[..., 1:2 * n:2]) * turn
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    return y


def near(got, want, x, rot, layout, scale=1.0):
    """Each place within the arithmetic's error; what is not rotated is copied."""
    y, n = x.double().abs(), rot // 2
    size = torch.zeros_like(y)
    if layout == "half":
        size[..., :n] = size[..., n:2 * n] = y[..., :n] + y[..., n:2 * n]
    else:
        size[..., 0:2 * n:2] = size[..., 1:2 * n:2] = y[..., 0:2 * n:2] + y[..., 1:2 * n:2]
    bound = 6e-7 * abs(scale) * size + torch.finfo(got.dtype).eps / 2 * want.abs() + 1e-37
    bound[..., rot:] = 0
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off - bound).max())


def randn(*shape, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(16, 16), (16, 4), (16, 2), (64, 64), (64, 32), (64, 20), (128, 128), (128, 64), (128, 6), (128, 0)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (3, 8, 2), (130, 5, 1), (1000, 4, 4)])
def test_sizes_and_layouts(dtype, layout, d, rot, T, Hq, Hkv):
    q, k = randn(T, Hq, d, dtype=dtype), randn(T, Hkv, d, dtype=dtype, seed=1)
    pos = torch.randint(0, 5000, (T,), device=DEV).int()
    f = frequencies(rot)
    for inverse in (False, True):
        a, b = kda.kda_rotary(q, k, pos, f, layout=layout, rotary_scale=1.25, inverse=inverse)
        sign = -1.0 if inverse else 1.0
        near(a, turned(q, pos, f, layout, 1.25, sign), q, rot, layout, 1.25)
        near(b, turned(k, pos, f, layout, 1.25, sign), k, rot, layout, 1.25)
        assert torch.equal(a[..., rot:], q[..., rot:])
    only, none = kda.kda_rotary(q, None, pos, f, layout=layout)
    assert none is None
    near(only, turned(q, pos, f, layout), q, rot, layout)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_and_negative_positions(dtype):
    """Where position * frequency is millions of radians: the reference takes the turns off in whole numbers."""
    d, T = 64, 40
    q = randn(T, 3, d, dtype=dtype)
    pos = torch.tensor([0, 1, 2, 1 << 20, (1 << 20) + 1, 2 ** 31 - 1, 2 ** 31 - 2, -1, -2 ** 31, -12345] * 4, device=DEV).int()
    f = torch.cat([frequencies(32), torch.full((16,), 1.0, dtype=torch.float64, device=DEV)])
    f[20], f[21], f[22], f[23] = 0.0, -0.75, 12.5, 3.0e-9
    turns = [[(int(p) * (int(float(x) / (2 * math.pi) * 2 ** 80))) % 2 ** 80 / 2 ** 80 for x in f] for p in pos.tolist()]
    angle = torch.tensor(turns, dtype=torch.float64, device=DEV) * 2 * math.pi
    n = 32
    z = torch.complex(q[..., :n].double(), q[..., n:].double()) * torch.exp(1j * angle)[:, None]
    want = torch.cat([z.real, z.imag], -1)
    got, _ = kda.kda_rotary(q, None, pos, f)
    # the frequency itself is known to 2^-53 of a radian: at 2^31 that is 2^-22 of one, at positions below 2^24 nothing
    slack = (pos.double().abs() * f.abs().max() * 2.0 ** -52)[:, None, None] * 4
    y = q.double().abs()
    size = (y[..., :n] + y[..., n:]).repeat(1, 1, 2)
    bound = (6e-7 + slack) * size + torch.finfo(DT[dtype]).eps / 2 * want.abs()
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_slices_of_a_projection_in_place_and_odd_strides(dtype, layout):
    T, Hq, Hkv, d = 50, 6, 2, 64
    f, pos = frequencies(32), torch.arange(T, device=DEV).int() + 70000
    for pad in (0, 1, 8):
        base = randn(T, (Hq + 2 * Hkv) * d + pad, dtype=dtype)
        view = lambda x: (x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)))
        q, k = view(base)
        want = kda.kda_rotary(q.contiguous(), k.contiguous(), pos, f, layout=layout)
        got = kda.kda_rotary(q, k, pos, f, layout=layout)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        work = base.clone()
        a, b = view(work)
        assert kda.kda_rotary(a, b, pos, f, layout=layout, q_out=a, k_out=b)[0] is a
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(work[:, (Hq + Hkv) * d:], base[:, (Hq + Hkv) * d:])


def test_angles_at_every_position():
    """Against turns counted with pi to 60 digits.  The angle is off by 2^-32 of a turn and by half a step of an eighth of one
    in 24 bits (1.5e-9 + 4.7e-8), its sine by two units of its last place and the scale's product (1.2e-7 + 6e-8),
    the sum's two products and itself by half a step each (1.2e-7 together): 3.6e-7 of |a| + |b|."""
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749446, 10 ** 61)
    d = 32 * 4
    pos = torch.tensor([0, 1, 3, 4097, (1 << 20) + 1, 2 ** 31 - 1, 2 ** 31 - 2, -1, -2 ** 31, -12345, 99999999], device=DEV).int()
    f = frequencies(d)
    f[:8] = torch.tensor([0.0, -0.75, 12.5, 3.0e-9, -1.0e-9, 0.3, 2 * math.pi, 1e6], dtype=torch.float64)
    turns = [[float((int(p) * Fraction(x) / (2 * pi)) % 1) for x in f.tolist()] for p in pos.tolist()]
    angle = torch.tensor(turns, dtype=torch.float64, device=DEV) * 2 * math.pi
    q, n = randn(pos.numel(), 5, d, dtype="f32"), d // 2
    for sign in (1, -1):
        z = torch.complex(q[..., :n].double(), q[..., n:].double()) * torch.exp(1j * sign * angle)[:, None]
        got, _ = kda.kda_rotary(q, None, pos, f, rotary_scale=1.0, inverse=sign < 0)
        size = (q.double().abs()[..., :n] + q.double().abs()[..., n:]).repeat(1, 1, 2)
        off = (got.double() - torch.cat([z.real, z.imag], -1)).abs() / size
        assert float(off.max()) <= 3.6e-7, (float(off.max()), int(off.argmax()))


def test_cosines_and_sines_of_angles_at_every_position():
    """The turned unit vectors, that is the cosine and the sine themselves.  The angle is off by 2^-32 of a turn and by half a step
    of an eighth of one in 24 bits, 16 * 2^-32 of a turn (1.5e-9 + 2.3e-8 radians, below 2^-25), either function by two units
    of its last place, at most 2^-22 of it."""
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749446, 10 ** 61)
    gen = torch.Generator().manual_seed(3)
    pos = torch.cat([torch.randint(-2 ** 31, 2 ** 31, (200,), generator=gen), torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1])]).int()
    d, f = 128, frequencies(128, 500000.0)
    f[::7] *= 1e5
    turns = [[float((int(p) * Fraction(x) / (2 * pi)) % 1) for x in f.tolist()] for p in pos.tolist()]
    angle = torch.tensor(turns, dtype=torch.float64, device=DEV) * 2 * math.pi
    unit = torch.zeros((pos.numel(), 1, d), device=DEV)
    unit[..., :d // 2] = 1
    got, _ = kda.kda_rotary(unit, None, pos.to(DEV), f)
    want = torch.cat([angle.cos(), angle.sin()], -1)[:, None]
    off = (got.double() - want).abs()
    assert bool((off <= 2.5e-8 + 2.0 ** -22 * want.abs() + 1e-15).all()), float((off - 2.0 ** -22 * want.abs()).max())


def test_the_inverse_is_the_gradient():
    T, H, d, rot = 7, 2, 16, 12
    f, pos = frequencies(rot), torch.arange(T, device=DEV).int() * 1000
    for layout in ("half", "interleaved"):
        x, g = randn(T, H, d, dtype="f32"), randn(T, H, d, dtype="f32", seed=4)
        grad, _ = kda.kda_rotary(g, None, pos, f, layout=layout, rotary_scale=0.8, inverse=True)
        want = x.double().clone().requires_grad_()
        n = rot // 2
        angle = (pos.double()[:, None] * f)[:, None]
        a, b = (want[..., :n], want[..., n:rot]) if layout == "half" else (want[..., 0:rot:2], want[..., 1:rot:2])
        u, v = 0.8 * (a * angle.cos() - b * angle.sin()), 0.8 * (b * angle.cos() + a * angle.sin())
        head = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
        (torch.cat([head, want[..., rot:]], -1) * g.double()).sum().backward()
        assert float((grad.double() - want.grad).abs().max()) < 5e-6
        # by differences: the map is linear, so a step of 1 is exact but for the arithmetic
        for t, h, i in ((0, 0, 0), (3, 1, 5), (6, 0, 11), (2, 1, 15)):
            up = x.clone()
            up[t, h, i] += 1
            y0, y1 = (kda.kda_rotary(z, None, pos, f, layout=layout, rotary_scale=0.8)[0].double() for z in (x, up))
            assert abs(float(((y1 - y0) * g.double()).sum()) - float(grad[t, h, i])) < 2e-5


def batch(rows, Hkv, d, ps, dtype, seed=0, extra=3, max_pages=None, behind=0):
    gen = torch.Generator().manual_seed(seed)
    lens = [n + past for n, past in rows]
    counts = [-(-n // ps) for n in lens]
    P, M = sum(counts) + extra, max_pages or max([1] + counts)
    perm = torch.randperm(P, generator=gen)
    table, at = torch.full((len(rows), M), -1, dtype=torch.int32), 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    cu = torch.tensor([0] + [n for n, _ in rows]).cumsum(0).int()
    T = int(cu[-1]) + behind
    return dict(k=randn(T, Hkv, d, dtype=dtype, seed=1), v=randn(T, Hkv, d, dtype=dtype, seed=2),
                k_pages=randn(P, Hkv, ps, d, dtype=dtype, seed=3), v_pages=randn(P, Hkv, ps, d, dtype=dtype, seed=4),
                block_table=table.to(DEV), seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV))


def places(rows, ps, table):
    """(token, position, page, slot) of every new token."""
    out, t = [], 0
    for b, (n, past) in enumerate(rows):
        for i in range(n):
            out.append((t, past + i, int(table[b, (past + i) // ps]), (past + i) % ps))
            t += 1
    return torch.tensor(out, device=DEV).view(-1, 4).unbind(1)


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ps", [1, 7, 16, 64])
@pytest.mark.parametrize("d,rot,layout", [(128, 128, "half"), (64, 20, "interleaved"), (16, 0, "half"), (64, 4, "half")])
def test_append(dtype, ps, d, rot, layout):
    rows = [(1, 0), (0, 5), (40, 13), (3, 100000), (0, 0), (17, 0), (129, 64)]
    Hq, Hkv = 6, 2
    a = batch(rows, Hkv, d, ps, dtype, behind=5)
    T = a["k"].shape[0]
    q, f = randn(T, Hq, d, dtype=dtype, seed=9), frequencies(rot)
    before = {n: a[n].clone() for n in ("k_pages", "v_pages")}
    q_out = torch.full_like(q, 7.0)
    got = kda.kda_cache_append(**a, q=q, q_out=q_out, inv_freq=f, layout=layout, rotary_scale=1.1)
    assert got is q_out and kda.kda_get_device_error() == 0
    t, pos, page, slot = places(rows, ps, a["block_table"])
    n = t.numel()
    near(q_out[:n], turned(q[:n], pos, f, layout, 1.1), q[:n], rot, layout, 1.1)
    assert bool((q_out[n:] == 7).all())                # tokens of no sequence
    near(a["k_pages"][page, :, slot], turned(a["k"][:n], pos, f, layout, 1.1), a["k"][:n], rot, layout, 1.1)
    assert torch.equal(a["v_pages"][page, :, slot], a["v"][:n])
    for name in ("k_pages", "v_pages"):                # every other place is as it was
        left = before[name].clone()
        left[page, :, slot] = a[name][page, :, slot]
        assert torch.equal(bits(left), bits(a[name]))
    again = dict(a, k_pages=before["k_pages"], v_pages=before["v_pages"])
    assert kda.kda_cache_append(**again, layout=layout) is None
    assert torch.equal(again["k_pages"][page, :, slot], a["k"][:n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_many_sequences_and_interleaved_pools(dtype):
    rows = [((b * 7) % 4, (b * 13) % 50) for b in range(3100)]
    a = batch(rows, 1, 16, 8, dtype)
    P = a["k_pages"].shape[0]
    pool = torch.zeros((P, 2, 1, 8, 16), dtype=DT[dtype], device=DEV)
    a.update(k_pages=pool[:, 0], v_pages=pool[:, 1])
    kda.kda_cache_append(**a)
    t, pos, page, slot = places(rows, 8, a["block_table"].cpu())
    assert torch.equal(pool[page, 0, :, slot], a["k"]) and torch.equal(pool[page, 1, :, slot], a["v"])
    assert kda.kda_get_device_error() == 0


def test_append_page_offsets_beyond_32_bits():
    a = batch([(300, 100)], 8, 128, 256, "bf16")
    P = (1 << 31) // (256 * 8 * 128) + 12
    k = torch.zeros((P, 8, 256, 128), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    a.update(k_pages=k, v_pages=v, block_table=torch.tensor([[P - 1, P - 3]], dtype=torch.int32, device=DEV))
    kda.kda_cache_append(**a)
    assert torch.equal(k[P - 1, :, 100:].transpose(0, 1), a["k"][:156]) and torch.equal(v[P - 3, :, :144].transpose(0, 1), a["v"][156:])
    assert kda.kda_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_bad_tables_lengths_and_borders_are_reported(dtype):
    rows, ps = [(5, 30), (20, 0), (3, 3)], 16
    for what, b, value, bit in [("block_table", (0, 2), -1, 0x20), ("block_table", (0, 2), 99, 0x20), ("block_table", (0, 2), 1 << 30, 0x20),
                                ("seq_lens", 0, 1 << 20, 0x20), ("seq_lens", 0, -1, 0x20), ("seq_lens", 0, 2 ** 31 - 1, 0x20),
                                ("seq_lens", 0, 2, 0x20), ("cu_seqlens", 0, 4, 0x1), ("cu_seqlens", 3, 1 << 20, 0x1)]:
        a = batch(rows, 2, 64, ps, dtype, max_pages=3)
        want = batch(rows, 2, 64, ps, dtype, max_pages=3)
        a[what][b] = value
        kda.kda_cache_append(**a)
        assert kda.kda_get_device_error() & bit
        t, pos, page, slot = places(rows, ps, want["block_table"])
        fine = (t >= 5) & (t < (25 if what == "cu_seqlens" else 28))
        assert torch.equal(a["k_pages"][page[fine], :, slot[fine]], a["k"][t[fine]])
        others = torch.ones(a["k_pages"].shape[0], dtype=torch.bool, device=DEV)
        others[want["block_table"][want["block_table"] >= 0].long()] = False
        assert torch.equal(a["k_pages"][others], want["k_pages"][others])


@pytest.mark.parametrize("B", [3, 40, 300])
def test_append_with_borders_in_any_order(B):
    """Every token is stored in the place that some sequence in order gives it, or not at all; where the first border is 0 a token
    that lies in one sequence alone is stored there; no other place changes."""
    gen = torch.Generator().manual_seed(B)
    T, ps, d = 2 * B + 7, 4, 16
    for kind in range(4):
        cu = torch.randint(0, T + 1, (B + 1,), generator=gen)
        if kind < 2:
            cu = cu.sort().values
            cu[torch.randint(0, B + 1, (2,), generator=gen)] = torch.tensor([T + 50, -3][kind])
        elif kind == 3:
            cu[torch.rand(B + 1, generator=gen) < 0.3] = 2 ** 31 - 1
        if kind != 2:
            cu[0] = 0
        cu = cu.int()
        lens, M = torch.full((B,), T), -(-T // ps)
        table = torch.arange(B * M, dtype=torch.int32).view(B, M)
        a = dict(k=randn(T, 1, d, dtype="f32", seed=kind), v=randn(T, 1, d, dtype="f32", seed=kind + 9), block_table=table.to(DEV),
                 seq_lens=lens.int().to(DEV), cu_seqlens=cu.to(DEV))
        pools = [torch.zeros((B * M, 1, ps, d), device=DEV) for _ in range(2)]
        kda.kda_cache_append(a["k"], a["v"], *pools, a["block_table"], a["seq_lens"], a["cu_seqlens"])
        falls = bool((cu[1:] < cu[:-1]).any() or (cu > T).any() or cu[0] != 0)
        assert kda.kda_get_device_error() == (0x1 if falls else 0)
        flat = pools[0].view(B, M * ps, d).cpu()
        k, c, stored = a["k"][:, 0].cpu(), cu.tolist(), [0] * T
        inside = [[b for b in range(B) if c[b] <= t < c[b + 1]] for t in range(T)]     # of any sequence, in order or not
        for b in range(B):
            for p in flat[b].any(1).nonzero()[:, 0].tolist():
                t = c[b + 1] - (T - p)                 # the token that b's borders put at position p
                assert 0 <= c[b] <= t < c[b + 1] <= T and (b > 0 or c[0] == 0) and torch.equal(flat[b, p], k[t])
                stored[t] += 1
        for t in range(T):
            assert stored[t] <= 1
            if len(inside[t]) == 1 and c[0] == 0:
                b = inside[t][0]
                assert stored[t] == (c[b] >= 0 and c[b + 1] <= T)
        assert torch.equal(pools[1].any(3), pools[0].any(3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_more_tokens_than_the_length_holds(dtype):
    """Tokens with a position below 0 are not stored; the others of their row are, and attention lets them see each other."""
    rows, ps = [(5, 30), (20, 0), (3, 3)], 16
    a, old = batch(rows, 2, 64, ps, dtype), batch(rows, 2, 64, ps, dtype)
    a["seq_lens"][1] = 13                              # the first seven of 20 lie before position 0
    q, f = randn(28, 4, 64, dtype=dtype), frequencies(64)
    out = kda.kda_cache_append(**a, q=q, inv_freq=f)
    assert kda.kda_get_device_error() == 0x20
    t, pos, page, slot = places([(5, 30), (13, 0), (3, 3)], ps, old["block_table"])
    t = torch.where(t >= 5, t + 7, t)                  # tokens 12 .. 24 at positions 0 .. 12
    near(a["k_pages"][page, :, slot], turned(a["k"][t], pos, f, "half"), a["k"][t], 64, "half")
    assert torch.equal(a["v_pages"][page, :, slot], a["v"][t])
    for name in ("k_pages", "v_pages"):
        left = old[name].clone()
        left[page, :, slot] = a[name][page, :, slot]
        assert torch.equal(bits(left), bits(a[name]))
    near(out[t], turned(q[t], pos, f, "half"), q[t], 64, "half")
    o = kda.kda_attention_prefill(out, a["k_pages"], a["v_pages"], a["block_table"], a["seq_lens"], a["cu_seqlens"], scale=0.1)
    assert kda.kda_get_device_error() == 0x20 and not o[5:12].any()
    cu = torch.tensor([0, 13], dtype=torch.int32, device=DEV)
    alone = kda.kda_attention_prefill(out[12:25].contiguous(), a["k_pages"], a["v_pages"], a["block_table"][1:2], a["seq_lens"][1:2], cu, scale=0.1)
    assert kda.kda_get_device_error() == 0
    # the same sums in an order that may differ: outputs twice rounded, below 3 in size
    assert float((o[12:25].double() - alone.double()).abs().max()) <= 2 * 3 * torch.finfo(DT[dtype]).eps


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_leaves_sequences_with_bad_borders_alone(dtype):
    """They count as empty: nothing of theirs is stored, and their queries' outputs stay as they were."""
    rows, ps = [(5, 30), (20, 0), (3, 3)], 16
    for b, value, left in ((0, 4, range(0, 5)), (0, -2, range(0, 5)), (3, 29, range(25, 28)), (3, 1 << 20, range(25, 28)),
                           (3, 24, range(25, 28))):
        a, old = batch(rows, 2, 64, ps, dtype), batch(rows, 2, 64, ps, dtype)
        a["cu_seqlens"][b] = value
        q = randn(28, 4, 64, dtype=dtype)
        out = torch.full_like(q, 7.0)
        kda.kda_cache_append(**a, q=q, q_out=out)
        assert kda.kda_get_device_error() == 0x1
        t, pos, page, slot = places(rows, ps, old["block_table"])
        bad = torch.tensor([int(i) in left for i in t], device=DEV)
        for name in ("k", "v"):
            pool = a[name + "_pages"][page, :, slot]
            assert torch.equal(bits(pool[bad]), bits(old[name + "_pages"][page, :, slot][bad]))
            assert torch.equal(pool[~bad], a[name][t[~bad]])
        assert bool((out[t[bad]] == 7).all()) and torch.equal(out[t[~bad]], q[t[~bad]])


def test_streams_and_graphs():
    rows = [(1, n) for n in (0, 31, 32, 500)]
    a = batch(rows, 2, 64, 16, "bf16")
    q, f = randn(4, 8, 64, dtype="bf16"), frequencies(64)
    base = {n: a[n].clone() for n in ("k_pages", "v_pages")}
    want = kda.kda_cache_append(**a, q=q, inv_freq=f)
    done = {n: a[n].clone() for n in base}
    side = torch.cuda.Stream()
    for n in base:
        a[n].copy_(base[n])
    side.wait_stream(torch.cuda.current_stream())
    got = kda.kda_cache_append(**a, q=q, inv_freq=f, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a[n], done[n]) for n in base)
    graph = torch.cuda.CUDAGraph()
    pos = torch.tensor([3, 5, 7, 9], dtype=torch.int32, device=DEV)
    with torch.cuda.graph(graph):
        out = kda.kda_cache_append(**a, q=q, inv_freq=f)
        turn, _ = kda.kda_rotary(q, None, pos, f)
    for n in base:
        a[n].copy_(base[n])
    pos += 11
    graph.replay()
    assert torch.equal(out, want) and all(torch.equal(a[n], done[n]) for n in base)
    assert torch.equal(turn, kda.kda_rotary(q, None, pos, f)[0])


def test_argument_checks():
    q, k, f = randn(4, 8, 64, dtype="bf16"), randn(4, 2, 64, dtype="bf16"), frequencies(64)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    for error, args, kw in [(TypeError, (q.half(), None, pos, f), {}), (TypeError, (q, k.float(), pos, f), {}),
                            (TypeError, (q, k, pos.long(), f), {}), (TypeError, (q, k, pos, f.float()), {}),
                            (ValueError, (q, k[:3], pos, f), {}), (ValueError, (q, k, pos[:3], f), {}),
                            (ValueError, (q.cpu(), k, pos, f), {}), (ValueError, (q, k.cpu(), pos, f), {}),
                            (ValueError, (q, k, pos, f), dict(layout="other")), (ValueError, (q[0], k, pos, f), {}),
                            (ValueError, (q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, f), {}),
                            (ValueError, (q, None, pos, f), dict(k_out=k)), (ValueError, (q, k, pos, f), dict(q_out=q[:, :4])),
                            (kda.KdaError, (q, k, pos, torch.cat([f, f])), {}), (kda.KdaError, (q, k, pos, f), dict(rotary_scale=math.inf)),
                            (kda.KdaError, (randn(4, 2, 32, dtype="bf16"), None, pos, f[:4]), {})]:
        with pytest.raises(error):
            kda.kda_rotary(*args, **kw)
    assert kda.kda_rotary(q[:0], k[:0], pos[:0], f)[0].shape == (0, 8, 64)
    a = batch([(3, 0), (1, 5)], 2, 64, 16, "bf16")
    q = randn(4, 8, 64, dtype="bf16")
    for error, over in [(TypeError, dict(v=a["v"].float())), (ValueError, dict(v=a["v"][:, :1])), (ValueError, dict(k_pages=a["k_pages"][0])),
                        (ValueError, dict(v_pages=a["v_pages"][:1])), (ValueError, dict(cu_seqlens=a["cu_seqlens"][:2])),
                        (ValueError, dict(q_out=q)), (TypeError, dict(seq_lens=a["seq_lens"].long())), (ValueError, dict(q=q[:2])),
                        (ValueError, dict(k_pages=a["k_pages"].transpose(1, 2).contiguous().transpose(1, 2)))]:
        with pytest.raises(error):
            kda.kda_cache_append(**{**a, **over})
    assert kda.kda_get_device_error() == 0
