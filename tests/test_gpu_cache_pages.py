"""kda_state_fork, kda_cache_fork, kda_cache_compact and kda_copy_pages against their definitions, step by step
in plain Python.  Everything here is moved, not computed: all comparisons are exact."""

import numpy as np
import pytest
import torch

import kda_gated_delta_03_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def pool_of(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(dtype)


# ---- states ----
def state_fork_reference(idx, parent):
    B = len(idx)
    out, first = [None] * B, {}
    for i, p in enumerate(parent):
        if 0 <= p < B and p not in first:
            first[p] = i
    free = [idx[r] for r in range(B) if r not in first]
    copies, extra = [], [i for i, p in enumerate(parent) if 0 <= p < B and first[p] != i]
    for p, i in first.items():
        out[i] = idx[p]
    for i, slot in zip(extra, free):
        out[i] = slot
        copies.append((idx[parent[i]], slot))
    for i, slot in zip([i for i, p in enumerate(parent) if not 0 <= p < B], free[len(extra):]):
        out[i] = slot
    return out, copies


@pytest.mark.parametrize("B,L,slot,dtype", [(1, 1, (1, 16, 16), torch.float32), (4, 2, (3, 16, 16), torch.bfloat16),
                                            (64, 1, (2, 128, 128), torch.float32), (257, 3, (1, 64, 64), torch.bfloat16),
                                            (1000, 1, (8,), torch.bfloat16), (8192, 1, (4,), torch.float32)])
@pytest.mark.parametrize("kind", ["same", "one", "random", "with_new", "all_new", "swap"])
def test_state_fork(B, L, slot, dtype, kind):
    rng = np.random.default_rng(B + len(kind))
    S = B + 3
    idx = rng.permutation(S)[:B]
    parent = {"same": np.arange(B), "one": np.full(B, B // 2), "random": rng.integers(0, B, B),
              "with_new": np.where(rng.random(B) < 0.3, -1, rng.integers(0, B, B)), "all_new": np.full(B, -1),
              "swap": np.arange(B)[::-1]}[kind]
    pool = pool_of((L, S, *slot), B, dtype)
    want_idx, copies = state_fork_reference(idx.tolist(), parent.tolist())
    want = pool.clone()
    for s, d in copies:
        want[:, d] = pool[:, s]
    out = kda.kda_state_fork(pool, dev(idx), dev(parent))
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    assert out.tolist() == want_idx and torch.equal(pool, want)
    assert sorted(out.tolist()) == sorted(idx.tolist())
    for i, p in enumerate(parent[:300]):               # every row holds its parent's state
        if p >= 0:
            assert torch.equal(pool[:, want_idx[i]], want[:, want_idx[i]])


def test_state_fork_of_several_pools_and_strided_layers():
    big = pool_of((2, 3, 10, 4, 16, 16), 1, torch.float32)
    a, b = big[:, 1], pool_of((1, 12, 40), 2, torch.float32)
    idx, parent = [7, 2, 9, 0], [1, 1, 3, 1]
    want_idx, copies = state_fork_reference(idx, parent)
    wb, wbig = b.clone(), big.clone()
    for s, d in copies:
        wbig[:, 1, d], wb[:, d] = big[:, 1, s], b[:, s]
    out = kda.kda_state_fork((a, b), dev(idx), dev(parent))
    torch.cuda.synchronize()
    assert out.tolist() == want_idx and torch.equal(big, wbig) and torch.equal(b, wb)


def test_state_fork_reports_bad_rows():
    pool = pool_of((1, 4, 8), 3, torch.float32)
    before = pool.clone()
    out = kda.kda_state_fork(pool, dev([0, 1, 2]), dev([0, 5, -7]))
    assert kda.kda_get_device_error() == 0x80
    assert out.tolist() == [0, 1, 2] and torch.equal(pool, before)
    out = kda.kda_state_fork(pool, dev([0, 1, 99]), dev([0, 0, 1]))
    assert kda.kda_get_device_error() == 0x2
    assert out.tolist() == [0, 99, 1] and torch.equal(pool, before)


# ---- cache fork ----
def cache_fork_reference(table, lens, parent, ref, ps, grow):
    """The new tables, and the copies (row, src, dst); None where the pool has no page left."""
    R2, M, P = len(parent), table.shape[1], len(ref)
    ref = ref.copy()
    first = {}
    for i, p in enumerate(parent):
        if p >= 0:
            first.setdefault(p, i)
    for r, n in enumerate(lens):
        for j in range(-(-n // ps)):
            ref[table[r, j]] -= 1
    out, rows = np.full((R2, M), -1, np.int32), []
    for i, p in enumerate(parent):
        n = int(lens[p]) if p >= 0 else 0
        copy = n % ps != 0 and first[p] != i
        shared = n // ps if copy else -(-n // ps)
        for j in range(shared):
            out[i, j] = table[p, j]
            ref[table[p, j]] += 1
        rows.append((p, n, copy, shared, n + int(grow[i])))
    free = [p for p in range(P) if ref[p] == 0][::-1]
    new_lens, copies, exhausted = [], [], False
    for i, (p, n, copy, shared, new) in enumerate(rows):
        have = new
        for j in range(shared, -(-new // ps)):
            if not free:
                have, exhausted = min(have, j * ps), True
                continue
            out[i, j] = free.pop()
            ref[out[i, j]] = 1
        if copy and out[i, n // ps] >= 0:
            copies.append((i, table[p, n // ps], out[i, n // ps]))
        new_lens.append(have)
    return out, new_lens, ref, copies, exhausted


def random_cache(R, M, ps, P, rng, groups=1):
    """Rows in groups that share their first whole pages; random pages of the pool."""
    lens = np.repeat(rng.integers(0, M * ps + 1, -(-R // groups)), groups)[:R]
    perm, at = rng.permutation(P), 0
    table = np.full((R, M), -1, np.int32)
    for r in range(R):
        c = -(-int(lens[r]) // ps)
        lead = r // groups * groups
        shared = int(lens[r]) // ps // 2 if r != lead else 0
        table[r, :shared] = table[lead, :shared]
        table[r, shared:c] = perm[at:at + c - shared]
        at += c - shared
    assert at <= P
    ref = np.bincount(table[table >= 0], minlength=P).astype(np.int32)
    return table, lens.astype(np.int32), ref


def run_fork(table, lens, parent, ref, ps, grow, pools, in_place=False):
    want_t, want_l, want_r, copies, exhausted = cache_fork_reference(table, lens, parent, ref, ps, grow)
    want = [p.clone() for p in pools]
    for _, s, d in copies:
        for w, p in zip(want, pools):
            w[:, d] = p[:, s]
    R2 = len(parent)
    src, dst = torch.full((R2,), -5, dtype=torch.int32, device=DEV), torch.full((R2,), -5, dtype=torch.int32, device=DEV)
    r = dev(ref)
    t2, l2, r2 = kda.kda_cache_fork(dev(table), dev(lens), dev(parent), r, ps, grow=dev(grow), pools=pools,
                                    ref_count_out=None if in_place else torch.empty_like(r), copy_src=src, copy_dst=dst)
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == (0x40 if exhausted else 0)
    assert np.array_equal(t2.cpu().numpy(), want_t)
    assert l2.tolist() == want_l
    assert np.array_equal(r2.cpu().numpy(), want_r)
    assert in_place or np.array_equal(r.cpu().numpy(), ref)
    exp = {i: (s, d) for i, s, d in copies}
    assert list(zip(src.tolist(), dst.tolist())) == [exp.get(i, (-1, -1)) for i in range(R2)]
    for w, p in zip(want, pools):
        assert torch.equal(w, p)
    return want_t, np.array(want_l, np.int32), want_r


@pytest.mark.parametrize("R,M,ps", [(1, 1, 1), (4, 9, 16), (6, 40, 7), (64, 12, 16), (300, 5, 3), (3, 2000, 1), (2100, 3, 4)])
@pytest.mark.parametrize("kind", ["same", "one", "random", "free", "reverse"])
def test_cache_fork(R, M, ps, kind):
    rng = np.random.default_rng(R * 7 + M + len(kind))
    P = 3 * R * M + 5
    table, lens, ref = random_cache(R, M - (M > 1), ps, P, rng, groups=2)
    table = np.concatenate([table, np.full((R, M - table.shape[1]), -1, np.int32)], 1)
    parent = {"same": np.arange(R), "one": np.full(R, R // 2), "random": rng.integers(-1, R, R), "free": np.full(R, -1),
              "reverse": np.arange(R)[::-1]}[kind]
    room = M * ps - np.where(parent >= 0, lens[parent], 0)
    grow = np.minimum(rng.integers(0, 2 * ps + 2, R), room)
    pools = [pool_of((2, P, 8), R), pool_of((1, P, 2, 16), M, torch.float32)]
    run_fork(table, lens, parent, ref, ps, grow, pools, in_place=kind in ("one", "free"))


@pytest.mark.parametrize("R,M,ps,slot", [(4, 9, 16, 1 << 19), (6, 40, 7, 1 << 17), (64, 12, 16, 8192), (300, 5, 3, 2048),
                                         (2100, 3, 4, 512), (4, 9, 16, 65536), (4, 9, 16, 65536 + 64)])
@pytest.mark.parametrize("kind", ["one", "random"])
def test_cache_fork_of_large_pages(R, M, ps, slot, kind):
    """More bytes than the bookkeeping's own CTAs move, and either side of that limit."""
    rng = np.random.default_rng(R + M + slot)
    P = 2 * R * M + 5
    table, lens, ref = random_cache(R, M - 1, ps, P, rng)
    table = np.concatenate([table, np.full((R, 1), -1, np.int32)], 1)
    parent = np.full(R, R // 2) if kind == "one" else rng.integers(-1, R, R)
    grow = rng.integers(0, ps + 1, R)
    run_fork(table, lens, parent, ref, ps, grow, [pool_of((2, P, slot), R)])


def test_cache_fork_of_pages_as_long_as_lengths_go():
    """A length and a page together pass 2^31 here."""
    ps = (1 << 30) + 5
    table, ref = np.array([[2], [0]], np.int32), np.array([1, 0, 1, 0], np.int32)
    run_fork(table, np.array([ps, ps - 1], np.int32), [0, 0, 1, 1, -1], ref, ps, [0, 0, 1, 0, 0], [pool_of((1, 4, 8), 1)])


def test_cache_fork_frees_every_row():
    rng = np.random.default_rng(8)
    table, lens, ref = random_cache(9, 6, 4, 300, rng, groups=3)
    for pools in ([], [pool_of((1, 300, 8), 1)]):
        _, _, left = run_fork(table, lens, np.zeros(0, np.int32), ref, 4, np.zeros(0, int), pools)
        assert not left.any()


def test_cache_fork_more_and_fewer_rows():
    rng = np.random.default_rng(3)
    table, lens, ref = random_cache(5, 6, 4, 200, rng)
    pools = [pool_of((1, 200, 8), 1)]
    run_fork(table, lens, [0, 0, 0, 1, 2, 2, -1, 4, 4, 4, 4], ref, 4, np.zeros(11, int), pools)
    run_fork(table, lens, [3], ref, 4, [0], pools)
    run_fork(table, lens, [-1, -1], ref, 4, [24, 7], pools)


def test_cache_fork_starts_rows_on_an_empty_cache():
    ref = np.zeros(50, np.int32)
    table, lens = np.full((0, 8), -1, np.int32), np.zeros(0, np.int32)
    run_fork(table, lens, [-1, -1, -1], ref, 16, [100, 0, 33], [pool_of((1, 50, 8), 1)])


@pytest.mark.parametrize("P", [0, 1, 9, 12])
def test_cache_fork_when_the_pages_run_out(P):
    table, lens = np.full((2, 6), -1, np.int32), np.zeros(2, np.int32)
    run_fork(table, lens, [-1, -1, -1], np.zeros(P, np.int32), 4, [17, 9, 24], [])


def test_cache_fork_copy_without_a_page_left():
    table = np.array([[0, 1, -1], [-1, -1, -1]], np.int32)
    run_fork(table, np.array([6, 0], np.int32), [0, 0], np.array([1, 1], np.int32), 4, [0, 0], [pool_of((1, 2, 8), 2)])


def test_cache_fork_many_steps_keep_the_counts():
    """Beam steps one after the other, table by table: the counts stay those of the table's own entries."""
    rng = np.random.default_rng(11)
    R, M, ps, P = 24, 30, 5, 900
    table, lens, ref = random_cache(R, 8, ps, P, rng)
    table = np.concatenate([table, np.full((R, M - 8), -1, np.int32)], 1)
    lens_g = np.repeat(lens[::4], 4)
    for r in range(R):                                 # one length a group
        table[r] = -1
    perm, at = rng.permutation(P), 0
    for r in range(R):
        c = -(-int(lens_g[r]) // ps)
        table[r, :c] = perm[at:at + c]
        at += c
    lens = lens_g
    ref = np.bincount(table[table >= 0], minlength=P).astype(np.int32)
    pools = [pool_of((2, P, 8), 5)]
    for step in range(12):
        parent = (rng.integers(0, 4, R) + np.arange(R) // 4 * 4).astype(np.int32)
        table, lens, ref = run_fork(table, lens, parent, ref, ps, np.ones(R, int), pools, in_place=step % 2 == 0)
        assert np.array_equal(ref, np.bincount(table[table >= 0], minlength=P))


def test_cache_fork_reports_bad_tables():
    """Bad parents, lengths, growth and pages are reported, the rest of the call goes on, nothing is written out of
    bounds."""
    table = np.array([[0, 1, 2], [3, 99, -1], [4, -1, -1]], np.int32)
    lens, ref = np.array([9, 6, 3], np.int32), np.array([1] * 5 + [0] * 5, np.int32)
    call = lambda t, l, p, g: kda.kda_cache_fork(dev(t), dev(l), dev(p), dev(ref), 4, grow=dev(g))
    t2, l2, r2 = call(table, lens, [0, 7, -3], [0, 0, 0])
    assert kda.kda_get_device_error() == 0x80 | 0x20   # two bad parents, and the page 99 that is given up
    assert t2.tolist() == [[0, 1, 2], [-1] * 3, [-1] * 3] and l2.tolist() == [9, 0, 0]
    assert r2.tolist() == [1, 1, 1, 0, 0] + [0] * 5
    t2, l2, _ = call(table, lens, [0, 1, 2], [0, 0, 0])
    assert kda.kda_get_device_error() == 0x20
    assert t2.tolist() == [[0, 1, 2], [3, -1, -1], [4, -1, -1]]
    t2, l2, _ = call(np.where(table == 99, 5, table), np.array([13, 6, -1], np.int32), [0, 1, 2], [0, 0, 0])
    assert kda.kda_get_device_error() == 0x20 and l2.tolist() == [0, 6, 0]
    t2, l2, _ = call(np.where(table == 99, 5, table), lens, [0, 1, 2], [4, -1, 0])
    assert kda.kda_get_device_error() == 0x20 and l2.tolist() == [12, 6, 3]


# ---- compaction and copies ----
@pytest.mark.parametrize("P,live", [(1, 0), (1, 1), (7, 3), (100, 100), (1000, 1), (1000, 500), (5000, 4800), (40000, 9000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_cache_compact(P, live, in_place):
    rng = np.random.default_rng(P + live)
    ref = np.zeros(P, np.int32)
    pages = rng.permutation(P)[:live]
    ref[pages] = rng.integers(1, 9, live)
    table = rng.choice(np.concatenate([pages, [-1]]), (13, 11)).astype(np.int32)
    pools = [pool_of((2, P, 8), P), pool_of((1, P, 3, 8), live, torch.float32)]
    is_live = ref > 0
    movers = [p for p in range(P) if is_live[p] and p >= live]
    holes = [p for p in range(P) if not is_live[p] and p < live]
    where = np.where(is_live, np.arange(P), -1)
    where[movers] = holes
    want_ref = np.zeros(P, np.int32)
    want_ref[where[is_live]] = ref[is_live]
    want_table = np.where(table >= 0, where[np.maximum(table, 0)], -1)
    want = [p.clone() for p in pools]
    for s, d in zip(movers, holes):
        for w, p in zip(want, pools):
            w[:, d] = p[:, s]
    t, r = dev(table), dev(ref)
    t2, r2, m = kda.kda_cache_compact(t, r, pools=pools, block_table_out=None if in_place else torch.empty_like(t),
                                      ref_count_out=None if in_place else torch.empty_like(r))
    torch.cuda.synchronize()
    assert kda.kda_get_device_error() == 0
    assert (t2 is t) == in_place and (r2 is r) == in_place
    assert np.array_equal(m.cpu().numpy(), where) and np.array_equal(r2.cpu().numpy(), want_ref)
    assert np.array_equal(t2.cpu().numpy(), want_table)
    for w, p in zip(want, pools):
        assert torch.equal(w, p)
    other = pool_of((1, P, 40), 77)                    # another pool of the same pages follows with the map
    want_o = other.clone()
    for s, d in zip(movers, holes):
        want_o[:, d] = other[:, s]
    kda.kda_copy_pages((other,), None, m)
    assert torch.equal(other, want_o)


@pytest.mark.parametrize("slot", [(8,), (40,), (1000,), (8192,), (3, 100, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
def test_copy_pages(slot, dtype):
    n = int(np.prod(slot)) * torch.empty(0, dtype=dtype).element_size()
    S, L = 37, 3
    pool = torch.randint(0, 255, (L, S, n), dtype=torch.uint8, device=DEV).view(dtype).view(L, S, *slot)
    if n % 16:
        with pytest.raises(kda.KdaError):
            kda.kda_copy_pages((pool,), dev([0]), dev([1]))
        return
    order = np.random.default_rng(1).permutation(S)
    src, dst = order[:18].copy(), order[18:36].copy()
    src[3], dst[5], dst[7] = -1, -1, src[7]            # skipped
    want = pool.clone()
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            want[:, d] = pool[:, s]
    kda.kda_copy_pages((pool,), dev(src), dev(dst))
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8)) and kda.kda_get_device_error() == 0
    kda.kda_copy_pages((pool,), dev([0, S]), dev([S + 5, 1]))
    assert kda.kda_get_device_error() == 0x20
    assert torch.equal(pool.view(torch.uint8), want.view(torch.uint8))


def test_copy_pages_beyond_32_bits():
    pool = torch.zeros((1, 5, 3 << 28), dtype=torch.bfloat16, device=DEV)
    pool[0, 3, -7:] = 5.0
    pool[0, 3, :9] = 6.0
    kda.kda_copy_pages((pool,), dev([3]), dev([4]))
    assert bool((pool[0, 4, -7:] == 5).all()) and bool((pool[0, 4, :9] == 6).all()) and not pool[0, 4, 9:-7].any()
    assert not pool[0, 2].any()


def test_argument_checks():
    pool = pool_of((1, 4, 8), 1)
    idx, table, ref = dev([0, 1]), dev([[0, 1], [2, 3]]), dev([1] * 4)
    with pytest.raises(TypeError):
        kda.kda_state_fork(pool, idx.long(), idx)
    with pytest.raises(ValueError):
        kda.kda_state_fork(pool[0], idx, idx)          # not [layers, slots, ...]
    with pytest.raises(ValueError):
        kda.kda_state_fork(pool.cpu(), idx, idx)
    with pytest.raises(ValueError):
        kda.kda_state_fork(pool_of((1, 4, 8, 8), 1).transpose(2, 3), idx, idx)
    with pytest.raises(kda.KdaError):
        kda.kda_state_fork(pool, idx, dev([0, 0]), state_idx_out=idx)
    with pytest.raises(kda.KdaError):                  # 9 pools
        kda.kda_state_fork([pool] * 9, idx, idx)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_state_fork(pool, torch.zeros(8193, dtype=torch.int32, device=DEV),
                           torch.zeros(8193, dtype=torch.int32, device=DEV))
    assert e.value.code == 6
    with pytest.raises(kda.KdaError):                  # a pool of another number of pages
        kda.kda_cache_fork(table, dev([2, 2]), idx, dev([1] * 5), 1, pools=(pool,))
    with pytest.raises(kda.KdaError):
        kda.kda_cache_fork(table, dev([2, 2]), idx, ref, 0)
    with pytest.raises(kda.KdaError):
        kda.kda_cache_fork(table, dev([2, 2]), idx, ref, 1, block_table_out=table)
    with pytest.raises(kda.KdaError):
        kda.kda_cache_fork(table, dev([2, 2]), idx, ref, 1, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        kda.kda_cache_compact(table, ref, page_map=dev([0]))
    assert kda.kda_get_device_error() == 0
