"""Outputs and workspaces that a decoding operator allocates itself belong to the stream that it is given: a block of
another stream's may still be in use there, or be handed out again before the given one is done with it."""

import pytest
import torch

import kda_gated_delta_03_gb300 as kda
from kda_gated_delta_03_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(*shape):
    return torch.randn(shape, device=DEV)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def attention():
    kv, table, lens, q = rand(2, 8, 2, 16, 64), i32(*range(8)).view(2, 4), i32(50, 64), rand(2, 4, 64)
    return lambda s: kda.kda_attention_decode(q, kv[0], kv[1], table, lens, scale=0.2, stream=s)


def select():
    logits, scores = rand(6, 1000), rand(2, 3)
    return lambda s: kda.kda_beam_select(logits, scores, stream=s)


def state_fork():
    states, idx, parent = rand(1, 6, 2, 16, 16), i32(3, 1), i32(1, 0)
    return lambda s: kda.kda_state_fork(states, idx, parent, stream=s)


def cache_fork():
    table, lens, ref, parent = i32(*range(8)).view(2, 4), i32(48, 64), torch.ones(8, dtype=torch.int32, device=DEV), i32(1, 0)
    return lambda s: kda.kda_cache_fork(table, lens, parent, ref, 16, stream=s)


def cache_compact():
    table, ref = i32(7, 5, -1, 2).view(2, 2), i32(0, 0, 1, 0, 0, 1, 0, 1)
    table_out, ref_out = table.clone(), ref.clone()
    return lambda s: kda.kda_cache_compact(table, ref, block_table_out=table_out, ref_count_out=ref_out, stream=s)


@pytest.mark.parametrize("make,own,workspace", [(attention, [0], True), (select, [0, 1, 2], True), (state_fork, [0], False),
                                                (cache_fork, [0, 1], True), (cache_compact, [2], True)])
def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch, make, own, workspace):
    side, here, given = torch.cuda.Stream(), torch.cuda.current_stream(), []
    new_workspace = binding._new_workspace

    def watched(need, dev):
        given.append(torch.cuda.current_stream())
        return new_workspace(need, dev)

    monkeypatch.setattr(binding, "_new_workspace", watched)
    call = make()
    many = lambda x: x if isinstance(x, tuple) else (x,)
    results = many(call(None))
    want = [results[i].clone() for i in own]
    torch.cuda.synchronize()
    del results
    blocks = [torch.empty_like(w) for w in want for _ in range(8)]
    ours = {b.data_ptr() for b in blocks}
    del blocks                                         # free blocks of this stream's, of the right sizes
    given.clear()
    side.wait_stream(here)
    results = many(call(side))
    got = [results[i] for i in own]
    side.synchronize()
    assert given == ([side] if workspace else [])
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert not ours & {g.data_ptr() for g in got}
