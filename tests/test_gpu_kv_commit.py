"""The commit's places: accepted nodes that have no page of their request move
nothing, neither rows nor the request's length."""
import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests._gpu import say

pytestmark = pytest.mark.gpu


def caches(pages, P=16, H=2, D=64):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(pages)
    return tuple(R_.cache(pages, P, H, D, "bf16", g) for _ in range(2))


@pytest.mark.parametrize("ctx,accepted", [
    (64, [0]),              # the first place past the table's row
    (63, [0, 1]),           # one in it, one past it
    (62, [0, 1, 2]),
    (2 ** 31 - 1, [0]),     # the sum would pass 32 bits
    (2 ** 31 - 4, [0, 1, 2]),
    (16, [0]),              # no page: -1
    (15, [0, 1]),
    (32, [0, 1]),           # no page: past the cache
    (14, [0, 1, 2])])
def test_paths_that_lie_in_place_need_pages_too(ctx, accepted):
    """Nothing moves in such a path, but its tokens are nowhere."""
    import torch
    say(f"commit in place ctx={ctx} accepted={accepted}")
    kc, vc = caches(4)
    before = kc.clone(), vc.clone()
    table = [[0, -1, 4, 1], [3, 2, 0, 1]]
    n = len(accepted)
    out = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    # the other request: three tokens in place
    K.k3_kv_commit(K.k3_kv_cache_of(kc, vc), 1, 0, R_.i32(table), 4, R_.i32([ctx, 20]),
                   R_.i32([accepted + [9] * (3 - n), [0, 1, 2]]), R_.i32([n, 3]), 3, 2, out)
    assert out.tolist() == [ctx, 23]
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


def test_paths_in_place_within_their_pages():
    """Up to the last place of the table's row."""
    import torch
    say("commit in place, within pages")
    kc, vc = caches(4)
    before = kc.clone()
    out = torch.full((3,), -5, dtype=torch.int32, device="cuda")
    K.k3_kv_commit(K.k3_kv_cache_of(kc, vc), 1, 0, R_.i32(np.tile([3, 1, 0, 2], (3, 1))), 4, R_.i32([61, 15, 7]),
                   R_.i32(np.tile(np.arange(3), (3, 1))), R_.i32([3, 2, 0]), 3, 3, out)
    assert out.tolist() == [64, 17, 7] and torch.equal(kc, before)


def plan(ctx, new, held, ring, state, table, n_pages, P=16):
    """The plan of a step without trees: held, ring's state, kv_lens, status."""
    zeros = lambda n: R_.i32(np.zeros(n))  # noqa: E731
    R, T, blocks = len(ctx), int(sum(new)), table.shape[1]
    o = [zeros(n) for n in (R, 2, R + 1, R, max(T, 1), max(T, 1), 2)]
    K.k3_kv_plan(R_.i32(ctx), R_.i32(new), None, R, T, n_pages, P, blocks, held, ring, state, table, *o[:6], None, 0,
                 o[6])
    return o[0], o[1], o[3], o[6]


@pytest.mark.parametrize("accepted,count", [([17, 19], 1), ([0, 17], 2), ([0, 1], 2), ([16, 18], 2)])
def test_a_request_not_served_leaves_the_others_rows_alone(accepted, count):
    """A request gives pages back, another takes them, and a step later the
    first is not served: the ids of its old pages are still in the table."""
    import torch
    say(f"commit after pages went to another request, accepted={accepted}")
    kc, vc = caches(4)
    table, ring = R_.i32([[0, 1, 2, -1], [-1] * 4]), R_.i32([3, -1, -1, -1])
    held, state, _, _ = plan([16, 0], [0, 0], R_.i32([3, 0]), ring, R_.i32([0, 1]), table, 4)
    assert held.tolist() == [1, 0]
    held, state, _, _ = plan([16, 0], [0, 40], held, ring, state, table, 4)
    assert held.tolist() == [1, 3] and table.tolist() == [[0, 1, 2, -1], [3, 1, 2, -1]]
    held, state, lens, status = plan([16, 40], [20, 3], held, ring, state, table, 4)
    assert status.tolist() == [1, 0] and lens.tolist() == [0, 43]
    before = kc.clone(), vc.clone()
    out = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    K.k3_kv_commit_ex(K.k3_kv_cache_of(kc, vc), 1, 0, table, 4, R_.i32([16, 40]), lens, R_.i32([accepted, [0, 2]]),
                      R_.i32([count, 2]), 2, 2, out)
    assert out.tolist() == [16, 42]
    for x, b in zip((kc, vc), before):
        b[2, 9] = b[2, 10]  # the other request's place 42 to 41
        assert torch.equal(x, b)


@pytest.mark.parametrize("lens,want", [
    ([40, 24, 0, 22], [13, 22, 30, 20]),
    ([14, 23, 31, 21], [10, 20, 31, 20]),
    ([15, 2 ** 31 - 1, -1, 2], [13, 22, 30, 20])])
def test_accepted_nodes_are_of_the_step(lens, want):
    """Places at or past kv_lens are not the step's."""
    import torch
    say(f"commit with kv_lens={lens}")
    kc, vc = caches(12)
    ctx, accepted, count = [10, 20, 30, 20], [[0, 2, 4], [1, 3, 9], [0, 1, 2], [2, 3, 4]], [3, 2, 1, 0]
    table = np.random.default_rng(1).permutation(12).reshape(4, 3)
    before, out = kc.clone(), torch.full((4,), -5, dtype=torch.int32, device="cuda")
    K.k3_kv_commit_ex(K.k3_kv_cache_of(kc, vc), 1, 0, R_.i32(table), 3, R_.i32(ctx), R_.i32(lens), R_.i32(accepted),
                      R_.i32(count), 3, 4, out)
    assert out.tolist() == want
    for r in range(4):
        moves = range(count[r]) if want[r] > ctx[r] else ()
        rows = [before[table[r][(ctx[r] + accepted[r][i]) // 16], (ctx[r] + accepted[r][i]) % 16].clone() for i in moves]
        for i, row in zip(moves, rows):
            before[table[r][(ctx[r] + i) // 16], (ctx[r] + i) % 16] = row
    assert torch.equal(kc, before)


def test_graph_of_a_commit():
    """Captured once, replayed with lengths that serve other requests, between eager calls."""
    import torch
    say("graph of a commit with kv_lens")
    kc, vc = caches(12)
    base = kc.clone(), vc.clone()
    table = R_.i32(np.arange(12).reshape(4, 3))
    st = [R_.i32(x) for x in ([10, 20, 30, 5], [0] * 4, np.tile([1, 3], (4, 1)), [2, 1, 2, 2], [0] * 4)]
    handle = K.k3_kv_cache_of(kc, vc)

    def call():
        K.k3_kv_commit_ex(handle, 1, 0, table, 3, st[0], st[1], st[2], st[3], 2, 4, st[4])

    def load(lens):
        st[1].copy_(R_.i32(lens))
        kc.copy_(base[0])
        vc.copy_(base[1])
        torch.cuda.synchronize()

    load([14, 24, 34, 9])
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lens, ctx in (([14, 0, 34, 0], [12, 20, 32, 5]), ([0, 22, 0, 9], [10, 21, 30, 7]), ([0] * 4, [10, 20, 30, 5]),
                      ([14, 24, 34, 9], [12, 21, 32, 7])):
        load(lens)
        call()
        torch.cuda.synchronize()
        want = kc.clone(), vc.clone(), st[4].tolist()
        load(lens)
        st[4].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and st[4].tolist() == want[2] == ctx
