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
