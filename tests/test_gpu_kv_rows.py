"""Attention of 17 to 32 rows to a key head (the streaming kernel's tiles of
two groups of 16), of requests with fewer places than nodes, and the whole
error over long rows."""
import math

import numpy as np
import pytest

from tests import _kv_norm as N
from tests import test_gpu_kv as kv
from tests._gpu import say

pytestmark = pytest.mark.gpu

FORMS = [(64, "bf16", "bf16"), (64, "f16", "f16"), (64, "bf16", "e4m3"), (64, "f16", "e4m3"),
         (128, "bf16", "bf16"), (128, "f16", "f16"), (128, "bf16", "e4m3"), (128, "f16", "e4m3")]
# places, nodes, query heads to a key head: 17 to 32 rows on average
GROUPS = [([3000, 70, 4100], [8, 5, 6], 4, 16), ([0, 31, 33, 4000], [3, 4, 2, 5], 8, 24),
          ([500, 2, 3333], [9, 1, 11], 3, 7), ([6000], [32], 1, 64), ([900, 0], [17, 17], 1, 16)]


def rows_of(s):
    """Rows to a key head of an average request."""
    return -(-s["q"].shape[0] * (s["q"].shape[1] // s["H"]) // len(s["lens"]))


@pytest.mark.parametrize("D,dt,cache", FORMS)
@pytest.mark.parametrize("ctx,new,G,P", GROUPS)
@pytest.mark.parametrize("trees", [True, False])
def test_two_groups_of_rows(D, dt, cache, ctx, new, G, P, trees):
    say(f"two groups D={D} {dt} {cache} ctx={ctx} new={new} G={G} trees={trees}")
    s = kv.attn_case(ctx, new, 2, G, D, dt, cache, P, D + G, trees=trees,
                     order="slots first" if P == 7 else "heads first")
    assert 17 <= rows_of(s) <= 32
    got, _ = kv.check_attn(s)
    say(f"  {N.check(got, N.exact(s), s):.3f} half steps as a whole")


@pytest.mark.parametrize("D,dt,cache", FORMS)
def test_two_groups_of_rows_with_bad_pages(D, dt, cache):
    say(f"two groups, bad pages D={D} {dt} {cache}")
    s = kv.attn_case([700, 5, 3000], [8, 5, 6], 2, 4, D, dt, cache, 16, 2, bad_pages=40)
    assert 17 <= rows_of(s) <= 32
    kv.check_attn(s)
    s["table"][:] = -1
    got, lse = kv.check_attn(s)
    assert not got.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("D,dt,cache", FORMS)
@pytest.mark.parametrize("trees,ctx,new,G", [(True, [70, 0, 33], [8, 5, 6], 4), (True, [3001, 500], [7, 9], 3),
                                             (False, [20, 0], [20, 30], 1), (False, [2050, 16], [5, 3], 7)])
def test_two_groups_of_rows_not_finite_where_not_seen(D, dt, cache, trees, ctx, new, G):
    assert 17 <= -(-sum(new) * G // len(new)) <= 32
    kv.test_attention_not_finite_where_not_seen(D, dt, cache, trees, ctx, new, G)


@pytest.mark.parametrize("D,dt,cache", [(128, "bf16", "bf16"), (64, "f16", "f16"), (256, "bf16", "e4m3")])
@pytest.mark.parametrize("new,G", [([7, 5, 3], 2), ([8, 9, 6], 4), ([40, 60, 21], 3), ([20, 9, 30], 8)])
@pytest.mark.parametrize("trees", [True, False])
def test_fewer_places_than_nodes(D, dt, cache, new, G, trees):
    """Lengths below the number of nodes: the first nodes' places are not in
    the cache, and causal rows of those nodes see nothing."""
    say(f"fewer places than nodes D={D} {dt} {cache} new={new} G={G} trees={trees}")
    s = kv.attn_case([0, 3, 0], new, 2, G, D, dt, cache, 16, 5, trees=trees)
    s["lens"] = np.array([1, new[1] - 2, new[2] - 1])
    got, lse = kv.check_attn(s)
    if not trees:
        for r, places in enumerate(s["lens"]):
            unseen = slice(int(s["cu"][r]), int(s["cu"][r]) + new[r] - int(places))
            assert not got[unseen].any() and (lse[unseen] == -math.inf).all()


@pytest.mark.parametrize("ctx,new,H,G,D,dt,cache,P,trees", [
    # one request over every workgroup, one token and trees
    ([30000], [1], 1, 8, 128, "bf16", "bf16", 16, True), ([30000], [1], 1, 4, 64, "f16", "f16", 16, True),
    ([30000], [1], 1, 8, 128, "bf16", "e4m3", 64, True), ([30000], [2], 1, 8, 256, "bf16", "bf16", 16, True),
    ([30000], [3], 1, 8, 128, "f16", "f16", 16, True), ([30000], [4], 1, 8, 64, "bf16", "e4m3", 16, True),
    ([30000], [40], 1, 8, 128, "bf16", "bf16", 16, True), ([30000], [40], 1, 8, 64, "f16", "e4m3", 16, True),
    ([30000], [20], 1, 8, 256, "bf16", "bf16", 16, True), ([30000], [9], 1, 8, 128, "bf16", "e4m3", 64, True),
    # several, over the places where the list of rows is renewed
    ([2040, 4090, 6150], [33, 20, 64], 2, 8, 128, "bf16", "bf16", 24, True),
    ([2040, 4090, 6150], [33, 20, 64], 1, 4, 64, "bf16", "bf16", 16, True),
    ([1020, 2040, 3100], [33, 20, 64], 1, 4, 256, "f16", "f16", 16, True),
    # a prompt behind a long context
    ([5000], [300], 1, 2, 128, "bf16", "bf16", 16, False), ([7000], [400], 1, 1, 64, "f16", "f16", 32, False)])
def test_whole_error_over_long_rows(ctx, new, H, G, D, dt, cache, P, trees):
    say(f"whole error ctx={ctx} new={new} H={H} G={G} D={D} {dt} {cache}")
    s = kv.attn_case(ctx, new, H, G, D, dt, cache, P, D + sum(new), trees=trees)
    got, _ = kv.run_attn(s)
    say(f"  {N.check(got, N.exact(s), s):.3f} half steps")


@pytest.mark.parametrize("D,dt,cache", [(128, "bf16", "bf16"), (64, "f16", "e4m3")])
@pytest.mark.parametrize("ctx,new,first", [([40, 700, 5, 300, 90], [1, 1, 1, 1, 130], 4),
                                           ([0] * 30 + [500], [0] * 30 + [90], 30),
                                           ([9, 100, 2000], [2, 33, 60], 1)])
def test_one_batch_in_two_calls(D, dt, cache, ctx, new, first):
    """The first requests with their own tokens, then the others by the rest
    of the arrays: what one call gives, to the reference's bound."""
    import torch
    import mxfp4_packed_weight_amd as K
    from tests import _kv as R_
    say(f"two calls D={D} {dt} {cache} new={new}")
    s = kv.attn_case(ctx, new, 2, 8, D, dt, cache, 16, 11, trees=False)
    T, Hq, _ = s["q"].shape
    out, lse = torch.full_like(s["q"], 7.0), torch.full((T, Hq), 7.0, device="cuda")
    ws = torch.empty(K.k3_tree_attention_workspace_bytes(T, Hq, 2, D), dtype=torch.uint8, device="cuda")
    c, blocks = K.k3_kv_cache_of(s["kc"], s["vc"], s["ks"], s["vs"]), s["table"].shape[1]
    table, cu, lens = R_.i32(s["table"]), R_.i32(s["cu"]), R_.i32(s["lens"])
    K.k3_tree_attention(s["q"], int(s["cu"][first]), Hq, c, table, blocks, cu, lens, first, None, 1, s["scale"], out,
                        ws, lse=lse)
    K.k3_tree_attention(s["q"], T, Hq, c, table[first:], blocks, cu[first:], lens[first:], len(new) - first, None, 1,
                        s["scale"], out, ws, lse=lse)
    R_.check_attention(out, lse, kv.reference(s), dt, int(max(s["lens"])))
