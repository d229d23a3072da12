"""Attention over the paged cache where it goes in tiles of many rows, in parts
of long ones, and over many requests; the workspace's bounds."""
import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests import test_gpu_kv as kv
from tests._gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx,new,H,G,D,dt,cache,P,trees", [
    # more blocks than are listed at a time, a full tile and one of 64 rows
    ([4500], [40], 1, 8, 128, "bf16", "bf16", 16, True),
    # one wave, two waves, three to 32 rows; e4m3
    ([2100, 0, 700, 65], [33, 1, 64, 9], 2, 4, 128, "bf16", "e4m3", 24, True),
    ([300, 4200], [5, 90], 1, 4, 64, "f16", "f16", 7, False),
    ([600, 64, 63], [100, 64, 65], 1, 4, 64, "bf16", "e4m3", 16, True),
    # causal tiles that begin and end inside blocks
    ([0], [700], 1, 1, 64, "f16", "f16", 16, False),
    ([100], [260], 1, 2, 128, "bf16", "bf16", 32, False),
    ([31, 0], [257, 255], 1, 3, 128, "f16", "e4m3", 16, False),
    # heads of 256: tiles of 128 rows
    ([2500, 60], [40, 30], 1, 8, 256, "bf16", "bf16", 16, True),
    ([1200], [150], 1, 2, 256, "f16", "e4m3", 16, False),
    ([33, 32, 31], [70, 33, 17], 2, 4, 256, "bf16", "e4m3", 24, True),
    # more query heads than a wave has rows
    ([50, 200], [10, 3], 1, 48, 64, "bf16", "bf16", 16, True)])
def test_tiles(ctx, new, H, G, D, dt, cache, P, trees):
    say(f"tiles ctx={ctx} new={new} H={H} G={G} D={D} {dt} {cache} P={P}")
    kv.check_attn(kv.attn_case(ctx, new, H, G, D, dt, cache, P, D + G, trees=trees))


@pytest.mark.parametrize("n,D,cache", [(40, 128, "bf16"), (40, 64, "e4m3"), (20, 256, "bf16"), (1, 128, "bf16")])
def test_one_long_row_in_many_parts(n, D, cache):
    """One request and one key head: its tiles are shared out to every workgroup."""
    say(f"many parts n={n} D={D} {cache}")
    kv.check_attn(kv.attn_case([30000], [n], 1, 8, D, "bf16", cache, 16, n + D))


@pytest.mark.parametrize("n,G", [(30, 8), (1, 4)])
@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (128, "e4m3"), (256, "bf16")])
def test_bad_pages_along_a_long_row(n, G, D, cache):
    """Pages that are not there in many blocks, also where the list of rows is renewed."""
    say(f"bad pages n={n} D={D} {cache}")
    s = kv.attn_case([5000, 300], [n, n], 1, G, D, "bf16", cache, 16, D, bad_pages=60)
    rng = np.random.default_rng(1)
    s["table"][0, rng.permutation(280)[:40]] = -1
    s["table"][0, 124:132] = s["pages"]  # from place 1984 to 2111: over the list's half
    kv.check_attn(s)


@pytest.mark.parametrize("R,every,n,G,H", [(1500, 3, 1, 2, 1), (4096, 40, 2, 1, 1), (520, 1, 5, 7, 1),
                                           (600, 40, 60, 8, 2)])
def test_many_requests(R, every, n, G, H):
    """More requests than a workgroup has threads, most of them without tokens."""
    say(f"many requests R={R} n={n} G={G}")
    rng = np.random.default_rng(R)
    new = np.where(np.arange(R) % every == every - 1, n, 0)
    ctx = rng.integers(0, 40, R)
    s = kv.attn_case(ctx, new, H, G, 64, "bf16", "bf16", 16, R, trees=False)
    kv.check_attn(s)


@pytest.mark.parametrize("ctx,new,H,G,D,cache", [
    ([700], [1], 2, 8, 128, "bf16"), ([700], [4], 2, 8, 128, "e4m3"), ([3000, 9], [40, 3], 2, 8, 128, "bf16"),
    ([3000, 20, 100, 9], [60, 4, 4, 4], 1, 8, 64, "bf16"), ([900], [60], 2, 8, 256, "bf16"),
    ([100] * 20, [1] * 20, 1, 3, 64, "bf16"),
    # as one request these rows would make a larger tile on fewer workgroups
    ([9000] * 2, [1] * 2, 2, 10, 128, "bf16"), ([9000] * 3, [1] * 3, 2, 8, 64, "bf16"),
    ([5000] * 2, [1] * 2, 2, 9, 256, "bf16"), ([9000] * 3, [2] * 3, 2, 8, 128, "e4m3")])
def test_workspace_is_as_large_as_said(ctx, new, H, G, D, cache):
    """Nothing past it is written, and what it held before does not matter."""
    import torch
    say(f"workspace ctx={ctx} new={new} D={D}")
    s = kv.attn_case(ctx, new, H, G, D, "bf16", cache, 16, 3)
    need = K.k3_tree_attention_workspace_bytes(s["q"].shape[0], s["q"].shape[1], H, D)
    guard = 1 << 20
    out = []
    for fill in (0x00, 0x7f, 0xff):
        ws = torch.full((need + guard,), fill, dtype=torch.uint8, device="cuda")
        ws[need:] = 0xa5
        out.append(kv.run_attn(s, ws=ws[:need]))
        assert (ws[need:] == 0xa5).all()
    for got, lse in out[1:]:
        assert torch.equal(got, out[0][0]) and torch.equal(lse, out[0][1])
    R_.check_attention(out[0][0], out[0][1], kv.reference(s), "bf16", int(max(s["lens"])))


@pytest.mark.parametrize("D,G,n", [(128, 8, 20), (64, 4, 60), (256, 4, 20), (128, 8, 2)])
def test_rows_without_a_number_keep_to_themselves(D, G, n):
    """NaN and infinities in one node's queries leave the other rows as they were."""
    import torch
    say(f"NaN queries D={D} n={n}")
    s = kv.attn_case([300, 20], [n, n], 1, G, D, "bf16", "bf16", 16, 4)
    want, lse = kv.run_attn(s)
    s["q"][1, 0, 5] = float("nan")
    s["q"][n, G - 1, 0] = float("inf")
    got, l2 = kv.run_attn(s)
    same = torch.ones(want.shape[:2], dtype=torch.bool, device="cuda")
    same[1, 0] = same[n, G - 1] = False
    assert torch.equal(got[same], want[same]) and torch.equal(l2[same], lse[same])
    assert got[1, 0].isnan().all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(20, 8), (1, 8), (9, 3)])
def test_key_scales_of_any_sign(D, n, G):
    """A head's scale may be 0 (all its scores are) or negative, and so may the call's."""
    import torch
    say(f"key scales D={D} n={n} G={G}")
    s = kv.attn_case([130, 3], [n, n], 3, G, D, "bf16", "e4m3", 16, 5)
    s["ks"].copy_(torch.tensor([0.0, -0.02, 0.02], device="cuda"))
    kv.check_attn(s)
    s["scale"] = -s["scale"]
    kv.check_attn(s)


@pytest.mark.parametrize("D,cache", [(128, "bf16"), (64, "e4m3"), (256, "bf16")])
def test_graph_of_tiles(D, cache):
    """Captured once, replayed with other lengths and rows between eager calls: the same bits."""
    import torch
    say(f"graph of tiles D={D} {cache}")
    T, H, G, n = 60, 2, 8, 20
    cases = [kv.attn_case(ctx, [n] * 3, H, G, D, "bf16", cache, 16, i) for i, ctx in
             enumerate(([900, 5, 300], [64, 640, 0], [1000, 1000, 1]))]
    pages, blocks = max(c["pages"] for c in cases), max(c["table"].shape[1] for c in cases)
    like = lambda x: torch.zeros((pages, H, 16, D), device="cuda").to(x.dtype).permute(0, 2, 1, 3)  # noqa: E731
    kc, vc = like(cases[0]["kc"]), like(cases[0]["vc"])
    scales = [None if cases[0][x] is None else cases[0][x].clone() for x in ("ks", "vs")]
    q, out = (torch.zeros((T, H * G, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.zeros((T, H * G), device="cuda")
    table, cu, lens = R_.i32(np.zeros((3, blocks))), R_.i32(np.arange(4) * n), R_.i32([0] * 3)
    mask = R_.i32(np.zeros((T, 1)))
    ws = torch.empty(K.k3_tree_attention_workspace_bytes(T, H * G, H, D), dtype=torch.uint8, device="cuda")
    handle = K.k3_kv_cache_of(kc, vc, *scales)

    def call():
        K.k3_tree_attention(q, T, H * G, handle, table, blocks, cu, lens, 3, mask, 1, D ** -0.5, out, ws, lse=lse)

    def load(c):
        raw = torch.uint8 if cache == "e4m3" else torch.int16
        for to, x in ((kc, c["kc"]), (vc, c["vc"])):
            to.view(raw)[:c["pages"]] = x.view(raw)
        for to, x in zip(scales, (c["ks"], c["vs"])):
            if to is not None:
                to.copy_(x)
        q.copy_(c["q"])
        t = np.full((3, blocks), -1)
        t[:, :c["table"].shape[1]] = c["table"]
        table.copy_(R_.i32(t))
        lens.copy_(R_.i32(c["lens"]))
        mask.copy_(R_.i32(c["mask"]))
        out.zero_()
        torch.cuda.synchronize()

    load(cases[0])
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for i in (1, 2, 0, 1):
        load(cases[i])
        call()
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        load(cases[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        R_.check_attention(out, lse, kv.reference(cases[i]), "bf16", int(max(cases[i]["lens"])))
