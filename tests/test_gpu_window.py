"""k3_window_attention on the GPU against 64-bit floats (tests/_window.py)."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests import _window as W
from tests._gpu import say
from tests.test_gpu_kv import run_attn

pytestmark = pytest.mark.gpu

RAGGED = ([0, 1, 15, 63, 64, 200, 700, 1301], [1, 1, 1, 1, 1, 1, 1, 1])
CHUNKS = ([0, 1, 30, 127, 500, 3], [1, 2, 3, 33, 64, 17])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("lens,H,G,P,window,sinks", [
    (RAGGED, 2, 8, 16, 128, 4), (RAGGED, 3, 5, 7, 1, 0), (RAGGED, 1, 1, 24, 300, 65), (CHUNKS, 2, 4, 16, 40, 1),
    (CHUNKS, 1, 5, 24, 100, 0)])
def test_window(D, dt, cache, lens, H, G, P, window, sinks):
    say(f"window D={D} {dt} {cache} lens={lens} H={H} G={G} P={P} window={window} sinks={sinks}")
    order = "slots first" if P == 7 else "heads first"
    W.check(W.case(*lens, H, G, D, dt, cache, P, D + G, window, sinks, order=order))


@pytest.mark.parametrize("ctx,new,H,G,D,P,window,sinks", [
    ([20000], [1], 1, 8, 128, 16, 5000, 4), ([9000], [2], 1, 4, 64, 32, 8000, 300), ([4096], [1], 2, 1, 256, 64, 1000, 1),
    ([3001, 7, 12000], [1, 1, 1], 2, 2, 128, 24, 4000, 16), ([9000, 2], [24, 30], 1, 4, 128, 16, 3500, 100)])
def test_window_split(ctx, new, H, G, D, P, window, sinks):
    """Long windows, shared out to many workgroups and joined."""
    say(f"window split ctx={ctx} new={new} H={H} G={G} D={D} window={window} sinks={sinks}")
    W.check(W.case(ctx, new, H, G, D, "bf16", "bf16", P, D + G, window, sinks))


@pytest.mark.parametrize("ctx,new,H,G,D,dt,cache", [
    ([0], [500], 2, 1, 64, "f16", "f16"), ([770, 0], [330, 265], 1, 3, 128, "bf16", "bf16"),
    ([300, 5, 0], [1, 450, 20], 1, 2, 128, "bf16", "e4m3"), ([1000], [300], 1, 1, 256, "bf16", "bf16"),
    ([900], [600], 1, 8, 128, "bf16", "bf16")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (65, 64), (100, 5), (257, 130), (400, 1), (5000, 7)])
def test_window_of_prompts(ctx, new, H, G, D, dt, cache, window, sinks):
    """Tiles whose rows' windows begin at different places, in the sinks' blocks and behind them."""
    say(f"window of prompts ctx={ctx} new={new} H={H} G={G} D={D} window={window} sinks={sinks}")
    W.check(W.case(ctx, new, H, G, D, dt, cache, 16, D + G, window, sinks))


@pytest.mark.parametrize("ctx,new,H,G,D,dt,cache,window,sinks", [
    ([0, 1, 30, 127, 500], [1, 2, 3, 33, 64], 2, 4, 128, "bf16", "bf16", 64, 2),
    ([700, 300], [64, 50], 1, 8, 64, "f16", "f16", 100, 70), ([900, 10], [40, 64], 1, 4, 256, "bf16", "e4m3", 200, 0),
    ([1500, 200, 3], [64, 64, 64], 1, 8, 128, "bf16", "e4m3", 333, 17), ([90, 100], [2, 3], 2, 2, 64, "bf16", "bf16", 32, 1)])
def test_window_of_trees(ctx, new, H, G, D, dt, cache, window, sinks):
    """A node's position is its depth in the tree; its ancestors are all seen."""
    say(f"window of trees ctx={ctx} new={new} H={H} G={G} D={D} window={window} sinks={sinks}")
    W.check(W.case(ctx, new, H, G, D, dt, cache, 16, D + G, window, sinks, trees=True))


def test_rows_that_see_nothing():
    """Empty masks over nothing, requests not served, pages that do not exist."""
    say("window with empty rows")
    for D, G in ((64, 8), (128, 1), (256, 4), (128, 40)):
        s = W.case([0, 0, 40, 10, 0, 9], [3, 1, 2, 5, 0, 4], 2, G, D, "bf16", "bf16", 16, 1, 32, 3, trees=True)
        s["mask"][[0, 2, 3]] = 0
        s["mask"][4] = 0      # over a context: sees the window before the tree
        s["lens"][3] = 0      # not served
        s["lens"][5] = 10 ** 6  # past the table's row
        got, lse = W.check(s)
        empty = [0, 2, 3, 6, 7, 8, 9, 10, 11, 12, 13, 14]
        assert not got[empty].any() and (lse[empty] == -math.inf).all()
    for n in (1, 40):
        s = W.case([500], [n], 1, 8, 128, "bf16", "bf16", 16, 2, 100, 20)
        s["table"][0, 24:33] = -1
        W.check(s)
        s["table"][:] = s["pages"]
        got, lse = W.check(s)
        assert not got.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("trees,ctx,new,G,D", [(False, [70, 333, 90], [1, 1, 2], 4, 128), (True, [700, 50], [20, 3], 4, 64),
                                               (False, [1000], [300], 1, 128), (True, [500, 31], [64, 60], 8, 128)])
def test_a_wide_window_is_no_window(trees, ctx, new, G, D):
    """window = 0 is k3_tree_attention to the bit; one past every row's context has its values."""
    import torch
    say(f"wide window ctx={ctx} new={new}")
    s = W.case(ctx, new, 2, G, D, "bf16", "bf16", 16, 3, 0, 5, trees=trees)
    want, want_lse = run_attn(s)
    got, lse = W.run(s)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    for window, sinks in ((5000, 0), (1 << 30, 1 << 30), (64, 1 << 30)):
        W.check(s | {"window": window, "sinks": sinks})


@pytest.mark.parametrize("D,dt,cache", [(64, "f16", "f16"), (128, "bf16", "bf16"), (256, "bf16", "bf16"),
                                        (128, "bf16", "e4m3"), (64, "f16", "e4m3")])
@pytest.mark.parametrize("trees,ctx,new,G", [(False, [300, 64], [1, 1], 3), (False, [420, 0], [150, 70], 1),
                                             (True, [300, 131], [64, 60], 8), (True, [200, 5], [2, 1], 4)])
def test_not_finite_where_not_seen(D, dt, cache, trees, ctx, new, G):
    """NaN and infinities before the windows, behind the sinks: rows that do
    not see them stay as they were, to the bit. At a place that some rows see:
    those rows alone have NaN."""
    import torch
    say(f"window with NaN D={D} {dt} {cache} trees={trees} new={new}")
    P, H, window, sinks = 16, 2, 70, 9
    s = W.case(ctx, new, H, G, D, dt, cache, P, 3, window, sinks, trees=trees)
    want, want_lse = W.run(s)
    raw = torch.uint8 if cache == "e4m3" else torch.int16
    nan = {"e4m3": 0x7f, "bf16": 0x7fc0, "f16": 0x7e00}[cache]
    inf = {"e4m3": 0xff, "bf16": 0xff80 - 0x10000, "f16": 0xfc00 - 0x10000}[cache]
    hidden = 0
    for r, L in enumerate(s["lens"]):
        for p in (~W.sees(s, r).any(0)).nonzero()[:, 0].tolist():
            page, at = int(s["table"][r, p // P]), p % P
            s["kc"].view(raw)[page, at] = nan
            s["vc"].view(raw)[page, at] = inf if p % 2 else nan
            hidden += 1
    assert hidden > 100
    got, lse = W.run(s)
    assert torch.equal(got, want) and torch.equal(lse, want_lse), "places before the windows were used"
    vis = W.sees(s, 0)
    some = vis.any(0) & ~vis.all(0)
    if not some.any():  # (one row)
        return
    p = int(some.nonzero()[0])
    assert p < int(s["lens"][0]) - int(new[0]) or not trees
    page, at = int(s["table"][0, p // P]), p % P
    s["vc"].view(raw)[page, at, 1, 5] = nan
    got, lse = W.run(s)
    rest = [d for d in range(D) if d != 5]
    for t in range(s["q"].shape[0]):
        if t < int(new[0]) and vis[t, p]:
            assert got[t, G:, 5].isnan().all()
            assert torch.equal(got[t, G:][:, rest], want[t, G:][:, rest])
        else:
            assert torch.equal(got[t], want[t]) and torch.equal(lse[t], want_lse[t]), t


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("G,new", [(8, [1, 1]), (4, [40, 20]), (2, [150, 1])])
def test_sharp_and_rising_scores(dt, G, new):
    import torch
    say(f"window with rising scores {dt} G={G}")
    s = W.case([700, 300], new, 1, G, 64, dt, dt, 16, 6, 333, 3, q_std=0.0)
    s["q"][:] = 4.0
    s["kc"].zero_()
    for r, L in enumerate(s["lens"]):
        for p in range(int(L)):
            s["kc"][int(s["table"][r, p // 16]), p % 16, 0] = (p % 97) / 16.0 if r else p / 64.0
    s["clean"] = R_.wide(s["kc"]), R_.wide(s["vc"])
    for scale in (s["scale"], -s["scale"], 0.0):
        W.check(s | {"scale": scale})


def test_many_requests_of_unlike_lengths():
    """More requests than a workgroup has threads, short and long ones, with and without tokens."""
    say("window over many requests")
    rng = np.random.default_rng(7)
    for R, n in ((700, 1), (300, 3)):
        ctx = rng.integers(0, 200, R)
        ctx[::97] = 3000
        W.check(W.case(ctx, rng.integers(0, n + 1, R), 1, 2, 64, "bf16", "bf16", 16, 8, 90, 2))


def test_strides_streams_and_graphs():
    """Rows inside wider ones, a side stream, a replayed graph whose lengths move on: the eager call's bits."""
    import torch
    say("window in strides, on streams, in graphs")
    s = W.case([900, 3, 500], [3, 20, 1], 2, 4, 128, "bf16", "bf16", 16, 7, 200, 4)
    want, want_lse = W.run(s)
    T, Hq, D = s["q"].shape
    wide = torch.zeros((T, Hq * D + 40), dtype=s["q"].dtype, device="cuda")
    wide[:, :Hq * D] = s["q"].reshape(T, Hq * D)
    out = torch.full((T, Hq * D + 72), 5.0, dtype=s["q"].dtype, device="cuda")
    got, _ = W.run(s, q=wide.as_strided((T, Hq, D), (Hq * D + 40, D, 1)), lse=False,
                   out=out.as_strided((T, Hq, D), (Hq * D + 72, D, 1)))
    assert torch.equal(got, want) and (out[:, Hq * D:] == 5.0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, lse = W.run(s, stream=side)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    ws = torch.empty(K.k3_tree_attention_workspace_bytes(T, Hq, 2, D), dtype=torch.uint8, device="cuda")
    c = K.k3_kv_cache_of(s["kc"], s["vc"])
    lens, cu, table = R_.i32(s["lens"]), R_.i32(s["cu"]), R_.i32(s["table"])
    args = (s["q"], T, Hq, c, table, s["table"].shape[1], cu, lens, 3, None, 1)
    out, lse = torch.zeros_like(s["q"]), torch.zeros((T, Hq), device="cuda")
    graphs = []
    for window in (200, 64):  # two graphs share the workspace
        graphs.append((window, torch.cuda.CUDAGraph()))
        with torch.cuda.graph(graphs[-1][1]):
            K.k3_window_attention(*args, window, 4, s["scale"], out, ws, lse=lse)
    for cut in (0, 1, 7):
        s["lens"] = np.array([903 - 40 * cut, 23 - cut // 7, 501 - 60 * cut])
        lens.copy_(R_.i32(s["lens"]))
        for window, g in graphs:
            g.replay()
            torch.cuda.synchronize()
            eager = W.run(s | {"window": window})
            assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_request_left_out():
    """cu that is not ascending within [0, T]: those requests' rows stay as
    they were; the others' are within the bound (how the work is cut depends on
    the whole batch, so not to the bit)."""
    say("window with unsound cu")
    s = W.case([300, 200, 100], [4, 5, 3], 1, 4, 64, "bf16", "bf16", 16, 9, 64, 2)
    want = [x[:4] for x in W.reference(s)]
    s["cu"] = np.array([0, 4, 10 ** 9, 12])
    got, lse = W.run(s)
    R_.check_attention(got[:4], lse[:4], want, "bf16", 304)
    assert (got[4:] == 7).all() and (lse[4:] == 7).all()


def test_two_calls_at_once():
    """On two streams, each with a workspace and outputs of its own: each has its own bits."""
    import torch
    say("two window calls at once")
    cases = [W.case([3000, 40], [1, 30], 2, 4, 128, "bf16", "bf16", 16, 10, 900, 4),
             W.case([800, 500, 60], [200, 1, 1], 2, 2, 64, "f16", "e4m3", 16, 11, 100, 1)]
    want = [W.run(s) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.empty(K.k3_tree_attention_workspace_bytes(*s["q"].shape[:2], 2, s["q"].shape[2]), dtype=torch.uint8,
                          device="cuda") for s in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, stream, ws in zip(cases, streams, spaces):
            with torch.cuda.stream(stream):  # (inputs of the call are made on it as well)
                got.append(W.call(s, ws=ws))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1]), i
