"""The e4m3 cache with an exponent for each page and head on the GPU: the
append against sequential arithmetic, bit for bit, and the attention against
64-bit floats (tests/_window.py)."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests import _window as W
from tests._gpu import say

pytestmark = pytest.mark.gpu


# ---- append -----------------------------------------------------------------------

def append_case(ctx, new, H, D, dt, P, seed, std=1.0, order="heads first", gap=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx), np.asarray(new)
    lens = ctx + new
    T, need = int(new.sum()), -(-lens // P)
    pages = int(need.sum()) + 2
    ids, off = rng.permutation(pages), np.concatenate([[0], np.cumsum(need)])
    table = np.full((len(ctx), max(1, int(need.max()))), -1)
    for r in range(len(ctx)):
        table[r, :need[r]] = ids[off[r]:off[r + 1]]
    kc, vc = (R_.cache(pages, P, H, D, "e4m3", g, order, None, 60.0) for _ in range(2))
    size = torch.exp2(2 * torch.randn((T, 1), generator=g, device="cuda")) * std
    rows = (torch.randn((T, 2 * H * D + gap), generator=g, device="cuda") * size).to(R_.torch_type(dt))
    # earlier exponents about what the rows need: some rise, some do not
    exps = torch.randint(117, 124, (2, pages, H), generator=g, device="cuda").to(torch.uint8)
    return {"T": T, "H": H, "D": D, "P": P, "dt": dt, "pages": pages, "kc": kc, "vc": vc, "table": table,
            "cu": np.concatenate([[0], np.cumsum(new)]), "lens": lens, "k_exp": exps[0].contiguous(),
            "v_exp": exps[1].contiguous(), "k_in": rows[:, :H * D], "v_in": rows[:, H * D:2 * H * D]}


def append(s, stream=None):
    c = K.k3_kv_cache_of(s["kc"], s["vc"])
    K.k3_kv_append(s["k_in"], s["v_in"], s["T"], c, s["k_exp"], s["v_exp"], R_.i32(s["table"]), s["table"].shape[1],
                   R_.i32(s["cu"]), R_.i32(s["lens"]), len(s["lens"]), stream=stream)


def same(s, want):
    import torch
    torch.cuda.synchronize()
    for name in "kv":
        assert np.array_equal(s[name + "_exp"].cpu().numpy(), want[name + "_exp"]), name
        got = R_.wide(s[name + "c"])
        bad = ~((got == want[name]) | (got.isnan() & want[name].isnan()))
        assert not bad.any(), (name, bad.nonzero()[:5].tolist(), got[bad][:5], want[name][bad][:5])


def check_append(s):
    want = W.append(s)
    append(s)
    same(s, want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("ctx,new,H,D,P", [
    ([0], [1], 1, 64, 16), ([5, 16, 31, 0], [1, 1, 1, 1], 2, 128, 16), ([3, 100, 0, 64], [60, 1, 33, 0], 3, 64, 24),
    ([0, 7], [300, 129], 2, 128, 32), ([10, 2], [70, 140], 1, 256, 64), ([1, 2, 3, 4, 5], [3, 2, 9, 4, 1], 8, 128, 4),
    ([100, 0], [250, 1000], 1, 64, 1000)])
def test_append(ctx, new, H, D, P, dt):
    say(f"append ctx={ctx} new={new} H={H} D={D} P={P} {dt}")
    order = "slots first" if P == 24 else "heads first"
    check_append(append_case(ctx, new, H, D, dt, P, H + D, order=order, gap=16 if P == 16 else 0))


@pytest.mark.parametrize("std", [1e-30, 1e-4, 3e3, 1e30])
def test_sizes_of_values(std):
    say(f"append of values of {std}")
    check_append(append_case([3, 20], [30, 50], 2, 64, "bf16", 16, 1, std=std))


def test_many_requests():
    """A search over more requests than a wave has lanes, with and without tokens."""
    say("append of many requests")
    rng = np.random.default_rng(2)
    for R in (64, 65, 700, 4096):
        new = rng.integers(0, 4, R)
        new[R // 2] = 50
        check_append(append_case(rng.integers(0, 30, R), new, 1, 64, "bf16", 8, R))


def test_borders_of_the_exponent():
    """Largest values at, above and below 448 times a power of two; zeros; old exponents out of range."""
    import torch
    say("append at the exponents' borders")
    s = append_case([0, 0, 0, 4, 4, 4, 0], [1, 1, 1, 1, 1, 1, 2], 1, 64, "bf16", 4 * 4, 3)
    x = torch.zeros((8, 64), device="cuda")
    x[0, 3], x[1, 4], x[2, 5] = 448.0, -450.0, 7.0
    x[3, 1] = 3.5  # earlier rows with the exponents 0, 255 and 200
    x[4], x[5, 0] = 0, 1e-20
    x[7, 63] = 3.3895313892515355e38  # bf16's largest
    s["k_in"] = x.bfloat16()
    s["v_in"] = -x.bfloat16()
    for r, e in ((3, 0), (4, 255), (5, 200)):
        for n in "kv":
            s[n + "_exp"][s["table"][r, 0]] = e
    want = W.append(s)
    assert want["k_exp"][s["table"][0, 0], 0] == 127 and want["k_exp"][s["table"][1, 0], 0] == 128
    assert want["k_exp"][s["table"][2, 0], 0] == 121
    append(s)
    same(s, want)


def test_rows_of_no_numbers_and_fp16s_largest():
    import torch
    say("append of NaN, infinities, fp16's largest")
    for dt in ("bf16", "f16"):
        s = append_case([0, 5], [6, 3], 1, 64, dt, 16, 4)
        for n in ("k_in", "v_in"):
            s[n] = s[n].clone()
            s[n][1, 3], s[n][2, 4], s[n][4, 5], s[n][7, 6] = math.nan, math.inf, -math.inf, math.nan
        check_append(s)
        s["k_in"][0, 0], s["k_in"][8, 1] = 65504.0, -61000.0
        check_append(s)
        s["k_in"][:] = math.inf
        check_append(s)


def test_appended_twice():
    """A second call with the same rows changes nothing."""
    import torch
    say("append twice")
    s = append_case([3, 20, 0], [30, 1, 5], 2, 128, "bf16", 16, 5)
    append(s)
    once = [s[n].clone() for n in ("k_exp", "v_exp")] + [s[n].view(torch.uint8).clone() for n in ("kc", "vc")]
    append(s)
    torch.cuda.synchronize()
    twice = [s[n] for n in ("k_exp", "v_exp")] + [s[n].view(torch.uint8) for n in ("kc", "vc")]
    assert all(torch.equal(a, b) for a, b in zip(once, twice))


def test_unsound_requests_and_pages():
    """Requests whose lengths do not fit are left out; pages outside the cache are not written."""
    say("append with unsound requests")
    s = append_case([3, 20, 0, 40, 9], [30, 1, 5, 10, 2], 2, 64, "bf16", 16, 6)
    s["table"][0, 1], s["table"][3, 2] = -1, s["pages"]
    s["lens"][1] = 0        # below its tokens: not served
    s["lens"][4] = 10 ** 6  # past the table's row
    check_append(s)
    s = append_case([3, 20, 8], [30, 1, 5], 2, 64, "bf16", 16, 7)
    s["T"] = 33  # the last request's tokens are past T
    check_append(s)
    s["T"], s["lens"][:] = 36, -1
    check_append(s)


def test_a_stream_a_graph_and_no_tokens():
    import torch
    say("append on a stream and in a graph")
    s = append_case([3, 20], [30, 1], 2, 128, "bf16", 16, 8)
    want = W.append(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    append(s, stream=side)
    side.synchronize()
    same(s, want)
    c = K.k3_kv_cache_of(s["kc"], s["vc"])
    table, cu, lens = R_.i32(s["table"]), R_.i32(s["cu"]), R_.i32(s["lens"])
    k, v = s["k_in"].clone(), s["v_in"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.k3_kv_append(k, v, s["T"], c, s["k_exp"], s["v_exp"], table, s["table"].shape[1], cu, lens, 2)
    for i in range(3):
        k.copy_(torch.randn_like(k.float()) * 2.0 ** i)
        v.copy_(torch.randn_like(k.float()))
        s["k_in"], s["v_in"] = k, v
        want = W.append(s)
        g.replay()
        same(s, want)
    K.k3_kv_append(k, v, 0, c, s["k_exp"], s["v_exp"], table, s["table"].shape[1], cu, lens, 2)
    same(s, want)


# ---- attention --------------------------------------------------------------------

LENS = ([0, 1, 15, 63, 64, 200, 700, 1301], [1, 1, 1, 1, 1, 1, 1, 1])
CHUNKS = ([0, 1, 30, 127, 500, 3], [1, 2, 3, 33, 64, 17])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,H,G,P,window,sinks", [
    (LENS, 2, 8, 16, 0, 0), (LENS, 3, 5, 4, 100, 3), (CHUNKS, 2, 4, 16, 0, 0), (CHUNKS, 1, 5, 24, 40, 1)])
def test_attention(D, dt, lens, H, G, P, window, sinks):
    say(f"block attention D={D} {dt} lens={lens} H={H} G={G} P={P} window={window}")
    order = "slots first" if P == 24 else "heads first"
    W.check(W.case(*lens, H, G, D, dt, "blocks", P, D + G, window, sinks, order=order))


@pytest.mark.parametrize("ctx,new,H,G,D,P,window", [
    ([20000], [1], 1, 8, 128, 16, 0), ([9000], [2], 2, 4, 64, 32, 0), ([4096], [1], 2, 1, 256, 64, 0),
    ([3001, 7, 12000], [1, 1, 1], 2, 2, 128, 24, 0), ([2900, 2], [64, 300], 1, 8, 128, 16, 0),
    ([770, 0], [330, 265], 1, 3, 128, 16, 0), ([0], [500], 2, 1, 64, 16, 0), ([1000], [300], 1, 1, 256, 64, 200),
    ([1500], [400], 1, 4, 128, 12, 300)])
def test_attention_split_and_of_prompts(ctx, new, H, G, D, P, window):
    say(f"block attention ctx={ctx} new={new} H={H} G={G} D={D} window={window}")
    W.check(W.case(ctx, new, H, G, D, "bf16", "blocks", P, D + G, window, 4))


@pytest.mark.parametrize("low", [1, 60, 100, 150, 190])
def test_pages_of_unlike_sizes(low):
    """Exponents far apart from page to page, and far from 127."""
    import torch
    say(f"block attention with exponents around {low}")
    for new in (1, 90):
        s = W.case([300], [new], 2, 4, 128, "bf16", "blocks", 16, 3, 0, 0)
        g = torch.Generator(device="cuda").manual_seed(low)
        s["v_exp"] = torch.randint(low, low + 20, s["v_exp"].shape, generator=g, device="cuda").to(torch.uint8)
        s["clean"] = (s["clean"][0], R_.wide(s["vc"]) * torch.exp2(s["v_exp"].cpu().double() - 127)[:, None, :, None])
        W.check(s)


def test_bad_pages_and_not_finite_codes():
    import torch
    say("block attention with bad pages and NaN")
    for new in (1, 40):
        s = W.case([500, 60], [new, 1], 2, 8, 128, "bf16", "blocks", 16, 4, 0, 0, bad_pages=5)
        want, want_lse = W.check(s)
        used = np.zeros((s["pages"], 16), bool)
        for r, L in enumerate(s["lens"]):
            for p in range(int(L)):
                if 0 <= s["table"][r, p // 16] < s["pages"]:
                    used[s["table"][r, p // 16], p % 16] = True
        junk = torch.from_numpy(~used).cuda()
        for x in (s["kc"], s["vc"]):
            x.view(torch.uint8)[junk] = 0x7f
        for n in ("k_exp", "v_exp"):  # exponents of pages of nobody
            s[n][torch.from_numpy(~used.any(1)).cuda()] = 255
        got, lse = W.run(s)
        assert torch.equal(got, want) and torch.equal(lse, want_lse)
        s["table"][:] = -1
        got, lse = W.run(s)
        assert not got.any() and (lse == -math.inf).all()


def test_a_step_appends_and_attends():
    """A prompt in two chunks and single tokens, appended and attended to as a
    server does: what the rows of the cache stand for decides."""
    import torch
    say("append and block attention, step by step")
    P, H, G, D, R = 16, 2, 4, 128, 3
    g = torch.Generator(device="cuda").manual_seed(9)
    blocks, pages = 20, 60
    table = np.random.default_rng(9).permutation(pages).reshape(R, blocks)
    s = append_case([1], [1], H, D, "bf16", P, 9)
    kc, vc = (R_.cache(pages, P, H, D, "e4m3", g) for _ in range(2))
    exps = torch.full((2, pages, H), 255, dtype=torch.uint8, device="cuda")
    s |= {"kc": kc, "vc": vc, "k_exp": exps[0], "v_exp": exps[1], "pages": pages, "table": table}
    ctx = np.zeros(R, int)
    for new in ([70, 5, 33], [50, 1, 0], [1, 1, 1], [1, 1, 1], [2, 0, 9]):
        new = np.array(new)
        T = int(new.sum())
        rows = (torch.randn((T, 2 * H * D), generator=g, device="cuda") *
                torch.exp2(torch.randn((T, 1), generator=g, device="cuda"))).bfloat16()
        s |= {"T": T, "cu": np.concatenate([[0], np.cumsum(new)]), "lens": ctx + new, "k_in": rows[:, :H * D],
              "v_in": rows[:, H * D:]}
        want = W.append(s)
        append(s)
        same(s, want)
        a = s | {"q": (torch.randn((T, H * G, D), generator=g, device="cuda") * 1.5).bfloat16(), "ks": None, "vs": None,
                 "mask": None, "words": 1, "scale": D ** -0.5, "window": 0, "sinks": 0,
                 "clean": tuple(want[n] * torch.exp2(torch.from_numpy(want[n + "_exp"]).double() - 127)[:, None, :, None]
                                for n in "kv")}
        a["clean"] = tuple(torch.nan_to_num(c, nan=0.0, posinf=0.0, neginf=0.0) for c in a["clean"])  # pages of nobody
        W.check(a)
        ctx = ctx + new
