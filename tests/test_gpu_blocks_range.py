"""k3_block_attention over values at the ends of the rows' type: exponents far
from page to page, products of code and power that no 16-bit number holds,
NaN outside the windows, and what k3_kv_append makes of the largest rows."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests import _window as W
from tests._gpu import say
from tests.test_gpu_blocks import append, append_case

pytestmark = pytest.mark.gpu

# rows to a key head: one and two tiles of the streaming kernel, the tiled kernel with and without paired waves
SIZES = [([300, 64], [1, 1], 3), ([300, 90], [4, 2], 4), ([301, 9], [8, 7], 4), ([420, 0], [150, 70], 1),
         ([500, 31], [64, 60], 8)]


def set_page(s, name, r, p, byte):
    """The page of request r's place p, with codes of 0 and an exponent."""
    import torch
    page = int(s["table"][r, p // s["P"]])
    s[name + "c"].view(torch.uint8)[page] = 0
    s[name + "_exp"][page] = byte
    return page


def cleaned(s):
    """What the codes and exponents stand for, in 64 bits."""
    import torch
    s["clean"] = tuple(R_.wide(s[n + "c"]) * torch.exp2(s[n + "_exp"].cpu().double() - 127)[:, None, :, None]
                       for n in "kv")


PAST = pytest.mark.parametrize("dt,byte,code", [("f16", 135, 0x78), ("f16", 140, 0x7e), ("f16", 254, 0x81),
                                                ("bf16", 247, 0x78), ("bf16", 254, 0xf0), ("bf16", 250, 0x7f)])


def places(ctx, new):
    """A new one, one at the windows' edge, one before them."""
    return ctx[0] + new[0] // 2, ctx[0] - 60, 200


@pytest.mark.parametrize("D", [64, 128, 256])
@PAST
@pytest.mark.parametrize("ctx,new,G", SIZES)
def test_values_past_the_type(D, dt, byte, code, ctx, new, G):
    """A value whose code times its power is infinite in the rows' type (or NaN): the rows that see it have no
    finite number there, the others, and all other numbers, stay as they were, to the bit."""
    import torch
    say(f"block attention with a value past {dt} byte={byte} code={code:#x} D={D} new={new} G={G}")
    P = 16
    for p in places(ctx, new):
        s = W.case(ctx, new, 2, G, D, dt, "blocks", P, 3, 70, 9)
        page = set_page(s, "v", 0, p, byte)
        want, want_lse = W.run(s)
        s["vc"].view(torch.uint8)[page, p % P, 1, 5] = code
        got, lse = W.run(s)
        assert want.isfinite().all() and torch.equal(lse, want_lse)
        vis = W.sees(s, 0)
        rest = [d for d in range(D) if d != 5]
        for t in range(s["q"].shape[0]):
            if t < new[0] and vis[t, p]:
                assert torch.equal(got[t, :G], want[t, :G])
                assert not got[t, G:, 5].isfinite().any(), (p, t, got[t, G:, 5])
                assert torch.equal(got[t, G:][:, rest], want[t, G:][:, rest]), (p, t)
            else:
                assert torch.equal(got[t], want[t]), (p, t)


@pytest.mark.parametrize("D", [64, 128, 256])
@PAST
@pytest.mark.parametrize("ctx,new,G", SIZES)
def test_keys_past_the_type(D, dt, byte, code, ctx, new, G):
    """The same for a key: rows that do not see it are within the bound. (Not to the bit: a wave raises its rows'
    references together, and the weights are rounded relative to them.)"""
    import torch
    say(f"block attention with a key past {dt} byte={byte} code={code:#x} D={D} new={new} G={G}")
    P = 16
    for p in places(ctx, new):
        s = W.case(ctx, new, 2, G, D, dt, "blocks", P, 3, 70, 9)
        page = set_page(s, "k", 0, p, byte)
        s["kc"].view(torch.uint8)[page, p % P, 1, 5] = code
        cleaned(s)
        got, lse = W.run(s)
        vis = W.sees(s, 0)
        rows = torch.tensor([t >= new[0] or not vis[t, p] for t in range(s["q"].shape[0])])
        assert rows.any()
        R_.check_attention(got.cpu()[rows], lse.cpu()[rows], [x[rows] for x in W.reference(s)], dt, int(max(s["lens"])))


@pytest.mark.parametrize("dt,byte", [("f16", 135), ("bf16", 247)])
@pytest.mark.parametrize("ctx,new,G", SIZES)
def test_the_largest_values_that_fit(dt, byte, ctx, new, G):
    """240 times 2^8 (2^120) is a number of the type, 256 times it is not."""
    import torch
    say(f"block attention with the largest values of {dt} new={new} G={G}")
    s = W.case(ctx, new, 1, G, 64, dt, "blocks", 16, 4, 0, 0)
    p = ctx[0] + new[0] - 1
    page = set_page(s, "v", 0, p, byte)
    s["vc"].view(torch.uint8)[page, p % 16, 0, ::2] = 0x77
    s["q"].zero_()  # (even weights: sums stay in range)
    got, _ = W.run(s)
    assert got.isfinite().all()
    t, L = new[0] - 1, int(s["lens"][0])
    want = 240 * 2.0 ** (byte - 127) / L
    v = got[t, :, ::2].double()
    # (beside it the other values, a few at most; two roundings to the type, and a sum of L numbers)
    off = (2 * R_.HALF_STEP[dt] + L * 2.0 ** -23) * want + 16
    assert ((v - want).abs() <= off).all(), ((v - want).abs().max(), off)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,G", SIZES)
def test_not_finite_outside_the_windows(D, ctx, new, G):
    """NaN in keys and values before the windows, behind the sinks, changes nothing."""
    import torch
    say(f"block attention with NaN outside the windows D={D} new={new} G={G}")
    for dt in ("bf16", "f16"):
        s = W.case(ctx, new, 2, G, D, dt, "blocks", 16, 3, 70, 9)
        want, want_lse = W.run(s)
        hidden = 0
        for r, L in enumerate(s["lens"]):
            for p in (~W.sees(s, r).any(0)).nonzero()[:, 0].tolist():
                page, at = int(s["table"][r, p // 16]), p % 16
                s["kc"].view(torch.uint8)[page, at] = 0x7f
                s["vc"].view(torch.uint8)[page, at] = 0xff if p % 2 else 0x7f
                hidden += 1
        assert hidden > 100
        got, lse = W.run(s)
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


def spread_exponents(s, low, high, seed):
    """Exponents of keys and values anywhere in [low, high]; the codes stand for themselves times their powers."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    for n in "kv":
        s[n + "_exp"] = torch.randint(low, high + 1, s[n + "_exp"].shape, generator=g, device="cuda").to(torch.uint8)
    cleaned(s)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,low,high", [("bf16", 11, 25), ("bf16", 120, 134), ("bf16", 190, 204), ("f16", 122, 134),
                                         ("f16", 104, 112), ("f16", 95, 103), ("f16", 104, 134)])
@pytest.mark.parametrize("ctx,new,G", SIZES)
def test_keys_and_values_of_unlike_sizes(D, dt, low, high, ctx, new, G):
    """Powers far apart from page to page, to both ends of fp16."""
    import torch
    say(f"block attention of exponents {low} to {high} {dt} D={D} new={new} G={G}")
    s = W.case(ctx, new, 2, G, D, dt, "blocks", 16, low, 0, 0)
    g = torch.Generator(device="cuda").manual_seed(high)
    for n in "kv":  # (codes of 11 bits' range and more: from subnormal ones up to 448)
        c = s[n + "c"]
        size = torch.exp2(2 * torch.randn(c.shape[:2], generator=g, device="cuda"))
        c.copy_((c.float() * size[..., None, None]).clamp(-448, 448).to(c.dtype))
    spread_exponents(s, low, high, low)
    s["scale"] = float(np.float32(D ** -0.5 * 2.0 ** (127 - high) / 4))  # the largest scores are a few tens
    got, lse = W.run(s)
    out, want_lse, mean_abs, spread, most = W.reference(s)
    if dt == "f16":
        # a product of code and power is off by 2^-25 where it is subnormal: the score by that of the sum of |q|,
        # the output by that; the bound has 258 2^-24 of `spread` and one subnormal's step of 2^-24
        q = s["q"].cpu().double().abs().sum(-1) * abs(s["scale"]) * 2.0 ** -25
        spread = spread + q / (258 * 2.0 ** -24)
    # Weights are relative to a reference within 2^8 of the largest, which is 1 or more itself, and below 2^-126 they
    # are none: a value of which nothing but such weights is left is off by up to 2^-126 of the largest value for
    # each place. The bound has 2 (2^-8 or more) of mean_abs, 2^-11 in fp16: so much more of it.
    keys = int(max(s["lens"]))
    mean_abs = mean_abs + keys * 2.0 ** -126 * most[..., None] / (2 * R_.HALF_STEP[dt])
    worst = R_.check_attention(got, lse, (out, want_lse, mean_abs, spread, most), dt, keys)
    print(f"  worst at {worst:.3f} of the bound", flush=True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("G,new", [(8, [1, 1]), (4, [40, 20]), (1, [150, 1])])
def test_the_largest_rows_appended(dt, G, new):
    """Rows at the type's largest and infinite ones at some places: rows that do not see them are as without
    them; fp16's largest come back as 61440, bf16's as an infinity."""
    import torch
    say(f"append and block attention of {dt}'s largest G={G} new={new}")
    P, H, D = 16, 2, 64
    ctx = [60, 33]
    s = append_case([0, 0], [c + n for c, n in zip(ctx, new)], H, D, dt, P, 7)
    s["k_in"], s["v_in"] = s["k_in"].clone(), s["v_in"].clone()
    big = float(torch.finfo(R_.torch_type(dt)).max)
    at = ctx[0] + new[0] - 1  # the first request's last place
    s["v_in"][at, 3], s["v_in"][at, 4], s["v_in"][at, D + 5] = big, -big, math.inf
    append(s)
    T = sum(new)
    g = torch.Generator(device="cuda").manual_seed(8)
    a = s | {"q": (torch.randn((T, H * G, D), generator=g, device="cuda") * 0.1).to(R_.torch_type(dt)), "ks": None,
             "vs": None, "mask": None, "words": 1, "scale": D ** -0.5, "window": 0, "sinks": 0,
             "cu": np.concatenate([[0], np.cumsum(new)]), "lens": np.array(ctx) + np.array(new), "T": T}
    codes = R_.wide(s["vc"])
    page = int(s["table"][0, at // P])
    assert codes[page, at % P, 0, 3] == (256 if dt == "bf16" else 240)
    got, lse = W.run(a)
    last = new[0] - 1
    for d in (3, 4):
        v = got[last, :G, d]
        assert (v.isfinite() if dt == "f16" else ~v.isfinite()).all(), v
    # without the last place's numbers
    s["vc"].view(torch.uint8)[page, at % P, 0, 3:5] = 0
    s["vc"].view(torch.uint8)[page, at % P, 1, 5] = 0
    want, want_lse = W.run(a)
    for t in range(T):
        if t != last:
            assert torch.equal(got[t], want[t]), t
    assert torch.equal(lse, want_lse)
