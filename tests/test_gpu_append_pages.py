"""k3_kv_append with numbers out of the ordinary where a page and head take
several waves, or more rows than these keep in registers; and the largest
number of pages and heads (tests/_window.py has the sequential reference)."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests import _window as W
from tests._gpu import say
from tests.test_gpu_blocks import append_case, check_append

pytestmark = pytest.mark.gpu


# a wave keeps 2048 / D rows: pages of two waves, of four, and of more than they keep
PAGES = [(64, 48), (64, 64), (64, 100), (64, 1000), (128, 24), (128, 64), (128, 300), (256, 12), (256, 20), (256, 200)]


def odd_rows(s, at, dt):
    """Rows `at` get one number out of the ordinary each."""
    import torch
    odd = [math.nan, math.inf, -math.inf, 65504.0, -61440.0, 61441.0, 3e38 if dt == "bf16" else -65504.0]
    for n in ("k_in", "v_in"):
        s[n] = s[n].clone()
        for i, t in enumerate(at):
            s[n][t, (37 * i + 5) % s[n].shape[1]] = odd[(i + (n == "v_in")) % len(odd)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D,P", PAGES)
def test_numbers_out_of_the_ordinary(D, P, dt):
    """One in every page at first, in one wave's rows only; then in many rows; then nothing else."""
    import torch
    say(f"append of odd numbers D={D} P={P} {dt}")
    ctx, new = [0, P // 2 + 1, 3], [2 * P + 3, P, P - 3]
    for at in ([0], [P - 1], [P, 2 * P + 2, 2 * P + 3 + P // 2], list(range(0, 4 * P, 7))):
        s = append_case(ctx, new, 2, D, dt, P, D + P + at[-1])
        odd_rows(s, at, dt)
        check_append(s)
    for value in (math.inf, -math.inf, math.nan):
        s = append_case(ctx, new, 2, D, dt, P, D)
        s["k_in"] = torch.full_like(s["k_in"], value)
        check_append(s)


@pytest.mark.parametrize("D,P", PAGES)
def test_earlier_exponents_out_of_the_ordinary(D, P):
    """The earlier rows' bytes are 254, 255, 0, and far below the new rows'."""
    import torch
    say(f"append to pages with odd exponents D={D} P={P}")
    ctx, new = [P // 2, 1, P - 1, 3 * P + P // 2], [P, P - 1, 2, P // 4]
    s = append_case(ctx, new, 2, D, "bf16", P, D)
    for r, e in enumerate((254, 255, 0, 60)):
        page = s["table"][r, ctx[r] // P]
        s["k_exp"][page], s["v_exp"][page] = e, 254 - min(e, 254)
    s["k_in"] = s["k_in"].clone()
    s["k_in"][3, 7] = math.nan
    check_append(s)


def test_most_pages_and_heads():
    """A quarter of a million pages of 256 heads: more work than one dimension of a launch takes. All but a few
    pages are outside the cache, which has 8."""
    import torch
    say("append to 2^18 pages of 256 heads")
    T, H, D, P = 1 << 20, 256, 64, 4
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 40 GB")
    rows = torch.empty((T, H * D), dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros((8, P, H, D), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    exps = torch.full((2, 8, H), 77, dtype=torch.uint8, device="cuda")
    table = torch.full((1, T // P), -1, dtype=torch.int32, device="cuda")
    blocks = {0: 3, 1: 5, T // P // 2: 0, T // P - 2: 7, T // P - 1: 1}
    g = torch.Generator(device="cuda").manual_seed(1)
    for b, page in blocks.items():
        table[0, b] = page
        rows[b * P:b * P + P] = (torch.randn((P, H * D), generator=g, device="cuda") * 2.0 ** (page - 4)).bfloat16()
    K.k3_kv_append(rows, rows, T, K.k3_kv_cache_of(kc, vc), exps[0], exps[1], table, T // P, R_.i32([0, T]),
                   R_.i32([T]), 1)
    torch.cuda.synchronize()
    for b, page in blocks.items():
        x = rows[b * P:b * P + P].cpu().double().view(P, H, D)
        e = np.array([W.exponent(float(a)) for a in x.abs().amax((0, 2))])
        codes = W.e4m3(x * torch.from_numpy(2.0 ** (127.0 - e))[:, None])
        for i, c in enumerate((kc, vc)):
            assert np.array_equal(exps[i, page].cpu().numpy(), e), b
            assert torch.equal(R_.wide(c)[page], codes), b
    for page in set(range(8)) - set(blocks.values()):
        assert (exps[:, page] == 77).all() and not R_.wide(kc)[page].any()
    del rows
    torch.cuda.empty_cache()
