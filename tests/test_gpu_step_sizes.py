"""The largest sizes of the step's calls, and caches whose bytes pass 32 bits."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests import _step as S
from tests import _window as W
from tests._gpu import say
from tests.test_gpu_blocks import append_case
from tests.test_gpu_blocks import append as append_rows
from tests.test_gpu_logprobs import call as logprobs_call
from tests.test_gpu_logprobs import check as check_logprobs
from tests.test_gpu_logprobs import logits

pytestmark = pytest.mark.gpu


def far(x, pages, at):
    """The cache's pages at the end of a larger one, past its first 4 GiB."""
    import torch
    y = torch.empty((pages, *x.permute(0, 2, 1, 3).shape[1:]), dtype=x.dtype, device="cuda").permute(0, 2, 1, 3)
    y[at:at + x.shape[0]] = x
    return y


@pytest.mark.parametrize("cache,new", [("bf16", 1), ("bf16", 40), ("e4m3", 1), ("blocks", 1), ("blocks", 40)])
def test_far_pages(cache, new):
    """Windowed attention and the one over exponents: the bits of the same pages in a small cache."""
    import torch
    say(f"far pages {cache} new={new}")
    H, P, D = 8, 64, 128
    s = W.case([900, 300], [new, 1], H, 8, D, "bf16", cache, P, 3, 500, 4)
    want, want_lse = W.run(s)
    n = s["pages"]
    pages = (5 << 30) // (P * H * D * (2 if cache == "bf16" else 1))
    at = pages - n
    t = dict(s)
    for name in ("kc", "vc"):
        t[name] = far(s[name], pages, at)
    if cache == "blocks":
        for name in ("k_exp", "v_exp"):
            e = torch.full((pages, H), 1, dtype=torch.uint8, device="cuda")
            e[at:] = s[name]
            t[name] = e
    t["table"] = np.where(s["table"] >= 0, s["table"] + at, -1)
    t["pages"] = pages
    got, lse = W.run(t)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


def test_far_pages_appended():
    import torch
    say("append to far pages")
    H, P, D = 8, 64, 128
    s = append_case([100, 7], [80, 200], H, D, "bf16", P, 5)
    want = W.append(s)
    n, pages = s["pages"], (5 << 30) // (P * H * D)
    at = pages - n
    t = dict(s)
    for name in ("kc", "vc"):
        t[name] = far(s[name], pages, at)
    for name in ("k_exp", "v_exp"):
        e = torch.full((pages, H), 9, dtype=torch.uint8, device="cuda")
        e[at:] = s[name]
        t[name] = e
    t["table"] = np.where(s["table"] >= 0, s["table"] + at, -1)
    t["pages"] = pages
    append_rows(t)
    torch.cuda.synchronize()
    for name in "kv":
        assert np.array_equal(t[name + "_exp"][at:].cpu().numpy(), want[name + "_exp"])
        assert (t[name + "_exp"][:at] == 9).all()
        assert torch.equal(R_.wide(t[name + "c"][at:]), want[name])


def test_the_largest_vocabulary():
    """2^24 logits, 64 alternatives: the most parts, and a token in the last of them."""
    say("logprobs of 2^24 logits")
    V = 1 << 24
    x = logits(2, V, "bf16", 3)
    x[0, V - 1] = 30.0
    x[1, V // 2:] = -math.inf
    check_logprobs(x, 1.0, [V - 1, V // 2 - 1], 64)


def test_the_most_rows():
    """2^20 rows, of few logits and of few values."""
    import torch
    say("2^20 rows")
    T = 1 << 20
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, 5), generator=g, device="cuda")
    tokens = torch.randint(0, 5, (T,), generator=g, device="cuda").int()
    o = logprobs_call(x, 1.0, tokens, 2)
    y, w = torch.empty((T, 8), dtype=torch.bfloat16, device="cuda"), torch.ones(8, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((T, 8), generator=g, device="cuda").bfloat16()
    y8, scales = torch.empty((T, 8), device="cuda").to(torch.float8_e4m3fn), torch.empty((T, 1), device="cuda")
    K.k3_add_rms_norm(rows, None, T, 8, w, 1e-6, y=y, y8=y8, scales=scales, group=8)
    torch.cuda.synchronize()
    z = torch.log_softmax(x.double(), 1)
    best, at = torch.sort(z, 1, descending=True)
    # (5 terms and values up to 6 or so: a few roundings of each, 2^-24 relative)
    assert ((o["logprob"] - z.gather(1, tokens.long()[:, None])[:, 0]).abs() < 1e-5).all()
    assert torch.equal(o["top"].long(), at[:, :2]) and ((o["top_logprob"] - best[:, :2]).abs() < 1e-5).all()
    S.check_norm({"y": y, "y8": y8, "scales": scales}, *S.norm(rows, None, w, 1e-6), "bf16", 8)
