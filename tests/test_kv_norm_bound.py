"""The bound on the attention's whole error sees what it is there for (mistakes
planted in the 64-bit reference, on the CPU), and lets the roundings pass."""
import numpy as np
import pytest
import torch

from tests import _kv as R_
from tests import _kv_norm as N


def case(L, n, G, D, dt, P=16):
    g = torch.Generator()
    g.manual_seed(L + n)
    pages = -(-L // P)
    k, v = (torch.randn((pages, P, 1, D), generator=g).to(R_.torch_type(dt)).double() for _ in range(2))
    q = (torch.randn((n, G, D), generator=g) * 1.5).to(R_.torch_type(dt))
    return {"q": q, "clean": (k, v), "ks": None, "vs": None, "table": np.arange(pages)[None], "cu": [0, n],
            "lens": [L], "mask": None, "scale": D ** -0.5, "P": P, "pages": pages, "H": 1, "dt": dt}


@pytest.mark.parametrize("L,n,dt", [(30000, 8, "bf16"), (30000, 1, "f16"), (300, 4, "bf16")])
def test_roundings_pass(L, n, dt):
    """Weights and outputs rounded as the kernels round them."""
    s = case(L, n, 8, 64, dt)
    want, t16 = N.exact(s), R_.torch_type(dt)
    k, v = (x.flatten(0, 1)[:L, 0] for x in s["clean"])
    x = torch.einsum("ngd,ld->ngl", s["q"].double(), k) * s["scale"]
    x = x.masked_fill(~R_.sees(n, L, None)[:, None], -np.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.einsum("ngl,ld->ngd", w.to(t16).double(), v) / w.sum(-1, keepdim=True)
    worst = N.check(o.to(t16), want, s)
    assert worst > 0.4


@pytest.mark.parametrize("n", [1, 40])
def test_a_wrong_block_is_seen(n):
    """Values of 64 places in the middle are another block's."""
    s = case(30000, n, 8, 64, "bf16")
    want, v = N.exact(s), s["clean"][1].clone()
    v[800:804] = s["clean"][1][900:904]
    with pytest.raises(AssertionError):
        N.check(N.exact(s, v=v), want, s)


@pytest.mark.parametrize("place", [2047, 2048, 29000])
def test_one_misplaced_row_is_seen(place):
    """A place's key and value are its neighbour's."""
    s = case(30000, 40, 8, 64, "bf16")
    want = N.exact(s)
    k, v = (x.clone() for x in s["clean"])
    a, b = place, place - 64
    for x in (k, v):
        x[a // 16, a % 16] = x[b // 16, b % 16]
    with pytest.raises(AssertionError):
        N.check(N.exact(s, k=k, v=v), want, s)
