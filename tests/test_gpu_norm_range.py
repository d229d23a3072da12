"""k3_add_rms_norm where the row's sum of squares leaves fp32's range and the
mean, or the result, does not (tests/_step.py has the 64-bit reference)."""
import math

import pytest

from tests import _step as S
from tests._gpu import say
from tests.test_gpu_norm import call, outputs

pytestmark = pytest.mark.gpu


def values(T, N, low, high, seed):
    """Signs and sizes between low and high, in 16 bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = low + (high - low) * torch.rand((T, N), generator=g, device="cuda", dtype=torch.float64)
    return (x * torch.where(torch.rand((T, N), generator=g, device="cuda") < 0.5, -1.0, 1.0)).bfloat16()


def run(x, r, w, eps, group):
    import torch
    o = outputs(*x.shape, "bf16", True, group)
    call(x, r, w, o, eps=eps, group=group)
    torch.cuda.synchronize()
    return o


SHAPES = [(3, 8, 8), (3, 520, 0), (300, 512, 128), (2, 7168, 7168), (300, 7168, 0), (300, 8192, 512), (1, 16384, 16384)]


@pytest.mark.parametrize("T,N,group", SHAPES)
@pytest.mark.parametrize("weight", [1.0, 1e15])
def test_mean_square_in_range_and_sum_not(T, N, group, weight):
    """Values about 1e19: their squares' sum passes 3.4e38, the mean is about 1e38."""
    import torch
    say(f"norm of large rows T={T} N={N} group={group} weight={weight}")
    x = values(T, N, 0.5e19, 1.3e19, N)
    r = values(T, N, 0, 1e18, N + 1)
    if T > 2:
        x[1], r[1] = values(1, N, 0, 1, 5)[0], 0
        x[1, 3] = 2.5e19 if N < 10 else 3e20  # one value has all
    w = (values(1, N, 0.7, 1.3, 3)[0].float() * weight).bfloat16()
    for eps in (1e-6, 1e30):
        S.check_norm(run(x, r, w, eps, group), *S.norm(x, r, w, eps), "bf16", group)


@pytest.mark.parametrize("T,N,group", SHAPES)
def test_mean_square_past_the_range(T, N, group):
    """Rows past it give 0, whatever the product with the weights is; infinities give NaN, in their places."""
    import torch
    say(f"norm of rows past fp32's range T={T} N={N} group={group}")
    x = values(T, N, 1e25, 1e26, N)
    x[0, 5] = math.inf
    w = values(1, N, 1e19, 2e19, 3)[0]
    o = run(x, None, w, 1e-6, group)
    assert torch.equal(o["sum"], x)
    odd = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    odd[0, 5] = True
    assert torch.equal(o["y"].isnan(), odd) and (o["y"][~odd] == 0).all()
    if group:
        groups = odd.view(T, -1, group).any(2)
        assert torch.equal(o["scales"].isnan(), groups) and (o["scales"][~groups] == 0).all()
        assert (o["y8"].float().view(T, -1, group)[~groups] == 0).all()


@pytest.mark.parametrize("T,N,group", SHAPES)
@pytest.mark.parametrize("size,eps", [(1e-25, 0.0), (3e-38, 0.0), (2.0 ** -131, 0.0), (1e-20, 1e-38), (1e-18, 1e-44),
                                      (1e-17, 0.0)])
def test_small_rows(T, N, group, size, eps):
    """Squares below fp32's range, with eps 0 or below it too."""
    import torch
    say(f"norm of small rows T={T} N={N} group={group} size={size} eps={eps}")
    x = values(T, N, 0.5 * size, 2 * size, N)
    if T > 2:
        x[1] = 0
        x[1, 3] = size
        x[2] = 0
    w = values(1, N, 0.7, 1.3, 3)[0]
    o = run(x, None, w, eps, group)
    rows = [t for t in range(T) if T <= 2 or t != 2]
    # (eps as the call has it, in fp32)
    s, y = S.norm(x[rows], None, w, float(torch.tensor(eps, dtype=torch.float32)))
    S.check_norm({k: None if v is None else v[rows] for k, v in o.items()}, s, y, "bf16", group)
    if T > 2:
        assert o["y"][2].isnan().all() if eps == 0 else (o["y"][2] == 0).all()


def test_in_place():
    """sum over the residual, y over the rows, on rows that go over twice and on others."""
    import torch
    say("norm of large and small rows in place")
    for T in (4, 400):
        x, r = values(T, 2048, 0.5e19, 1e19, 1), values(T, 2048, 0, 1e19, 2)
        x[1::2], r[1::2] = values(T, 2048, 1, 2, 3)[1::2], values(T, 2048, 1, 2, 4)[1::2]
        w = values(1, 2048, 0.7, 1.3, 3)[0]
        want = run(x, r, w, 1e-6, 0)
        S.check_norm(want, *S.norm(x, r, w, 1e-6), "bf16", 0)
        call(x, r, w, {"sum": r, "y": x, "y8": None, "scales": None})
        torch.cuda.synchronize()
        assert torch.equal(r, want["sum"]) and torch.equal(x, want["y"])
