"""k3_add_rms_norm on the GPU against 64-bit floats (tests/_step.py)."""
import math

import pytest

import mxfp4_packed_weight_amd as K
from tests import _step as S
from tests._gpu import say

pytestmark = pytest.mark.gpu


def rows(T, N, kind, g, std=1.0, stride=None):
    import torch
    x = torch.randn((T, stride or N), generator=g, device="cuda") * std
    return x.to(S.torch_type(kind))[:, :N]


def outputs(T, N, kind, y, group, pad=0):
    import torch
    dt = S.torch_type(kind)
    junk = lambda d: torch.full((T, N + pad), 7.0, device="cuda").to(d)  # noqa: E731
    o = {"sum": junk(dt)[:, :N], "y": junk(dt)[:, :N] if y else None, "y8": None, "scales": None}
    if group:
        o["y8"] = junk(torch.float8_e4m3fn)[:, :N]
        o["scales"] = torch.full((T, N // group), -7.0, device="cuda")
    return o


def call(x, r, w, o, eps=1e-6, group=0, **kw):
    T, N = x.shape
    K.k3_add_rms_norm(x, r, T, N, w, eps, sum_out=o["sum"], y=o["y"], y8=o["y8"], scales=o["scales"], group=group, **kw)


CASES = [(1, 8, "bf16", 0), (1, 7168, "bf16", 0), (1, 7168, "f16", 7168), (3, 64, "f16", 32), (2, 16384, "bf16", 128),
         (5, 16384, "f16", 16384), (1, 8192, "bf16", 512), (1, 8200, "bf16", 8200), (300, 1000, "bf16", 1000),
         (257, 512, "f16", 256), (700, 2048, "bf16", 64), (1, 40, "f16", 40), (600, 8, "bf16", 8), (2, 520, "bf16", 0),
         (513, 4096, "bf16", 32), (400, 9216, "f16", 512)]


@pytest.mark.parametrize("T,N,kind,group", CASES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(T, N, kind, group, residual):
    import torch
    say(f"norm T={T} N={N} {kind} group={group} residual={residual}")
    g = torch.Generator(device="cuda").manual_seed(T + N)
    x = rows(T, N, kind, g, stride=N + 24)
    r = rows(T, N, kind, g, std=5.0, stride=N + 8) if residual else None
    w = (1 + 0.3 * torch.randn(N, generator=g, device="cuda")).to(x.dtype)
    s, y = S.norm(x, r, w, 1e-6)
    for with_y in ((True, False) if group else (True,)):
        o = outputs(T, N, kind, with_y, group, pad=16)
        call(x, r, w, o, group=group)
        torch.cuda.synchronize()
        S.check_norm(o, s, y, kind, group)
        for t in (o["sum"], o["y"], o["y8"]):  # what is behind the rows stays
            if t is not None:
                assert (t._base[:, N:].float() == 7).all()


def test_in_place_and_without_sum():
    """sum over the residual and y over x give what separate outputs do."""
    import torch
    say("norm in place")
    T, N = 40, 7168
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = rows(T, N, "bf16", g), rows(T, N, "bf16", g, std=3.0)
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    a = outputs(T, N, "bf16", True, 0)
    call(x, r, w, a)
    none = outputs(T, N, "bf16", True, 0) | {"sum": None}
    call(x, r, w, none)
    call(x, r, w, {"sum": r, "y": x, "y8": None, "scales": None})
    torch.cuda.synchronize()
    assert torch.equal(r, a["sum"]) and torch.equal(x, a["y"]) and torch.equal(none["y"], a["y"])


def test_rows_of_zeros_and_of_no_numbers():
    """Zero rows, zero groups, NaN and infinities stay in their rows."""
    import torch
    say("norm of zeros, NaN, infinities")
    T, N, group = 6, 256, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = rows(T, N, "bf16", g).clone()
    x[0] = 0
    x[1, 64:128] = 0
    x[2, 5] = math.nan
    x[3, 70] = math.inf
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    o = outputs(T, N, "bf16", True, group)
    call(x, None, w, o, group=group)
    for eps in (0.0,):  # a row of zeros without eps is 0 times infinity
        z = outputs(T, N, "bf16", True, group)
        call(x, None, w, z, eps=eps, group=group)
    torch.cuda.synchronize()
    assert (o["y"][0] == 0).all() and (o["scales"][0] == 0).all() and (o["y8"][0].float() == 0).all()
    assert z["y"][0].isnan().all()
    assert o["scales"][1, 1] == 0 and (o["y8"][1, 64:128].float() == 0).all() and o["scales"][1, 0] > 0
    assert o["y"][2].isnan().all() and o["scales"][2].isnan().all()
    assert (o["y"][3, :64] == 0).all() and o["y"][3, 70].isnan() and o["scales"][3, 1].isnan()
    assert o["scales"][3, 0] == 0
    s, y = S.norm(x[4:], None, w, 1e-6)
    S.check_norm({k: None if v is None else v[4:] for k, v in o.items()}, s, y, "bf16", group)


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e12])
def test_sizes_of_values(std):
    """Norms of small and large rows; a row far below eps has small scales."""
    import torch
    say(f"norm of values of {std}")
    T, N = 9, 512
    g = torch.Generator(device="cuda").manual_seed(3)
    x = rows(T, N, "bf16", g, std=std)
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    o = outputs(T, N, "bf16", True, 128)
    call(x, None, w, o, group=128)
    torch.cuda.synchronize()
    S.check_norm(o, *S.norm(x, None, w, 1e-6), "bf16", 128)


@pytest.mark.parametrize("group", [128, 512])
def test_small_rows_with_small_weights(group):
    """No eps: the factor of the row over the scale is past fp32's range, the codes are not."""
    import torch
    say(f"norm of small rows with small weights group={group}")
    T, N = 9, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    x = ((1 + torch.rand((T, N), generator=g, device="cuda")) * 3e-19).bfloat16()
    w = torch.full((N,), 1e-18, dtype=torch.bfloat16, device="cuda")
    o = outputs(T, N, "bf16", True, group)
    call(x, None, w, o, eps=0.0, group=group)
    torch.cuda.synchronize()
    S.check_norm(o, *S.norm(x, None, w, 0.0), "bf16", group)


def test_another_stream_and_a_graph():
    """On a stream of its own, and replayed with other inputs."""
    import torch
    say("norm on a stream and in a graph")
    T, N = 33, 1024
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r = rows(T, N, "bf16", g), rows(T, N, "bf16", g)
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    o = outputs(T, N, "bf16", True, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(x, r, w, o, group=128, stream=side)
    side.synchronize()
    S.check_norm(o, *S.norm(x, r, w, 1e-6), "bf16", 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, r, w, o, group=128)
    for i in range(4):
        x.copy_(rows(T, N, "bf16", g, std=1 + i))
        graph.replay()
        torch.cuda.synchronize()
        S.check_norm(o, *S.norm(x, r, w, 1e-6), "bf16", 128)


def test_no_rows():
    import torch
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    K.k3_add_rms_norm(x, None, 0, 64, w, 1e-6, y=x)
