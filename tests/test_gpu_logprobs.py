"""k3_token_logprobs on the GPU against 64-bit floats, row by row
(tests/_step.py)."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _step as S
from tests._gpu import say

pytestmark = pytest.mark.gpu


def call(x, beta, tokens, k, stream=None, ws=None, outs=None):
    import torch
    T, V = x.shape
    junk = lambda *s: torch.full(s, -7.5, device="cuda")  # noqa: E731
    o = outs or {"logprob": junk(T), "entropy": junk(T), "lse": junk(T),
                 "top": torch.full((T, k), -77, dtype=torch.int32, device="cuda"), "top_logprob": junk(T, k)}
    if ws is None:
        ws = torch.empty(K.k3_token_logprobs_workspace_bytes(T, V, k), dtype=torch.uint8, device="cuda")
    K.k3_token_logprobs(x, T, V, beta, tokens, k, o["logprob"], o["entropy"], o["lse"], o["top"] if k else None,
                        o["top_logprob"] if k else None, ws, stream=stream)
    return o


def check(x, beta, tokens, k):
    import torch
    o = call(x, beta, torch.tensor(np.asarray(tokens, np.int32), device="cuda"), k)
    torch.cuda.synchronize()
    got = {n: v.cpu().numpy() for n, v in o.items()}
    S.check_logprobs(got, S.logprobs(x, beta, tokens, k), x.shape[1])
    return got


def logits(T, V, kind, seed, std=3.0, stride=None, lead=0):
    """Rows whose first is `lead` values from a 16-byte boundary."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = stride or V
    x = torch.empty(T * stride + lead, dtype=S.torch_type(kind), device="cuda")
    x.copy_(torch.randn(x.shape, generator=g, device="cuda") * std)
    return x[lead:].view(T, stride)[:, :V]


SHAPES = [(1, 1), (1, 2), (3, 7), (2, 63), (1, 64), (5, 65), (2, 511), (2, 512), (3, 513), (1, 1023), (2, 1025),
          (4, 4095), (1, 4097), (1, 8200), (2, 32001), (1, 131072), (3, 200003), (40, 9001), (2100, 1030)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_shapes(T, V, kind):
    k = min(V, [5, 20, 64, 1, 0][(T + V) % 5])
    say(f"logprobs T={T} V={V} {kind} k={k}")
    x = logits(T, V, kind, T + V, stride=V + V % 3, lead=V % 5)
    check(x, [1.0, 0.6, 1.9][V % 3], np.random.default_rng(V).integers(0, V, T), k)


@pytest.mark.parametrize("k", [1, 20, 64])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_equal_logits(kind, k):
    """Ties go to the lower index, within and between the parts of a row."""
    import torch
    say(f"logprobs of equal logits {kind} k={k}")
    V = 20011
    x = torch.round(logits(6, V, kind, 3, std=1.5))
    x[0] = 2.5
    x[1] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0).to(x.dtype)
    x[2] = 0
    x[2, V - 3:] = 1
    x[3] = -1
    x[3, ::777] = 4
    check(x, 1.0, [0, V - 1, V - 1, 777, 5, 6], k)


def test_rising_and_falling_rows():
    """Every next logit is among the largest; none is."""
    import torch
    say("logprobs of sorted rows")
    V = 12345
    x = torch.arange(V, device="cuda", dtype=torch.float32)[None].repeat(3, 1) * 1e-3
    x[1] = x[1].flip(0)
    x[2, :6000] = 20
    check(x, 1.0, [V - 1, 0, 3], 64)
    check(x[:, 1:], 1.0, [1, 2, 3], 20)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_masked_rows(kind):
    """-inf: part of a row, all but a few, all; the type's lowest number; a token that is masked."""
    import torch
    say(f"logprobs of masked rows {kind}")
    V = 5003
    x = logits(8, V, kind, 11).clone()
    low = torch.finfo(x.dtype).min
    x[0, 100:4000] = -math.inf
    x[1] = -math.inf
    x[2] = -math.inf
    x[2, [17, 4999, 300]] = torch.tensor([1.0, 2.0, 1.0], device="cuda", dtype=x.dtype)
    x[3] = low
    x[4, 5:] = low
    x[5] = low
    x[5, 3000:] = -math.inf
    x[6] = -math.inf
    x[6, V - 1] = -3.0
    x[7, :4500] = -math.inf
    for k in (0, 5, 64):
        check(x, 1.0, [200, 0, 300, 7, 6, 4000, V - 1, 4600], k)


@pytest.mark.parametrize("k", [0, 7])
@pytest.mark.parametrize("beta", [0.01, 1.0, 1.9])
def test_large_numbers(beta, k):
    """Logits about 1e30 and beyond, of both signs, alone and with ordinary ones, in one part and in several."""
    import torch
    say(f"logprobs of large numbers beta={beta} k={k}")
    for T, V in ((6, 2003), (6, 70001)):
        x = logits(T, V, "f32", 17, std=1.0).clone()
        sizes = torch.tensor([0.9e30, 1e30, 1.1e30, 1e38], device="cuda")
        big = sizes[(x.abs() * 1000).long() % 4]
        x[0] = big[0].clamp(max=1.1e30)
        x[1] = -big[1]
        x[2, ::3] = -big[2, ::3]
        x[3, V // 2:] = big[3, V // 2:]
        x[4, :V - 2] = -big[4, :V - 2]
        x[5] = -1e38
        x[5, 1::2] = -math.inf
        check(x, beta, [0, 1, 2, V - 1, V - 1, V // 2 | 1], k)


def test_rows_of_no_numbers():
    """NaN and +inf: the row's figures are NaN, other rows' are not; NaN is not listed."""
    import torch
    say("logprobs of NaN and infinities")
    V = 3001
    x = logits(7, V, "f32", 12).clone()
    x[1, 1500] = math.nan
    x[2, 7] = math.inf
    x[3] = math.nan
    x[4] = math.nan
    x[4, [9, 2000]] = torch.tensor([1.0, -math.inf], device="cuda")
    x[5, 3000] = -math.nan
    check(x, 1.0, [3, 3, 7, 0, 9, 1, 2], 20)
    check(x.bfloat16(), 1.0, [3, 3, 7, 0, 9, 1, 2], 20)


def test_tokens_out_of_range_and_left_out():
    import torch
    say("logprobs of padded tokens")
    x = logits(5, 1000, "bf16", 13)
    got = check(x, 1.0, [-1, 1000, 2 ** 31 - 1, -2 ** 31, 999], 3)
    assert np.isneginf(got["logprob"][:4]).all() and np.isfinite(got["logprob"][4])
    lse = torch.zeros(5, device="cuda")
    ws = torch.empty(K.k3_token_logprobs_workspace_bytes(5, 1000, 0), dtype=torch.uint8, device="cuda")
    K.k3_token_logprobs(x, 5, 1000, 1.0, None, 0, None, None, lse, None, None, ws)
    torch.cuda.synchronize()
    assert np.array_equal(lse.cpu().numpy(), got["lse"])


@pytest.mark.parametrize("beta", [2.0 ** -20, 0.01, 30.0, 2.0 ** 20])
def test_temperatures(beta):
    """From an even distribution to one on the largest logit."""
    say(f"logprobs at beta={beta}")
    x = logits(3, 9000, "f32", 14)
    check(x, beta, [1, 2, 3], 8)


def test_same_bits_on_a_stream_and_in_a_graph():
    """A second call, one on another stream and replays of a graph give the same bits; two graphs share a workspace."""
    import torch
    say("logprobs on a stream and in graphs")
    T, V, k = 3, 50021, 20
    x = logits(T, V, "bf16", 15)
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    ws = torch.empty(K.k3_token_logprobs_workspace_bytes(T, V, k), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    same = lambda a, b: all(torch.equal(a[n].view(torch.int32), b[n].view(torch.int32)) for n in a)  # noqa: E731
    a, b = call(x, 0.7, tokens, k, ws=ws), call(x, 0.7, tokens, k, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = call(x, 0.7, tokens, k)
    side.synchronize()
    torch.cuda.synchronize()
    assert same(a, b) and same(a, c)
    graphs, outs = [], []
    for beta in (0.7, 1.0):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(x, beta, tokens, k, ws=ws))
    for i in range(3):
        x.copy_(logits(T, V, "bf16", 20 + i))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for beta, o in zip((0.7, 1.0), outs):
            assert same(o, call(x, beta, tokens, k, ws=ws))


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own."""
    import torch
    say("two calls of logprobs at once")
    xs = [logits(2, 70001, "f32", 30), logits(5, 40000, "bf16", 31)]
    tokens = [torch.arange(x.shape[0], dtype=torch.int32, device="cuda") for x in xs]
    want = [call(x, 0.9, t, 20) for x, t in zip(xs, tokens)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for x, t, stream in zip(xs, tokens, streams):
            with torch.cuda.stream(stream):
                got.append(call(x, 0.9, t, 20))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(o[n].view(torch.int32), want[i % 2][n].view(torch.int32)) for n in o), i
