"""The example of decoding with windowed layers and a cache with exponents, run
whole, and a layer's calls of it captured into a graph."""
import os
import sys

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests._gpu import say

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, EXAMPLES)
    try:
        import window_decode
    finally:
        sys.path.remove(EXAMPLES)
    return window_decode


@pytest.mark.parametrize("requests,tokens,window,sinks", [(3, 40, 16, 2), (2, 20, 0, 0), (1, 1, 1, 0)])
def test_window_decode(example, requests, tokens, window, sinks):
    """The tokens are those that the sequences, run as prompts, would have
    chosen: all but those where rounding (another order of the same products,
    codes of pages whose exponent rose later) decides between two tokens, given
    as one in ten, as for drafted trees."""
    say(f"window decode, {requests} requests, window {window}")
    produced, same, worth, again = example.run(requests, tokens, window, sinks, log=say)
    assert produced == requests * tokens and worth.shape == again.shape == (requests, tokens)
    assert (worth <= 0).all() and (again <= 0).all() and same >= 0.9 * produced


def test_a_step_in_a_graph():
    """Norm, append, both attentions and the scores of a step, replayed with
    other inputs and longer requests: each replay has the eager calls' bits."""
    import torch
    say("a step with a window and exponents in a graph")
    g = torch.Generator(device="cuda").manual_seed(3)
    R, H, Hq, D, P, blocks, V, N = 5, 2, 8, 64, 16, 12, 1003, 512
    pages = R * blocks
    table = R_.i32(np.random.default_rng(3).permutation(pages).reshape(R, blocks))
    cu = R_.i32(np.arange(R + 1))
    rows, width = (Hq + 2 * H) * D, torch.randn((N, (Hq + 2 * H) * D), generator=g, device="cuda") * N ** -0.5
    unembed = (torch.randn((Hq * D, V), generator=g, device="cuda") * 0.1).bfloat16()
    width, ones = width.bfloat16(), torch.ones(N, dtype=torch.bfloat16, device="cuda")

    def state():
        k16, v16 = (torch.zeros((pages, H, P, D), dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3) for _ in "kv")
        k8, v8 = (torch.zeros((pages, H, P, D), device="cuda").to(torch.float8_e4m3fn).permute(0, 2, 1, 3) for _ in "kv")
        zeros = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        return {"x": zeros(R, N), "change": zeros(R, N), "h": zeros(R, N), "lens": zeros(R, dtype=torch.int32),
                "slots": zeros(R, dtype=torch.int32), "c16": K.k3_kv_cache_of(k16, v16), "c8": K.k3_kv_cache_of(k8, v8),
                "caches": (k16, v16, k8, v8), "exps": zeros(2, pages, H, dtype=torch.uint8),
                "out": zeros(2, R, Hq, D), "turned": zeros(R, Hq, D), "lp": zeros(3, R, dtype=torch.float32),
                "top": zeros(R, 4, dtype=torch.int32), "tlp": zeros(R, 4, dtype=torch.float32),
                "tokens": zeros(R, dtype=torch.int32),
                "ws": zeros(K.k3_tree_attention_workspace_bytes(R, Hq, H, D), dtype=torch.uint8),
                "lws": zeros(max(1, K.k3_token_logprobs_workspace_bytes(R, V, 4)), dtype=torch.uint8)}

    def step(s):
        K.k3_add_rms_norm(s["x"], s["change"], R, N, ones, 1e-6, sum_out=s["x"], y=s["h"])
        qkv = s["h"] @ width
        q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + H) * D], qkv[:, (Hq + H) * D:]
        K.k3_qk_norm_rope(q, k, v, R, Hq, ones[:D], ones[:D], 1e-6, None, 0, False, s["lens"], s["turned"], s["c16"],
                          s["slots"])
        K.k3_window_attention(s["turned"], R, Hq, s["c16"], table, blocks, cu, s["lens"], R, None, 1, 40, 3, 0.125,
                              s["out"][0], s["ws"])
        K.k3_kv_append(k, v, R, s["c8"], s["exps"][0], s["exps"][1], table, blocks, cu, s["lens"], R)
        K.k3_block_attention(s["turned"], R, Hq, s["c8"], s["exps"][0], s["exps"][1], table, blocks, cu, s["lens"], R,
                             0, 0, 0.125, s["out"][1], s["ws"])
        logits = s["out"].sum(0).view(R, -1) @ unembed
        K.k3_token_logprobs(logits, R, V, 0.9, s["tokens"], 4, s["lp"][0], s["lp"][1], s["lp"][2], s["top"], s["tlp"],
                            s["lws"])

    a, b = state(), state()
    step(b)
    torch.cuda.synchronize()
    b = state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    length = np.array([0, 30, 75, 100, 15])
    for _ in range(5):
        length = length + 1
        for s in (a, b):
            g.manual_seed(int(length[0]))
            s["x"].copy_(torch.randn((R, N), generator=g, device="cuda"))
            s["change"].copy_(torch.randn((R, N), generator=g, device="cuda"))
            s["tokens"].copy_(torch.randint(0, V, (R,), generator=g, device="cuda"))
            s["lens"].copy_(R_.i32(length))
            at = torch.tensor(length - 1, device="cuda")
            s["slots"].copy_(table.long().gather(1, (at // P)[:, None]).squeeze(1) * P + at % P)
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("x", "h", "out", "exps", "lp", "top", "tlp"):
            x, y = a[name], b[name]
            assert torch.equal(x, y) and not (x.is_floating_point() and x.isnan().any()), name
        for x, y in zip(a["caches"], b["caches"]):
            assert torch.equal(x.float(), y.float())
