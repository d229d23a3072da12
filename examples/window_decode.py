"""Greedy decoding with two kinds of layers: a sliding window with sinks over a
16-bit cache, and all places over a cache in 8 bits with an exponent for each
page and head.

Each step plans its pages on the device (k3_kv_plan), and for each layer adds
the residual and norms (k3_add_rms_norm), appends and attends, and runs the
routed experts (k3_moe_layer_batched). What the step's tokens were worth is
scored in the end (k3_token_logprobs). At the end the whole sequences are run
once more as prompts, and the choices compared.

    python examples/window_decode.py [--requests 4] [--tokens 48] [--window 32] [--sinks 4]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import tree_decode as base  # noqa: E402
from tree_decode import EPS, EXPERTS, HEAD_DIM, HEADS, HIDDEN, INTER, K, PAGE, QUERY_HEADS, TOPK, VOCAB, i32  # noqa: E402

LAYERS = base.LAYERS
ALTERNATIVES = 3


class Cache(base.Cache):
    """The first layer's cache as it was; the second one's in 8 bits with exponents."""

    def __init__(self, requests, places):
        super().__init__(requests, places, "bf16")
        shape = (self.pages, HEADS, PAGE, HEAD_DIM)
        k, v = (torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn).permute(0, 2, 1, 3) for _ in range(2))
        self.layers[1] = K.k3_kv_cache_of(k, v)
        self.k_exp, self.v_exp = (torch.zeros((self.pages, HEADS), dtype=torch.uint8, device="cuda") for _ in range(2))


class Decoder(base.Decoder):
    def __init__(self, seed, window, sinks):
        super().__init__(seed)
        self.window, self.sinks = window, sinks
        self.weights = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")

    def attend(self, i, rows, plan, cache):
        """One layer's attention of rows [T, queries, keys and values]."""
        T = rows.shape[0]
        a, b = QUERY_HEADS * HEAD_DIM, (QUERY_HEADS + HEADS) * HEAD_DIM
        q, k, v = rows[:, :a], rows[:, a:b], rows[:, b:]
        turned = torch.empty((T, QUERY_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(turned)
        ws = torch.empty(K.k3_tree_attention_workspace_bytes(T, QUERY_HEADS, HEADS, HEAD_DIM), dtype=torch.uint8,
                         device="cuda")
        norm = (T, QUERY_HEADS, self.ones, self.ones, EPS, self.inv_freq, HEAD_DIM, False, plan.positions, turned)
        scale = HEAD_DIM ** -0.5
        if i == 0:
            K.k3_qk_norm_rope(q, k, v, *norm, cache.layers[i], plan.slots)
            K.k3_window_attention(turned, T, QUERY_HEADS, cache.layers[i], cache.table, cache.blocks, plan.cu,
                                  plan.kv_lens, cache.requests, None, 1, self.window, self.sinks, scale, out, ws)
            return out
        # the step's keys in rows of their own first: their exponents need whole pages
        step_k, step_v = torch.empty((2, T, 1, HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        step = K.k3_kv_cache_of(step_k, step_v)
        K.k3_qk_norm_rope(q, k, v, *norm, step, torch.arange(T, dtype=torch.int32, device="cuda"))
        K.k3_kv_append(step_k.view(T, HEADS, HEAD_DIM), v, T, cache.layers[i], cache.k_exp, cache.v_exp, cache.table,
                       cache.blocks, plan.cu, plan.kv_lens, cache.requests)
        K.k3_block_attention(turned, T, QUERY_HEADS, cache.layers[i], cache.k_exp, cache.v_exp, cache.table,
                             cache.blocks, plan.cu, plan.kv_lens, cache.requests, 0, 0, scale, out, ws)
        return out

    def step(self, tokens, plan, cache):
        """Logits [T, VOCAB] of the step's tokens."""
        T = tokens.numel()
        x = self.embed[tokens.long()]
        h, y, change = torch.empty_like(x), torch.empty_like(x), None
        expert_ws = torch.empty(K.k3_moe_batched_workspace_bytes(T, EXPERTS, HIDDEN, INTER, TOPK), dtype=torch.uint8,
                                device="cuda")
        for i in range(LAYERS):
            K.k3_add_rms_norm(x, change, T, HIDDEN, self.weights, EPS, sum_out=x, y=h)
            change = self.attend(i, h @ self.qkv[i], plan, cache).view(T, -1) @ self.out[i]
            K.k3_add_rms_norm(x, change, T, HIDDEN, self.weights, EPS, sum_out=x, y=h)
            K.k3_moe_layer_batched(h, self.router[i], self.pools[i].table, EXPERTS, HIDDEN, INTER, TOPK, T, y,
                                   expert_ws)
            change = torch.empty_like(x)
            K.k3_add_rms_norm(y, None, T, HIDDEN, self.weights, EPS, y=change)
        K.k3_add_rms_norm(x, change, T, HIDDEN, self.weights, EPS, y=h)
        return h.float() @ self.unembed.float()


def score(logits, tokens):
    """Log probabilities of tokens [T], and the entropy and best alternatives beside them."""
    T = logits.shape[0]
    out = [torch.empty(T, device="cuda") for _ in range(2)]
    top = torch.empty((T, ALTERNATIVES), dtype=torch.int32, device="cuda")
    top_logprob = torch.empty((T, ALTERNATIVES), device="cuda")
    ws = torch.empty(K.k3_token_logprobs_workspace_bytes(T, VOCAB, ALTERNATIVES), dtype=torch.uint8, device="cuda")
    K.k3_token_logprobs(logits, T, VOCAB, 1.0, tokens, ALTERNATIVES, *out, None, top, top_logprob, ws)
    return out[0], out[1], top, top_logprob


def run(requests, tokens, window, sinks, seed=0, log=print):
    model = Decoder(seed, window, sinks)
    rng = np.random.default_rng(seed)
    text = [list(rng.integers(0, VOCAB, 5 + 9 * r)) for r in range(requests)]
    prompts = [len(t) for t in text]
    places = max(prompts) + tokens
    cache = Cache(requests, places)
    step, new, worth = i32(np.concatenate(text)), prompts, []
    for _ in range(tokens):
        plan = cache.plan(new, None)
        logits = model.step(step, plan, cache)
        cache.ctx = plan.kv_lens
        last = logits[plan.cu[1:].long() - 1]  # each request's next token
        step = last.argmax(-1).int()
        worth.append(score(last, step)[0])
        for t, n in zip(text, step.tolist()):
            t.append(n)
        new = [1] * requests
    worth = torch.stack(worth, 1)
    # the sequences as prompts: what would each place have chosen, and what was it worth?
    again, whole = Cache(requests, places), [len(t) - 1 for t in text]
    logits = model.step(i32(np.concatenate([t[:-1] for t in text])), again.plan(whole, None), again)
    chosen = i32(np.concatenate([t[1:] for t in text]))
    logprob, _, top, _ = score(logits, chosen)
    ends = np.cumsum(whole)
    rows = i32(np.stack([np.arange(e - tokens, e) for e in ends])).long()
    same = int((top[:, 0] == chosen)[rows].sum())
    off = float((logprob[rows] - worth).abs().mean())
    log(f"{requests * tokens} tokens of {requests} requests, {float(worth.mean()):.3f} nats each; {same} of them are what a "
        f"prompt of the same tokens would have chosen, whose log probabilities are {off:.3f} away on the average")
    return requests * tokens, same, worth, logprob[rows]


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--requests", type=int, default=4)
    a.add_argument("--tokens", type=int, default=48, help="tokens per request")
    a.add_argument("--window", type=int, default=32, help="places that the first layer sees (0: all)")
    a.add_argument("--sinks", type=int, default=4, help="first tokens that it sees as well")
    o = a.parse_args(argv)
    if o.requests < 1 or o.tokens < 1 or o.window < 0 or o.sinks < 0:
        a.error("requests and tokens of 1 at least, window and sinks of 0 at least")
    run(o.requests, o.tokens, o.window, o.sinks)


if __name__ == "__main__":
    main()
