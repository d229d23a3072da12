"""Greedy decoding with drafted trees: the paged cache calls and the expert
layer together, on a small decoder with random weights.

Each step drafts a tree per request out of what followed the last token
before, plans the step on the device (k3_kv_plan), and for each layer appends
and attends (k3_qk_norm_rope, k3_tree_attention) and runs the routed experts
(k3_moe_layer_batched). The drafts that greedy decoding would have chosen are
kept (k3_kv_commit_ex). At the end the whole sequences are run once more as
prompts, and the tokens compared with what that would have chosen.

    python examples/tree_decode.py [--requests 4] [--tokens 64] [--cache e4m3]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_packed_weight_amd as K  # noqa: E402
from gen import device  # noqa: E402

HIDDEN, INTER, EXPERTS, TOPK = 512, 256, 16, 4
LAYERS, QUERY_HEADS, HEADS, HEAD_DIM = 2, 8, 2, 64
VOCAB, PAGE, WORDS, EPS = 211, 16, 1, 1e-6
CACHES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def i32(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def zeros(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Decoder:
    """The weights, and one step over a planned batch."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.embed, self.unembed = normal(VOCAB, HIDDEN, std=1.0), normal(HIDDEN, VOCAB, std=HIDDEN ** -0.5)
        rows = (QUERY_HEADS + 2 * HEADS) * HEAD_DIM
        self.qkv = [normal(HIDDEN, rows, std=HIDDEN ** -0.5) for _ in range(LAYERS)]
        self.out = [normal(QUERY_HEADS * HEAD_DIM, HIDDEN, std=HIDDEN ** -0.5) for _ in range(LAYERS)]
        self.router = [normal(EXPERTS, HIDDEN, std=HIDDEN ** -0.5) for _ in range(LAYERS)]
        self.pools = [device.build_expert_pool(seed, 70 + i, EXPERTS, HIDDEN, INTER, 114, 120)
                      for i in range(LAYERS)]
        self.ones = torch.ones(HEAD_DIM, dtype=torch.bfloat16, device="cuda")
        half = HEAD_DIM // 2
        self.inv_freq = torch.tensor(10000.0 ** (-np.arange(half) / half), dtype=torch.float32, device="cuda")

    @staticmethod
    def normed(x):
        x = x.float()
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)).to(torch.bfloat16)

    def step(self, tokens, plan, cache):
        """Logits [T, VOCAB] of the step's tokens."""
        T = tokens.numel()
        x = self.embed[tokens.long()]
        ws = torch.empty(K.k3_tree_attention_workspace_bytes(T, QUERY_HEADS, HEADS, HEAD_DIM),
                         dtype=torch.uint8, device="cuda")
        expert_ws = torch.empty(K.k3_moe_batched_workspace_bytes(T, EXPERTS, HIDDEN, INTER, TOPK),
                                dtype=torch.uint8, device="cuda")
        q = torch.empty((T, QUERY_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        attended = torch.empty_like(q)
        for i in range(LAYERS):
            rows = self.normed(x) @ self.qkv[i]
            a, b = QUERY_HEADS * HEAD_DIM, (QUERY_HEADS + HEADS) * HEAD_DIM
            K.k3_qk_norm_rope(rows[:, :a], rows[:, a:b], rows[:, b:], T, QUERY_HEADS, self.ones, self.ones, EPS,
                              self.inv_freq, HEAD_DIM, False, plan.positions, q, cache.layers[i], plan.slots)
            K.k3_tree_attention(q, T, QUERY_HEADS, cache.layers[i], cache.table, cache.blocks, plan.cu, plan.kv_lens,
                                cache.requests, plan.mask, WORDS, HEAD_DIM ** -0.5, attended, ws)
            x = x + attended.view(T, -1) @ self.out[i]
            h = self.normed(x)
            y = torch.empty_like(h)
            K.k3_moe_layer_batched(h, self.router[i], self.pools[i].table, EXPERTS, HIDDEN, INTER, TOPK, T, y,
                                   expert_ws)
            x = x + self.normed(y)
        return self.normed(x).float() @ self.unembed.float()


class Cache:
    """Pages of all layers, who holds which, and which are free."""

    def __init__(self, requests, places, kind):
        self.requests, self.blocks = requests, -(-places // PAGE) + 1
        self.pages = requests * self.blocks
        shape = (LAYERS, self.pages, HEADS, PAGE, HEAD_DIM)
        k, v = (torch.zeros(shape, device="cuda").to(CACHES[kind]).permute(0, 1, 3, 2, 4) for _ in range(2))
        scale = torch.full((HEADS,), 2.0 ** -5, device="cuda") if kind == "e4m3" else None
        self.layers = [K.k3_kv_cache_of(k[i], v[i], scale, scale) for i in range(LAYERS)]
        self.layer_stride = k.stride(0)
        self.table = torch.full((requests, self.blocks), -1, dtype=torch.int32, device="cuda")
        self.ctx, self.held = zeros(requests), zeros(requests)
        self.ring, self.ring_state = i32(np.arange(self.pages)), i32([0, self.pages])

    def plan(self, new, parents):
        """The plan of a step with new[r] tokens per request."""
        T, R = int(sum(new)), self.requests
        p = argparse.Namespace(cu=zeros(R + 1), kv_lens=zeros(R), slots=zeros(T), positions=zeros(T),
                               mask=None if parents is None else zeros(T, WORDS), status=zeros(2))
        held, state = zeros(R), zeros(2)
        K.k3_kv_plan(self.ctx, i32(new), None if parents is None else i32(parents), R, T, self.pages, PAGE,
                     self.blocks, self.held, self.ring, self.ring_state, self.table, held, state, p.cu, p.kv_lens,
                     p.slots, p.positions, p.mask, WORDS, p.status)
        self.held, self.ring_state = held, state
        return p

    def commit(self, plan, accepted, counts):
        out = zeros(self.requests)
        K.k3_kv_commit_ex(self.layers[0], LAYERS, self.layer_stride, self.table, self.blocks, self.ctx, plan.kv_lens,
                          i32(accepted), i32(counts), len(accepted[0]), self.requests, out)
        self.ctx = out


def draft(root, followers, nodes):
    """A tree below `root` of the tokens that followed each before: tokens and parents, breadth first."""
    tokens, parents, at = [root], [-1], 0
    while at < len(tokens) and len(tokens) < nodes:
        for t in followers.get(tokens[at], [])[:2]:
            if len(tokens) < nodes:
                tokens.append(t)
                parents.append(at)
        at += 1
    return tokens, parents


def accepted_path(tokens, parents, choice):
    """The nodes that greedy decoding would have taken, from the root on, and the token after them."""
    path = [0]
    while True:
        want = choice[path[-1]]
        child = [i for i in range(len(tokens)) if parents[i] == path[-1] and tokens[i] == want]
        if not child:
            return path, want
        path.append(child[0])


def remember(followers, a, b):
    seen = followers.setdefault(a, [])
    if b in seen:
        seen.remove(b)
    seen.insert(0, b)


def run(requests, tokens, nodes, kind, seed=0, log=print):
    model = Decoder(seed)
    rng = np.random.default_rng(seed)
    text = [list(rng.integers(0, VOCAB, 5 + 9 * r)) for r in range(requests)]
    prompts = [len(t) for t in text]
    places = max(prompts) + tokens + 2 * nodes
    cache = Cache(requests, places, kind)
    followers = [{} for _ in range(requests)]
    plan = cache.plan(prompts, None)
    logits = model.step(i32(np.concatenate(text)), plan, cache)
    cache.ctx = plan.kv_lens
    ends = np.cumsum(prompts)
    roots = logits[i32(ends - 1).long()].argmax(-1).tolist()
    steps, turns = 0, 0  # turns: of the requests that had tokens in a step
    while min(len(t) - p for t, p in zip(text, prompts)) < tokens:
        # a request that has its tokens has no nodes: it keeps its pages, and waits
        trees = [draft(root, f, nodes) if len(t) - p < tokens else ([], [])
                 for root, f, t, p in zip(roots, followers, text, prompts)]
        new = [len(t) for t, _ in trees]
        plan = cache.plan(new, sum((p for _, p in trees), []))
        assert plan.status.tolist() == [0, 0]
        choice = model.step(i32(sum((t for t, _ in trees), [])), plan, cache).argmax(-1).tolist()
        accepted, counts, first = np.zeros((requests, nodes)), [], 0
        for r, (toks, parents) in enumerate(trees):
            if not toks:
                counts.append(0)
                continue
            path, root = accepted_path(toks, parents, choice[first:first + len(toks)])
            accepted[r, :len(path)] = path
            counts.append(len(path))
            for t in [toks[i] for i in path]:
                remember(followers[r], text[r][-1], t)
                text[r].append(t)
            roots[r] = root
            first += len(toks)
        cache.commit(plan, accepted, counts)
        steps += 1
        turns += sum(n > 0 for n in new)
    produced = sum(len(t) - p for t, p in zip(text, prompts))
    # the sequences as prompts: what would each place have chosen?
    again = Cache(requests, places, kind)
    whole = [len(t) for t in text]
    logits = model.step(i32(np.concatenate(text)), again.plan(whole, None), again)
    first, same = 0, 0
    for t, p in zip(text, prompts):
        choice = logits[first:first + len(t)].argmax(-1).tolist()
        same += sum(a == b for a, b in zip(choice[p - 1:-1], t[p:]))
        first += len(t)
    log(f"{produced} tokens of {requests} requests in {steps} steps ({produced / turns:.2f} to a request and step); "
        f"{same} of them are what a prompt of the same tokens would have chosen")
    return produced, turns, same


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--requests", type=int, default=4)
    a.add_argument("--tokens", type=int, default=64, help="tokens per request, at least")
    a.add_argument("--nodes", type=int, default=8, help="nodes of a drafted tree, at most 32")
    a.add_argument("--cache", choices=sorted(CACHES), default="bf16")
    o = a.parse_args(argv)
    if not 1 <= o.nodes <= 32 * WORDS:
        a.error(f"--nodes outside [1, {32 * WORDS}]")
    run(o.requests, o.tokens, o.nodes, o.cache)


if __name__ == "__main__":
    main()
