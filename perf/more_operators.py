"""More operators of a decoding step, as they are measured.

The residual's addition with the norm (16-bit and 8-bit outputs), attention
with a sliding window and sinks over the paged cache, the append to a cache
held in 8 bits with an exponent for each page and head, the attention over
it, and the log probabilities of the tokens. Where ``own`` is false, ``run``
computes them in elementary torch operations; where it is true it calls the
framework.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "e4m3": 1, "f32": 4}
_E4M3_MAX = 448.0


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # the norm before one token's router and experts: nothing but latency
        {"name": "norm_one", "op": "norm", "T": 1, "hidden": 7168, "dt": "bf16", "y": True, "group": 0},
        # a batch's drafts, for a product in 8 bits with scales of 128 values
        {"name": "norm_batch_e4m3", "op": "norm", "T": 2048, "hidden": 7168, "dt": "bf16", "y": False, "group": 128},
        # a long prompt: 16 bits for the router, 8 bits with a scale per row for the product
        {"name": "norm_prompt_both", "op": "norm", "T": 16384, "hidden": 7168, "dt": "bf16", "y": True, "group": 7168},
        # one token of each of 64 requests whose contexts are far longer than the window
        {"name": "window_decode", "op": "window", "R": 64, "ctx": 8191, "n": 1, "trees": False, "window": 1024,
         "sinks": 4, "H": 8, "G": 8, "D": 128, "dt": "bf16", "cache": "bf16", "page": 16},
        # verification of drafted trees of up to 64 nodes in a layer with a window
        {"name": "window_trees", "op": "window", "R": 32, "ctx": 8000, "n": 64, "trees": True, "window": 2048,
         "sinks": 16, "H": 8, "G": 8, "D": 128, "dt": "bf16", "cache": "e4m3", "page": 64},
        # two prompts' chunks, a head of its own for each query head
        {"name": "window_prompt_f16", "op": "window", "R": 2, "ctx": 6000, "n": 2048, "trees": False, "window": 1000,
         "sinks": 5, "H": 16, "G": 1, "D": 64, "dt": "f16", "cache": "f16", "page": 32},
        # one new token for each of 64 requests: most of their pages hold earlier rows
        {"name": "append_decode", "op": "append", "R": 64, "ctx": 8191, "n": 1, "H": 8, "D": 128, "dt": "bf16",
         "page": 16},
        # the chunks of long prompts
        {"name": "append_prompt", "op": "append", "R": 4, "ctx": 4000, "n": 8192, "H": 8, "D": 128, "dt": "bf16",
         "page": 16},
        # ordinary decoding over the 8-bit cache
        {"name": "block_decode", "op": "block", "R": 64, "ctx": 8191, "n": 1, "window": 0, "sinks": 0, "H": 8,
         "G": 8, "D": 128, "dt": "bf16", "page": 16},
        # the last chunks of two long prompts
        {"name": "block_prompt", "op": "block", "R": 2, "ctx": 6000, "n": 512, "window": 0, "sinks": 0, "H": 8,
         "G": 8, "D": 128, "dt": "bf16", "page": 64},
        # one answer's token with its five best alternatives, from 16-bit logits
        {"name": "logprobs_one", "op": "logprobs", "T": 1, "V": 131072, "stride": 131072, "dt": "bf16", "k": 5,
         "temperature": 1.0},
        # the scores of a prompt's tokens, an odd vocabulary in padded rows of fp32
        {"name": "logprobs_prompt", "op": "logprobs", "T": 1000, "V": 150001, "stride": 150016, "dt": "f32", "k": 20,
         "temperature": 0.7},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "window", "window", "append", "block", "logprobs"])
    page = rng.choice([16, 16, 24, 32, 64])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op == "norm":
        group = rng.choice([0, 32, 64, 128, 1])  # 1: a scale per row
        hidden = 8 * _log(rng, 8, 2048) if group < 2 else group * _log(rng, 1, 16384 // group)
        T = _log(rng, 1, max(2, min(16384, 16384 * 7168 // hidden)))
        return {"op": op, "T": T, "hidden": hidden, "dt": dt, "y": group == 0 or rng.random() < 0.4,
                "group": hidden if group == 1 else group}
    if op in ("window", "block"):
        kind = rng.choice(["one", "trees", "prompt"] if op == "window" else ["one", "few", "prompt"])
        D = rng.choice([64, 128, 128, 256])
        H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 5, 8])
        R = _log(rng, 1, {"one": 64, "trees": 32, "few": 32, "prompt": 2}[kind])
        scores = 2e8 * 128 / D / (R * H * G)  # of the padded batch, for each query head
        n = {"one": 1, "trees": _log(rng, 2, 64), "few": _log(rng, 2, 8),
             "prompt": _log(rng, 65, max(66, min(2048, int(scores ** 0.5))))}[kind]
        most = max(16, min(int(scores / n), 131072, int(2.6e8 / (R * H * D))))
        case = {"op": op, "R": R, "ctx": _log(rng, 16, most), "n": n, "H": H, "G": G, "D": D, "dt": dt, "page": page}
        if op == "window":
            return case | {"trees": kind == "trees", "window": _log(rng, 64 if kind == "trees" else 1, 8192),
                           "sinks": rng.choice([0, 1, 4, 16, 100]), "cache": rng.choice([dt, dt, "e4m3"])}
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        return case | {"window": window, "sinks": rng.choice([0, 4]) if window else 0}
    if op == "append":
        D, H, R = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
        most = max(1, min(int(2.4e7 * 8 / (R * H * D)), 65536 // R))
        return {"op": op, "R": R, "ctx": _log(rng, 1, 8192), "n": _log(rng, 1, min(most, 8192)), "H": H, "D": D,
                "dt": dt, "page": page}
    V = _log(rng, 1000, 200000)
    kind = rng.choice(["bf16", "f16", "f32"])
    T = _log(rng, 1, max(2, min(4096, int(6e8 / _SIZE[kind] / V))))
    return {"op": op, "T": T, "V": V, "stride": V + rng.choice([0, 0, -V % 64]), "dt": kind,
            "k": rng.choice([0, 1, 5, 20]), "temperature": rng.choice([1.0, 0.7, 1.5])}


# ---- inputs -------------------------------------------------------------------

def _lengths(case):
    """Committed and new lengths of a ragged batch: spread evenly, the last the longest."""
    R = case["R"]
    ctx = [max(1, round(case["ctx"] * (r + 1) / R)) for r in range(R)]
    new = [max(1, round(case["n"] * ((7 * r + R) % R + 1) / R)) for r in range(R)]
    return ctx, new


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=_DEV)


def _tree(n, rs):
    """Parents of a drafted tree of n nodes, in an order where parents come first; node 0 is the root."""
    at = np.arange(n)
    p = np.maximum(0, at - 1 - (rs.random_sample(n) * np.minimum(at, 6)).astype(np.int64))
    p[:1] = -1
    return p


def _normal(shape, g, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32) * scale).to(dt)


def _exponents(amax):
    """The bytes e + 127 of the smallest powers of two 2^e with amax <= 448 2^e."""
    m, e = torch.frexp(amax.float())  # amax = m 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).int()
    return torch.where(amax > 0, (e + 127).clamp(1, 254), torch.ones_like(e)).to(torch.uint8)


def _power(byte):
    return torch.ldexp(torch.ones(byte.shape, device=byte.device), byte.int() - 127)


def _cache(shape, g, kind, scale=None):
    """Keys or values as a cache holds them, [pages, heads, page, D] in memory, seen as [pages, page, heads, D];
    with `scale` "blocks" also the exponents [pages, heads]."""
    pages, page, H, D = shape
    out = torch.empty((pages, H, page, D), dtype=_DT[kind], device=_DEV)
    exps = torch.empty((pages, H), dtype=torch.uint8, device=_DEV)
    for p in range(0, pages, 1024):  # in parts, for the random numbers' sake
        x = torch.randn(out[p:p + 1024].shape, generator=g, device=_DEV, dtype=torch.float32)
        if scale == "blocks":  # pages differ in size
            x = x * torch.exp2(2 * torch.randn(x.shape[:2], generator=g, device=_DEV))[..., None, None]
            exps[p:p + 1024] = e = _exponents(x.abs().amax((2, 3)))
            x = x / _power(e)[..., None, None]
        elif kind == "e4m3":
            x = x / scale[:, None, None]
        out[p:p + 1024] = (x.clamp(-_E4M3_MAX, _E4M3_MAX) if kind == "e4m3" else x).to(out.dtype)
    return (out.permute(0, 2, 1, 3), exps) if scale == "blocks" else out.permute(0, 2, 1, 3)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    s = {"case": case, "op": case["op"]}

    if case["op"] == "norm":
        T, N, dt = case["T"], case["hidden"], _DT[case["dt"]]
        big = 1 + 20 * (torch.rand((N,), generator=g, device=_DEV) < 0.003)  # some channels are large, as in models
        s |= {"T": T, "hidden": N, "eps": 1e-6, "group": case["group"], "x": _normal((T, N), g, dt),
              "residual": (_normal((T, N), g, torch.float32, 3.0) * big).to(dt),
              "w": _normal((N,), g, torch.float32, 0.2).add(1).to(dt),
              "sum": torch.zeros((T, N), dtype=dt, device=_DEV),
              "y": torch.zeros((T, N), dtype=dt, device=_DEV) if case["y"] else None, "y8": None, "scales": None}
        if case["group"]:
            s |= {"y8": torch.zeros((T, N), dtype=torch.float8_e4m3fn, device=_DEV),
                  "scales": torch.zeros((T, N // case["group"]), device=_DEV)}
        return s

    if case["op"] == "logprobs":
        T, V, k = case["T"], case["V"], case["k"]
        rows = torch.empty((T, case["stride"]), dtype=_DT[case["dt"]], device=_DEV)
        for t in range(0, T, 256):
            x = torch.randn((min(256, T - t), case["stride"]), generator=g, device=_DEV) * 2.5
            x += 4 * (torch.rand(x.shape, generator=g, device=_DEV) < 2e-4)  # a few likely tokens
            if t % 512 == 0:  # a grammar's mask over part of the vocabulary
                x[:, V // 3:V // 2] = -math.inf
            rows[t:t + 256] = x
        s |= {"T": T, "V": V, "k": k, "rows": rows, "logits": rows[:, :V], "beta": 1.0 / case["temperature"],
              "tokens": _i32(rs.randint(0, V, T)), "logprob": torch.zeros(T, device=_DEV),
              "entropy": torch.zeros(T, device=_DEV), "lse": torch.zeros(T, device=_DEV),
              "top": _i32(np.zeros((T, k))) if k else None,
              "top_logprob": torch.zeros((T, k), device=_DEV) if k else None}
        return s

    # a paged cache, and a step's new tokens at the requests' ends
    R, H, D, P = case["R"], case["H"], case["D"], case["page"]
    ctx, new = (np.array(v) for v in _lengths(case))
    order = rs.permutation(R)
    ctx, new = ctx[order], new[order]
    lens = ctx + new
    T, blocks = int(new.sum()), int(-(-lens.max() // P))
    need = -(-lens // P)
    first = ctx // P if case["op"] == "append" else np.zeros(R, int)  # only the pages that are written
    n_pages = int((need - first).sum()) + 1
    pages, off = rs.permutation(n_pages), np.concatenate([[0], np.cumsum(need - first)])
    table = np.full((R, blocks), -1)
    for r in range(R):
        table[r, first[r]:need[r]] = pages[off[r]:off[r + 1]]
    s |= {"R": R, "T": T, "H": H, "D": D, "P": P, "blocks": blocks, "n_pages": n_pages, "table": _i32(table),
          "cu": _i32(np.concatenate([[0], np.cumsum(new)])), "kv_lens": _i32(lens), "longest": int(lens.max()),
          "most": case["n"], "k_scale": None, "v_scale": None, "k_exp": None, "v_exp": None}
    dt = _DT[case["dt"]]
    if case["op"] == "window":
        if case["cache"] == "e4m3":
            r = torch.rand((2, H), generator=g, device=_DEV)
            s |= {"k_scale": (0.01 + 0.01 * r[0]).contiguous(), "v_scale": (0.01 + 0.01 * r[1]).contiguous()}
        s |= {"k": _cache((n_pages, P, H, D), g, case["cache"], s["k_scale"]),
              "v": _cache((n_pages, P, H, D), g, case["cache"], s["v_scale"])}
    else:
        s["k"], s["k_exp"] = _cache((n_pages, P, H, D), g, "e4m3", "blocks")
        s["v"], s["v_exp"] = _cache((n_pages, P, H, D), g, "e4m3", "blocks")
    if case["op"] == "append":
        # a token's keys next to its values, in rows of both; the step's tokens differ in size
        size = torch.exp2(torch.randn((T, 1), generator=g, device=_DEV))
        s["kv"] = (_normal((T, 2 * H * D), g, torch.float32) * size).to(dt)
        s |= {"k_in": s["kv"][:, :H * D], "v_in": s["kv"][:, H * D:]}
        return s
    Hq = H * case["G"]
    words, mask = -(-case["n"] // 32), None
    if case.get("trees"):
        mask = np.zeros((T, words * 32), np.uint8)
        row = 0
        for k in new:
            p = _tree(k, rs)
            for i in range(k):
                if i:
                    mask[row + i] = mask[row + p[i]]
                mask[row + i, i] = 1
            row += k
        mask = _i32(np.packbits(mask, axis=1, bitorder="little").view(np.int32))
    s |= {"Hq": Hq, "words": words, "mask": mask, "window": case["window"], "sinks": case["sinks"],
          "scale": D ** -0.5, "q": _normal((T, Hq * D), g, dt, 1.5).view(T, Hq, D),
          "out": torch.zeros((T, Hq, D), dtype=dt, device=_DEV), "lse": torch.zeros((T, Hq), device=_DEV)}
    return s


# ---- one pass -----------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_cache(s):
    """The cache's handle, made once as a program would."""
    import mxfp4_packed_weight_amd as K
    if "handle" not in s:
        s["handle"] = K.k3_kv_cache_of(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s["handle"]


def _own_workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device=_DEV)
    return s["ws"]


def _own_norm(s):
    import mxfp4_packed_weight_amd as K
    K.k3_add_rms_norm(s["x"], s["residual"], s["T"], s["hidden"], s["w"], s["eps"], sum_out=s["sum"], y=s["y"],
                      y8=s["y8"], scales=s["scales"], group=s["group"])
    return {"sum": s["sum"], "y": s["y"], "y8": s["y8"], "scales": s["scales"]}


def _own_window(s):
    import mxfp4_packed_weight_amd as K
    c = _own_cache(s)
    ws = _own_workspace(s, lambda: K.k3_tree_attention_workspace_bytes(s["T"], s["Hq"], s["H"], s["D"]))
    K.k3_window_attention(s["q"], s["T"], s["Hq"], c, s["table"], s["blocks"], s["cu"], s["kv_lens"], s["R"],
                          s["mask"], s["words"], s["window"], s["sinks"], s["scale"], s["out"], ws, lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_block(s):
    import mxfp4_packed_weight_amd as K
    c = _own_cache(s)
    ws = _own_workspace(s, lambda: K.k3_tree_attention_workspace_bytes(s["T"], s["Hq"], s["H"], s["D"]))
    K.k3_block_attention(s["q"], s["T"], s["Hq"], c, s["k_exp"], s["v_exp"], s["table"], s["blocks"], s["cu"],
                         s["kv_lens"], s["R"], s["window"], s["sinks"], s["scale"], s["out"], ws, lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    import mxfp4_packed_weight_amd as K
    K.k3_kv_append(s["k_in"], s["v_in"], s["T"], _own_cache(s), s["k_exp"], s["v_exp"], s["table"], s["blocks"],
                   s["cu"], s["kv_lens"], s["R"])
    return {"k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


def _own_logprobs(s):
    import mxfp4_packed_weight_amd as K
    ws = _own_workspace(s, lambda: K.k3_token_logprobs_workspace_bytes(s["T"], s["V"], s["k"]))
    K.k3_token_logprobs(s["logits"], s["T"], s["V"], s["beta"], s["tokens"], s["k"], s["logprob"], s["entropy"],
                        s["lse"], s["top"], s["top_logprob"], ws)
    return {k: s[k] for k in ("logprob", "entropy", "lse", "top", "top_logprob")}


def _plain_norm(s):
    T, N = s["T"], s["hidden"]
    h = s["x"].float() + s["residual"].float()
    s["sum"].copy_(h.to(s["sum"].dtype))
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["w"].float()
    if s["y"] is not None:
        s["y"].copy_(y.to(s["y"].dtype))
    if s["group"]:
        y = y.view(T, -1, s["group"])
        scale = y.abs().amax(-1, keepdim=True) / _E4M3_MAX
        s["scales"].copy_(scale.squeeze(-1))
        codes = (y / torch.where(scale > 0, scale, torch.ones_like(scale))).clamp(-_E4M3_MAX, _E4M3_MAX)
        s["y8"].copy_(codes.view(T, N).to(torch.float8_e4m3fn))
    return {"sum": s["sum"], "y": s["y"], "y8": s["y8"], "scales": s["scales"]}


def _raw(cache):
    return cache.view(torch.uint8 if cache.element_size() == 1 else torch.int16)


def _gathered(s, cache, page, at, scale, exps):
    """Rows of a cache at [R, L] places, [R, H, L, D] in 32 bits."""
    x = _raw(cache)[page, at].contiguous().view(cache.dtype).float().permute(0, 2, 1, 3)
    if scale is not None:
        x = x * scale[:, None, None]
    if exps is not None:
        x = x * _power(exps[page]).permute(0, 2, 1)[..., None]
    return x.contiguous()


def _plain_attention(s):
    R, T, H, D, P, n, L = s["R"], s["T"], s["H"], s["D"], s["P"], s["most"], s["longest"]
    G = s["Hq"] // H
    dev = s["q"].device
    cu, lens = s["cu"].long(), s["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[r]
    j = torch.arange(L, device=dev)
    there = j < lens[:, None]
    page = torch.where(there, s["table"].long()[:, j // P], torch.zeros_like(j))
    at = (j % P).expand(R, L)
    k = _gathered(s, s["k"], page, at, s["k_scale"], s["k_exp"])
    v = _gathered(s, s["v"], page, at, s["v_scale"], s["v_exp"])
    q = torch.zeros((R, n, H, G, D), device=dev)
    q[r, i] = s["q"].float().view(T, H, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(R, H, n * G, D)
    ctx = lens - new
    node = j - ctx[:, None]  # a key's place among the new ones, below zero for committed ones
    sees = torch.zeros((R, n, L), dtype=torch.bool, device=dev)
    if s["mask"] is None:
        rows, position = node[r] <= i[:, None], ctx[r] + i
    else:
        word = s["mask"].long().gather(1, (node[r] >> 5).clamp(0, s["words"] - 1))
        own_bits = there[r] & (node[r] >= 0) & (((word >> (node[r] & 31)) & 1) == 1)
        rows, position = (node[r] < 0) | own_bits, ctx[r] + own_bits.sum(1) - 1
    if s["window"]:
        near = (j < s["sinks"]) | (j > position[:, None] - s["window"])
        rows = rows & (near if s["mask"] is None else near | own_bits)
    sees[r, i] = rows
    sees = (sees & there[:, None]).repeat_interleave(G, 1)[:, None]
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    x = torch.where(sees, x, torch.full((), -math.inf, device=dev))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(-1)
    s["out"].copy_(o.view(R, H, n, G, D).permute(0, 2, 1, 3, 4)[r, i].reshape(T, s["Hq"], D).to(s["out"].dtype))
    s["lse"].copy_(lse.view(R, H, n, G).permute(0, 2, 1, 3)[r, i].reshape(T, s["Hq"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_append(s):
    """The new rows among the pages' earlier ones, in 32 bits, then every page that got any in 8 bits again."""
    T, H, D, P = s["T"], s["H"], s["D"], s["P"]
    cu, lens = s["cu"].long(), s["kv_lens"].long()
    t = torch.arange(T, device=cu.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    ctx = (lens - (cu[1:] - cu[:-1]))[r]
    place = ctx + t - cu[r]
    begins = (place == ctx) | (place % P == 0)  # the first new row of a page
    to = begins.long().cumsum(0) - 1            # the page's number among those that are written
    r, place0, ctx = r[begins], place[begins], ctx[begins]
    page = s["table"].long()[r, place0 // P]
    base = place0 // P * P
    slot = torch.arange(P, device=cu.device)
    old = (base[:, None] + slot < ctx[:, None])[..., None, None]  # rows that were there before
    new = torch.zeros((len(page), P), dtype=torch.bool, device=cu.device)
    new[to, place % P] = True
    new = new[..., None, None]
    for cache, exps, rows in ((s["k"], s["k_exp"], s["k_in"]), (s["v"], s["v_exp"], s["v_in"])):
        codes = _raw(cache)[page].contiguous()
        x = torch.zeros((len(page), P, H, D), device=cu.device)
        x[to, place % P] = rows.float().view(T, H, D)
        e = _exponents(x.abs().amax((1, 3)))
        was = exps[page]
        e = torch.where(base[:, None] < ctx[:, None], torch.maximum(e, was), e)
        x = torch.where(old, codes.view(cache.dtype).float() * _power(was)[:, None, :, None], x)
        x = (x / _power(e)[:, None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(cache.dtype)
        _raw(cache)[page] = torch.where(old | new, x.view(torch.uint8), codes)
        exps[page] = e
    return {"k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


def _plain_logprobs(s):
    T, V, k = s["T"], s["V"], s["k"]
    x = s["logits"].float()
    z = x * s["beta"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    p = e / total
    s["lse"].copy_(lse.squeeze(1))
    s["logprob"].copy_((z.gather(1, s["tokens"].long()[:, None]) - lse).squeeze(1))
    s["entropy"].copy_((torch.log(total) - torch.where(p > 0, p * (z - m), torch.zeros_like(p)).sum(1, keepdim=True))
                       .squeeze(1))
    at = torch.arange(V, device=x.device)
    left = x.clone() if k else None
    for i in range(k):  # the largest left, the first of its equals
        top = left.amax(1, keepdim=True)
        first = torch.where(left == top, at, V).amin(1, keepdim=True)
        s["top"][:, i] = first.squeeze(1).int()
        s["top_logprob"][:, i] = (z.gather(1, first) - lse).squeeze(1)
        left.scatter_(1, first, -math.inf)
    return {k: s[k] for k in ("logprob", "entropy", "lse", "top", "top_logprob")}


_PLAIN = {"norm": _plain_norm, "window": _plain_attention, "block": _plain_attention, "append": _plain_append,
          "logprobs": _plain_logprobs}
_OWN = {"norm": _own_norm, "window": _own_window, "block": _own_block, "append": _own_append,
        "logprobs": _own_logprobs}


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        T, N = case["T"], case["hidden"]
        out = 2 * case["y"] + (1 + 4 / case["group"] if case["group"] else 0)
        return {"bytes": int(T * N * (3 * 2 + out)) + 2 * N, "flops": 10 * T * N}
    if op == "logprobs":
        T, V = case["T"], case["V"]
        return {"bytes": T * V * _SIZE[case["dt"]] + T * (16 + 8 * case["k"]), "flops": 6 * T * V}
    ctx, new = _lengths(case)
    H, D, P, T = case["H"], case["D"], case["page"], sum(new)
    if op == "append":
        pages = sum((c + n - 1) // P - c // P + 1 for c, n in zip(ctx, new))
        return {"bytes": 2 * T * H * D * 3 + 4 * pages * H, "flops": 4 * T * H * D}
    Hq, window, sinks = H * case["G"], case["window"], case["sinks"]
    keys = pairs = 0
    for c, n in zip(ctx, new):
        gap = max(0, c - window + 1 - sinks) if window else 0  # between the sinks and the first row's window
        keys += c + n - gap
        last = [c + i for i in range(n)]
        if case.get("trees"):
            pairs += n * (c - gap + 1)
        else:
            pairs += sum(p + 1 - (max(0, p - window + 1 - sinks) if window else 0) for p in last)
    size = 1 if op == "block" else _SIZE[case["cache"]]
    return {"bytes": 2 * keys * H * D * size + T * Hq * (4 * D + 4) + 4 * keys // P
            + (2 * keys * H // P if op == "block" else 0), "flops": 4 * D * Hq * pairs}


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "window": _exact_attention, "block": _exact_attention, "append": _exact_append,
            "logprobs": _exact_logprobs}[s["op"]](s)


def _exact_norm(s):
    out = {k: [] for k in ("sum", "y", "y8", "scales")}
    for t in range(0, s["T"], 1024):
        h = s["x"][t:t + 1024].double() + s["residual"][t:t + 1024].double()
        y = h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / s["hidden"] + s["eps"]) * s["w"].double()
        out["sum"].append(h)
        out["y"].append(y)
        if s["group"]:
            y = y.unflatten(1, (-1, s["group"]))
            a = y.abs().amax(-1) / _E4M3_MAX
            out["scales"].append(a)
            out["y8"].append(torch.nan_to_num(y / a[..., None], nan=0.0).flatten(1))
    out = {k: torch.cat(v) if v else None for k, v in out.items()}
    return out if s["y"] is not None else out | {"y": None}


def _exact_rows(s, cache, scale, exps, r, L, h):
    """The first L rows of request r and key head h, [L, D] in 64 bits."""
    pages = s["table"][r, :-(-L // s["P"])].long()
    x = _raw(cache)[pages][:, :, h].contiguous().view(cache.dtype).double()
    if scale is not None:
        x = x * scale[h].double()
    if exps is not None:
        x = x * torch.exp2(exps[pages, h].double() - 127)[:, None, None]
    return x.flatten(0, 1)[:L]


def _exact_attention(s):
    H, G = s["H"], s["Hq"] // s["H"]
    cu, lens = s["cu"].tolist(), s["kv_lens"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    for r in range(s["R"]):
        n, L = cu[r + 1] - cu[r], lens[r]
        sees = np.ones((n, L), bool)
        if s["mask"] is None:
            sees[:, L - n:] = np.tril(np.ones((n, n), bool))
            position = np.arange(L - n, L)
        else:
            bits = np.unpackbits(s["mask"][cu[r]:cu[r + 1]].cpu().numpy().view(np.uint8), axis=1, bitorder="little")
            sees[:, L - n:] = bits[:, :n]
            position = L - n + bits[:, :n].sum(1, dtype=np.int64) - 1
        if s["window"]:
            for i in range(n):
                sees[i, s["sinks"]:max(s["sinks"], position[i] - s["window"] + 1)] = False
        hidden = torch.from_numpy(~sees).to(out.device)
        for h in range(H):
            k = _exact_rows(s, s["k"], s["k_scale"], s["k_exp"], r, L, h)
            v = _exact_rows(s, s["v"], s["v_scale"], s["v_exp"], r, L, h)
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][cu[r]:cu[r + 1], g].double() @ k.T) * s["scale"]
                x = x.masked_fill(hidden, -math.inf)
                lse[cu[r]:cu[r + 1], g] = torch.logsumexp(x, -1)
                out[cu[r]:cu[r + 1], g] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def _exact_append(s):
    """Codes and exponents request by request; codes of earlier rows have no value in 64 bits apart from theirs."""
    P, H, D = s["P"], s["H"], s["D"]
    cu, lens, table = (s[k].tolist() for k in ("cu", "kv_lens", "table"))
    out = {}
    for name in ("k", "v"):
        cache, exps = s[name].double(), s[name + "_exp"].cpu().numpy().astype(int)
        rows = s[name + "_in"].double().view(s["T"], H, D)
        sizes = rows.abs().amax(-1).cpu().numpy()
        for r in range(s["R"]):
            ctx = lens[r] - (cu[r + 1] - cu[r])
            for b in range(ctx // P, -(-lens[r] // P)):
                page, first, last = table[r][b], max(ctx, b * P), min(lens[r], b * P + P)
                t = cu[r] + first - ctx
                amax = sizes[t:t + last - first].max(0)
                e = np.array([127 + math.ceil(math.log2(a / 448)) if a else 1 for a in amax])
                if first > b * P:
                    e = np.maximum(e, exps[page])
                    fall = torch.tensor(2.0 ** (exps[page] - e), device=cache.device)
                    cache[page, :first - b * P] *= fall[:, None]
                exps[page] = e
                power = torch.tensor(2.0 ** (127.0 - e), device=cache.device)
                cache[page, first - b * P:last - b * P] = rows[t:t + last - first] * power[:, None]
        out[name], out[name + "_exp"] = cache, exps.astype(np.uint8)
    return out


def _exact_logprobs(s):
    T, k = s["T"], s["k"]
    tokens = s["tokens"].long()
    logprob, entropy, lse = (torch.zeros(T, dtype=torch.float64, device=tokens.device) for _ in range(3))
    top = np.zeros((T, k), np.int32)
    best = torch.zeros((T, k), dtype=torch.float64, device=tokens.device)
    for t in range(T):
        z = s["logits"][t].double() * s["beta"]
        z = z - torch.logsumexp(z, 0)
        lse[t] = torch.logsumexp(s["logits"][t].double() * s["beta"], 0)
        logprob[t] = z[tokens[t]]
        likely = z[z > -math.inf]
        entropy[t] = -(torch.exp(likely) * likely).sum()
        if k:
            value, at = torch.sort(s["logits"][t].double(), descending=True, stable=True)
            top[t], best[t] = at[:k].cpu().numpy(), z[at[:k]]
    return {"logprob": logprob, "entropy": entropy, "lse": lse, "top": top if k else None,
            "top_logprob": best if k else None}
