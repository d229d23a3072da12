"""The paged key/value cache operators, as they are measured.

Four operators of one decoding step with drafted trees: the plan of the step
(block tables, slots, positions, tree masks), the query/key norm and rotation
with the append to the cache, the attention that reads the cache, and the
commit of the accepted path. Where ``own`` is false, ``run`` computes them in
elementary torch operations; where it is true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_E4M3_MAX = 448.0


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a small batch, one token each, no trees
        {"name": "plan_decode", "op": "plan", "R": 16, "ctx": 4096, "n": 1, "trees": False, "page": 16},
        # a full server: a thousand requests, each with a tree of up to 64 drafts
        {"name": "plan_trees", "op": "plan", "R": 1024, "ctx": 16384, "n": 64, "trees": True, "page": 16},
        # one token of one request: nothing but latency
        {"name": "qk_one", "op": "qk", "T": 1, "H": 8, "G": 8, "D": 128, "rot": 128, "inter": False,
         "dt": "bf16", "cache": "bf16", "page": 16, "pos": 4096},
        # the drafts of a batch, 8-bit cache, half of each head rotated in adjacent pairs
        {"name": "qk_drafts", "op": "qk", "T": 1000, "H": 4, "G": 8, "D": 128, "rot": 64, "inter": True,
         "dt": "bf16", "cache": "e4m3", "page": 64, "pos": 131072},
        # a long prompt
        {"name": "qk_prompt", "op": "qk", "T": 16384, "H": 8, "G": 8, "D": 128, "rot": 128, "inter": False,
         "dt": "bf16", "cache": "bf16", "page": 16, "pos": 32768},
        # one token of one request over a cache that ends inside a page
        {"name": "attn_one", "op": "attn", "R": 1, "ctx": 4096, "n": 1, "trees": False, "H": 8, "G": 8,
         "D": 128, "dt": "bf16", "cache": "bf16", "page": 16},
        # ordinary decoding: one token for each of 64 requests of ragged lengths
        {"name": "attn_decode", "op": "attn", "R": 64, "ctx": 8191, "n": 1, "trees": False, "H": 8, "G": 8,
         "D": 128, "dt": "bf16", "cache": "bf16", "page": 16},
        # verification of drafted trees of up to 64 nodes
        {"name": "attn_trees", "op": "attn", "R": 32, "ctx": 8000, "n": 64, "trees": True, "H": 8, "G": 8,
         "D": 128, "dt": "bf16", "cache": "bf16", "page": 16},
        # two long documents, trees of up to 32 nodes, 8-bit cache with large pages
        {"name": "attn_long_e4m3", "op": "attn", "R": 2, "ctx": 131000, "n": 32, "trees": True, "H": 8,
         "G": 8, "D": 128, "dt": "bf16", "cache": "e4m3", "page": 64},
        # two prompts' last chunks, a head of its own for each query head
        {"name": "attn_prompt_f16", "op": "attn", "R": 2, "ctx": 4000, "n": 2048, "trees": False, "H": 16,
         "G": 1, "D": 64, "dt": "f16", "cache": "f16", "page": 32},
        # a few requests of a shallow model
        {"name": "commit_few", "op": "commit", "R": 8, "layers": 4, "path": 3, "H": 4, "D": 128,
         "cache": "bf16", "page": 16, "ctx": 4096},
        # a batch through every layer of a deep model
        {"name": "commit_batch", "op": "commit", "R": 64, "layers": 48, "path": 6, "H": 8, "D": 128,
         "cache": "bf16", "page": 16, "ctx": 8192},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "qk", "attn", "attn", "commit"])
    page = rng.choice([16, 16, 24, 32, 64])
    if op == "plan":
        trees = rng.random() < 0.6
        return {"op": op, "R": _log(rng, 1, 1024), "ctx": _log(rng, 16, 16384), "n": _log(rng, 1, 64),
                "trees": trees, "page": page}
    if op == "qk":
        D = rng.choice([64, 128, 256])
        H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 5, 8])
        most = max(2, min(16384, 16384 * 80 * 128 // ((G + 2) * H * D)))
        dt = rng.choice(["bf16", "f16"])
        return {"op": op, "T": _log(rng, 1, most), "H": H, "G": G, "D": D,
                "rot": rng.choice([D, D, D // 2]), "inter": rng.random() < 0.4, "dt": dt,
                "cache": rng.choice([dt, "e4m3"]), "page": page, "pos": _log(rng, 16, 131072)}
    if op == "attn":
        kind = rng.choice(["one", "trees", "trees", "prompt"])
        D = rng.choice([64, 128, 128, 256])
        H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 5, 8])
        R = _log(rng, 1, {"one": 64, "trees": 32, "prompt": 2}[kind])
        scores = 2e8 * 128 / D / (R * H * G)  # of the padded batch, for each query head
        n = {"one": 1, "trees": _log(rng, 2, 64), "prompt": _log(rng, 65, max(66, min(2048, int(scores ** 0.5))))}[kind]
        most = max(16, min(int(scores / n), 131072, int(2.6e8 / (R * H * D))))
        dt = rng.choice(["bf16", "bf16", "f16"])
        return {"op": op, "R": R, "ctx": _log(rng, 16, most), "n": n, "trees": kind == "trees", "H": H, "G": G,
                "D": D, "dt": dt, "cache": rng.choice([dt, dt, "e4m3"]), "page": page}
    return {"op": op, "R": _log(rng, 1, 64), "layers": _log(rng, 1, 48), "path": rng.randint(1, 6),
            "H": rng.choice([1, 4, 8]), "D": rng.choice([64, 128]), "cache": rng.choice(["bf16", "f16", "e4m3"]),
            "page": page, "ctx": _log(rng, 16, 8192)}


# ---- inputs -------------------------------------------------------------------

def _lengths(case):
    """Committed and drafted lengths of a ragged batch: spread evenly, the last the longest."""
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


def _cache(shape, g, kind, scale):
    """Keys or values as a cache holds them, [pages, heads, page, D] in memory, seen as [pages, page, heads, D]."""
    pages, page, H, D = shape
    out = torch.empty((pages, H, page, D), dtype=_DT[kind], device=_DEV)
    for p in range(0, pages, 1024):  # in parts, for the random numbers' sake
        x = torch.randn(out[p:p + 1024].shape, generator=g, device=_DEV, dtype=torch.float32)
        if kind == "e4m3":
            x = (x / scale[:, None, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
        out[p:p + 1024] = x.to(out.dtype)
    return out.permute(0, 2, 1, 3)


def _scales(case, g):
    if case["cache"] != "e4m3":
        return None, None
    r = torch.rand((2, case["H"]), generator=g, device=_DEV, dtype=torch.float32)
    s = 0.01 + 0.01 * r
    return s[0].contiguous(), s[1].contiguous()


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    P = case["page"]

    if case["op"] == "plan":
        R = case["R"]
        ctx, new = (np.array(v) for v in _lengths(case))
        done = np.arange(R) % 8 == 7  # these requests have ended: their pages go back
        was = ctx + rs.randint(0, 2 * P, R)  # the step before may have held more
        was = np.where(rs.random_sample(R) < 0.5, ctx, was)
        held = -(-was // P)
        ctx, new = np.where(done, 0, ctx), np.where(done, 0, new)
        order = rs.permutation(R)
        blocks = -(-(case["ctx"] + max(case["n"], 2 * P)) // P) + 1
        n_pages = int((-(-(np.array(_lengths(case)[0]) + case["n"] + 2 * P) // P)).sum()) + R
        ctx, new, held = ctx[order], new[order], held[order]
        pages = rs.permutation(n_pages)
        table = np.full((R, blocks), -1)
        off = np.concatenate([[0], np.cumsum(held)])
        for r in range(R):
            table[r, :held[r]] = pages[off[r]:off[r + 1]]
        free = pages[off[R]:]
        ring = np.full(n_pages, -1)
        head = int(rs.randint(n_pages))
        ring[(head + np.arange(len(free))) % n_pages] = free
        T = int(new.sum())
        parents = np.concatenate([_tree(k, rs) for k in new]) if case["trees"] and T else None
        s |= {"R": R, "T": T, "P": P, "n_pages": n_pages, "blocks": blocks, "words": -(-case["n"] // 32),
              "most": case["n"], "ctx": _i32(ctx), "new": _i32(new), "held": _i32(held), "ring": _i32(ring),
              "ring_state": _i32([head, len(free)]), "table": _i32(table),
              "parents": None if parents is None else _i32(parents),
              "held_out": _i32(np.zeros(R)), "ring_out": _i32([0, 0]), "cu": _i32(np.zeros(R + 1)),
              "kv_lens": _i32(np.zeros(R)), "slots": _i32(np.zeros(T)), "positions": _i32(np.zeros(T)),
              "status": _i32([0, 0]),
              "mask": _i32(np.zeros((T, -(-case["n"] // 32)))) if parents is not None else None}
        return s

    H, D = case["H"], case["D"]
    ks, vs = _scales(case, g)
    s |= {"H": H, "D": D, "P": P, "k_scale": ks, "v_scale": vs}

    if case["op"] == "qk":
        T, Hq = case["T"], H * case["G"]
        dt = _DT[case["dt"]]
        n_pages = -(-T // P) * 5 // 4 + 1
        pages = rs.permutation(n_pages)
        at = np.arange(T) + int(rs.randint(P)) * (T % P != 0)
        slots = pages[(at // P) % n_pages] * P + at % P
        first = int(rs.randint(max(1, case["pos"] - T + 1)))
        half = case["rot"] // 2
        s |= {"T": T, "Hq": Hq, "dt": dt, "rot": case["rot"], "inter": case["inter"], "eps": 1e-6,
              "n_pages": n_pages, "qkv": (x := _normal((T, (Hq + 2 * H) * D), g, dt, 1.5)),
              "q_in": x[:, :Hq * D], "k_in": x[:, Hq * D:(Hq + H) * D], "v_in": x[:, (Hq + H) * D:],
              "wq": _normal((D,), g, torch.float32, 0.2).add(1).to(dt),
              "wk": _normal((D,), g, torch.float32, 0.2).add(1).to(dt),
              "inv_freq": torch.tensor(10000.0 ** (-np.arange(half) / half), dtype=torch.float32, device=_DEV),
              "positions": _i32(first + np.arange(T)), "slots": _i32(slots),
              "q_out": torch.zeros((T, Hq, D), dtype=dt, device=_DEV),
              "k": _cache((n_pages, P, H, D), g, case["cache"], ks),
              "v": _cache((n_pages, P, H, D), g, case["cache"], vs)}
        return s

    if case["op"] == "attn":
        R, Hq = case["R"], H * case["G"]
        ctx, new = (np.array(v) for v in _lengths(case))
        order = rs.permutation(R)
        ctx, new = ctx[order], new[order]
        lens = ctx + new
        T, blocks = int(new.sum()), int(-(-lens.max() // P))
        need = -(-lens // P)
        n_pages = int(need.sum()) + 1
        pages, off = rs.permutation(n_pages), np.concatenate([[0], np.cumsum(need)])
        table = np.full((R, blocks), -1)
        for r in range(R):
            table[r, :need[r]] = pages[off[r]:off[r + 1]]
        words, mask = -(-case["n"] // 32), None
        if case["trees"]:
            mask = np.zeros((T, words * 32), np.uint8)
            row = 0
            for k in new:
                p = _tree(k, rs)
                for i in range(k):
                    if i:
                        mask[row + i] = mask[row + p[i]]
                    mask[row + i, i] = 1
                row += k
            mask = np.packbits(mask, axis=1, bitorder="little").view(np.int32)
        s |= {"R": R, "T": T, "Hq": Hq, "n_pages": n_pages, "blocks": blocks, "most": case["n"],
              "longest": int(lens.max()), "words": words, "scale": D ** -0.5,
              "q": _normal((T, Hq * D), g, _DT[case["dt"]], 1.5).view(T, Hq, D),
              "k": _cache((n_pages, P, H, D), g, case["cache"], ks),
              "v": _cache((n_pages, P, H, D), g, case["cache"], vs), "table": _i32(table),
              "cu": _i32(np.concatenate([[0], np.cumsum(new)])), "kv_lens": _i32(lens),
              "mask": None if mask is None else _i32(mask),
              "out": torch.zeros((T, Hq, D), dtype=_DT[case["dt"]], device=_DEV),
              "lse": torch.zeros((T, Hq), dtype=torch.float32, device=_DEV)}
        return s

    # commit: every request drafted a root and `path` levels of `wide` nodes; the accepted nodes are
    # ones behind the first `path`, so that a second pass over the same state moves the same rows
    R, layers, path = case["R"], case["layers"], case["path"]
    wide = path + 2
    n = 1 + path * wide
    ctx = np.array([max(1, case["ctx"] * (r + 1) // R) for r in range(R)])[rs.permutation(R)]
    first, need = ctx // P, -(-(ctx + n) // P)
    n_pages = int((need - first).sum()) + 1
    pages, blocks, at = rs.permutation(n_pages), int(need.max()), 0
    table = np.full((R, blocks), -1)
    for r in range(R):
        table[r, first[r]:need[r]] = pages[at:at + need[r] - first[r]]
        at += need[r] - first[r]
    level = 1 + np.arange(path) * wide
    accepted = np.zeros((R, path + 1))
    accepted[:, 1:] = level + path + rs.randint(0, wide - path, (R, path))
    shape = (layers * n_pages, P, H, D)
    k, v = (_cache(shape, g, case["cache"], sc).unflatten(0, (layers, n_pages)) for sc in (ks, vs))
    s |= {"R": R, "layers": layers, "n_pages": n_pages, "blocks": blocks, "most": path + 1, "k": k, "v": v,
          "table": _i32(table), "ctx": _i32(ctx), "accepted": _i32(accepted),
          "n_accepted": _i32(1 + np.arange(R) % (path + 1)), "ctx_out": _i32(np.zeros(R))}
    return s


# ---- one pass -----------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_cache(s, k, v):
    """The cache's handle, made once as a program would."""
    import mxfp4_packed_weight_amd as K
    if "handle" not in s:
        s["handle"] = K.k3_kv_cache_of(k, v, s["k_scale"], s["v_scale"])
    return s["handle"]


def _own_plan(s):
    import mxfp4_packed_weight_amd as K
    K.k3_kv_plan(s["ctx"], s["new"], s["parents"], s["R"], s["T"], s["n_pages"], s["P"], s["blocks"], s["held"],
                 s["ring"], s["ring_state"], s["table"], s["held_out"], s["ring_out"], s["cu"], s["kv_lens"],
                 s["slots"], s["positions"], s["mask"], s["words"], s["status"])
    return _plan_outputs(s)


def _plan_outputs(s):
    return {k: s[k] for k in ("table", "ring", "held_out", "ring_out", "cu", "kv_lens", "slots", "positions",
                              "mask", "status")}


def _own_qk(s):
    import mxfp4_packed_weight_amd as K
    K.k3_qk_norm_rope(s["q_in"], s["k_in"], s["v_in"], s["T"], s["Hq"], s["wq"], s["wk"], s["eps"], s["inv_freq"],
                      s["rot"], s["inter"], s["positions"], s["q_out"], _own_cache(s, s["k"], s["v"]), s["slots"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_attn(s):
    import mxfp4_packed_weight_amd as K
    c = _own_cache(s, s["k"], s["v"])
    if "ws" not in s:
        s["ws"] = torch.empty(K.k3_tree_attention_workspace_bytes(s["T"], s["Hq"], s["H"], s["D"]),
                              dtype=torch.uint8, device=_DEV)
    K.k3_tree_attention(s["q"], s["T"], s["Hq"], c, s["table"], s["blocks"], s["cu"], s["kv_lens"], s["R"],
                        s["mask"], s["words"], s["scale"], s["out"], s["ws"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_commit(s):
    import mxfp4_packed_weight_amd as K
    K.k3_kv_commit(_own_cache(s, s["k"][0], s["v"][0]), s["layers"], s["k"].stride(0), s["table"], s["blocks"],
                   s["ctx"], s["accepted"], s["n_accepted"], s["most"], s["R"], s["ctx_out"])
    return {"k": s["k"], "v": s["v"], "ctx": s["ctx_out"]}


def _plain_plan(s):
    R, T, P, N = s["R"], s["T"], s["P"], s["n_pages"]
    dev = s["ctx"].device
    ctx, new, held = s["ctx"].long(), s["new"].long(), s["held"].long()
    head, count = s["ring_state"][0].long(), s["ring_state"][1].long()
    need = (ctx + new + P - 1) // P
    pops, push = (need - held).clamp(min=0), (held - need).clamp(min=0)
    before = pops.cumsum(0) - pops
    served = (pops == 0) | (before + pops <= count)
    taken = torch.where(served, pops, torch.zeros_like(pops))
    back = push.cumsum(0) - push
    col = torch.arange(s["blocks"], device=dev)
    old = s["table"].long()
    # pages taken from the ring's head, in the requests' order
    j = col[None] - held[:, None]
    take = (j >= 0) & (j < taken[:, None])
    popped = s["ring"].long()[(head + before[:, None] + j) % N]
    # pages given back at the ring's tail; where nothing is given back the value goes to a place past the end
    j = col[None] - need[:, None]
    give = (j >= 0) & (j < push[:, None])
    at = torch.where(give, (head + count + back[:, None] + j) % N, torch.full_like(j, N))
    longer = torch.cat([s["ring"], s["ring"].new_zeros(1)])
    longer[at.reshape(-1)] = s["table"].reshape(-1)
    s["ring"].copy_(longer[:N])
    s["table"].copy_(torch.where(take, popped, old))
    s["held_out"].copy_(torch.where(served, need, held))
    s["ring_out"].copy_(torch.stack([(head + taken.sum()) % N, count - taken.sum() + push.sum()]))
    s["cu"][1:] = new.cumsum(0)
    s["cu"][0] = 0
    s["kv_lens"].copy_(torch.where(served, ctx + new, torch.zeros_like(ctx)))
    s["status"].copy_(torch.stack([(~served).sum(), (new.sum() - T).clamp(min=0)]))
    if T:
        t = torch.arange(T, device=dev)
        r = torch.searchsorted(s["cu"][1:].long(), t, right=True)
        i = t - s["cu"].long()[r]
        p = ctx[r] + i
        slot = s["table"].long()[r, p // P] * P + p % P
        s["slots"].copy_(torch.where(served[r], slot, torch.full_like(slot, -1)))
        if s["parents"] is None:
            s["positions"].copy_(p)
        else:
            # who is whose ancestor: the one-step relation, squared until it reaches the root
            n = s["most"]
            sees = torch.eye(n, device=dev).repeat(R, 1, 1)
            up = s["parents"].long()
            sees[r, i, torch.where(up >= 0, up, i)] = 1
            for _ in range(max(1, (n - 1).bit_length())):
                sees = (sees @ sees).clamp(max=1)
            rows = sees[r, i]  # [T, n]
            s["positions"].copy_(ctx[r] + rows.sum(1).long() - 1)
            bits = torch.zeros((T, s["words"] * 32), dtype=torch.int64, device=dev)
            bits[:, :n] = rows.long()
            word = (bits.view(T, s["words"], 32) << torch.arange(32, device=dev)).sum(2)
            s["mask"].copy_(torch.where(word >= 2 ** 31, word - 2 ** 32, word))
    return _plan_outputs(s)


def _to_cache(cache, slots, x, scale):
    """Rows [T, H, D] in 32 bits into a cache, rounded once."""
    if scale is not None:
        x = (x / scale[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
    x = x.to(cache.dtype)
    P = cache.shape[1]
    raw = torch.uint8 if x.element_size() == 1 else torch.int16
    cache.view(raw)[slots // P, slots % P] = x.view(raw)


def _norm_rotate(x, w, s):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    rot, half = s["rot"], s["rot"] // 2
    if s["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_qk(s):
    T, Hq, H, D = s["T"], s["Hq"], s["H"], s["D"]
    x = s["qkv"].view(T, Hq + 2 * H, D)
    slots = s["slots"].long()
    s["q_out"].copy_(_norm_rotate(x[:, :Hq], s["wq"], s).to(s["dt"]))
    _to_cache(s["k"], slots, _norm_rotate(x[:, Hq:Hq + H], s["wk"], s), s["k_scale"])
    _to_cache(s["v"], slots, x[:, Hq + H:].float(), s["v_scale"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _gathered(cache, page, at, scale):
    """Rows of a cache at [R, L] places, [R, H, L, D] in 32 bits."""
    raw = cache.view(torch.uint8 if cache.element_size() == 1 else torch.int16)[page, at]
    x = raw.contiguous().view(cache.dtype).float().permute(0, 2, 1, 3)
    return (x if scale is None else x * scale[:, None, None]).contiguous()


def _plain_attn(s):
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
    k, v = _gathered(s["k"], page, at, s["k_scale"]), _gathered(s["v"], page, at, s["v_scale"])
    q = torch.zeros((R, n, H, G, D), device=dev)
    q[r, i] = s["q"].float().view(T, H, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(R, H, n * G, D)
    node = j - (lens - new)[:, None]  # a key's place among the drafted, below zero for committed ones
    sees = torch.zeros((R, n, L), dtype=torch.bool, device=dev)
    if s["mask"] is None:
        sees[r, i] = node[r] <= i[:, None]
    else:
        word = s["mask"].long().gather(1, (node[r] >> 5).clamp(0, s["words"] - 1))
        sees[r, i] = (node[r] < 0) | (((word >> (node[r] & 31)) & 1) == 1)
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


def _plain_commit(s):
    P, most = s["P"], s["most"]
    i = torch.arange(most, device=s["ctx"].device)
    take = i < s["n_accepted"].long()[:, None]
    src = s["ctx"].long()[:, None] + s["accepted"].long()
    dst = s["ctx"].long()[:, None] + i
    src = torch.where(take, src, dst)  # the others stay where they are
    table = s["table"].long()
    for x in (s["k"], s["v"]):
        x = x.view(torch.uint8 if x.element_size() == 1 else torch.int16)
        moved = x[:, table.gather(1, src // P), src % P]
        x[:, table.gather(1, dst // P), dst % P] = moved
    s["ctx_out"].copy_(s["ctx"] + s["n_accepted"])
    return {"k": s["k"], "v": s["v"], "ctx": s["ctx_out"]}


_PLAIN = {"plan": _plain_plan, "qk": _plain_qk, "attn": _plain_attn, "commit": _plain_commit}
_OWN = {"plan": _own_plan, "qk": _own_qk, "attn": _own_attn, "commit": _own_commit}


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    size = {"bf16": 2, "f16": 2, "e4m3": 1}
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        kept = [r for r in range(case["R"]) if r % 8 != 7]
        T = sum(new[r] for r in kept)
        words = -(-case["n"] // 32) if case["trees"] else 0
        # lengths and held pages in, lengths, held pages and prefix out; slots, positions and masks of
        # the tokens, their parents, and the table entries of the pages that they are in
        pages = sum(-(-new[r] // case["page"]) for r in kept)
        return {"bytes": 4 * (7 * case["R"] + T * (2 + words + (1 if words else 0)) + 2 * pages), "flops": 0}
    H, D = case["H"], case["D"]
    if case["op"] == "qk":
        T, Hq = case["T"], H * case["G"]
        return {"bytes": T * D * (2 * Hq * 2 + 2 * H * (2 + size[case["cache"]])) + 8 * T,
                "flops": T * D * (Hq + H) * 8}
    if case["op"] == "attn":
        ctx, new = _lengths(case)
        Hq, T = H * case["G"], sum(new)
        keys = sum(c + n for c, n in zip(ctx, new))
        pairs = sum(n * c + (n if case["trees"] else n * (n + 1) // 2) for c, n in zip(ctx, new))
        return {"bytes": 2 * keys * H * D * size[case["cache"]] + T * Hq * (4 * D + 4) + 4 * keys // case["page"],
                "flops": 4 * D * Hq * pairs}
    moved = sum(r % (case["path"] + 1) for r in range(case["R"]))
    return {"bytes": 4 * moved * H * D * size[case["cache"]] * case["layers"] + 8 * case["R"] + 8 * moved,
            "flops": 0}


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "qk": _exact_qk, "attn": _exact_attn, "commit": _exact_commit}[s["op"]](s)


def _exact_plan(s):
    """Request by request, as an allocator on the host would."""
    P, N = s["P"], s["n_pages"]
    ctx, new, held = (s[k].cpu().numpy().astype(int) for k in ("ctx", "new", "held"))
    ring, table = s["ring"].cpu().numpy().astype(int), s["table"].cpu().numpy().astype(int)
    head, count = s["ring_state"].cpu().tolist()
    parents = None if s["parents"] is None else s["parents"].cpu().numpy()
    out = {"held_out": held.copy(), "kv_lens": ctx + new, "cu": np.concatenate([[0], np.cumsum(new)]),
           "slots": np.full(s["T"], -1), "positions": np.zeros(s["T"], int)}
    mask = None if parents is None else np.zeros((s["T"], s["words"] * 32), np.uint8)
    wanted = taken = given = missed = 0
    for r in range(s["R"]):
        need = -(-(ctx[r] + new[r]) // P)
        fits = need <= held[r] or wanted + need - held[r] <= count
        wanted += max(0, need - held[r])
        if not fits:
            out["kv_lens"][r] = 0
            missed += 1
        else:
            for b in range(held[r], need):
                table[r, b] = ring[(head + taken) % N]
                taken += 1
            for b in range(need, held[r]):
                ring[(head + count + given) % N] = table[r, b]
                given += 1
            out["held_out"][r] = need
        for i in range(new[r]):
            t, p = out["cu"][r] + i, ctx[r] + i
            if fits:
                out["slots"][t] = table[r, p // P] * P + p % P
            depth = i
            if parents is not None:
                depth, a = 0, i
                mask[t, a] = 1
                while parents[out["cu"][r] + a] >= 0:
                    a = parents[out["cu"][r] + a]
                    mask[t, a] = 1
                    depth += 1
            out["positions"][t] = ctx[r] + depth
    out |= {"table": table, "ring": ring, "ring_out": np.array([(head + taken) % N, count - taken + given]),
            "status": np.array([missed, 0])}
    out["mask"] = None if mask is None else np.packbits(mask, axis=1, bitorder="little").view(np.int32)
    return {k: None if v is None else np.ascontiguousarray(v, dtype=np.int32) for k, v in out.items()}


def _exact_qk(s):
    T, Hq, H, D, P = s["T"], s["Hq"], s["H"], s["D"], s["P"]
    x = s["qkv"].double().view(T, -1, D)
    turn = s["positions"].double().view(T, 1) * s["inv_freq"].double().view(1, -1)
    if s["inter"]:
        one = torch.arange(0, s["rot"], 2, device=x.device)
        other = one + 1
    else:
        one = torch.arange(s["rot"] // 2, device=x.device)
        other = one + s["rot"] // 2

    def head(h, w):
        y = x[:, h]
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + s["eps"]) * w.double()
        z = y.clone()
        z[:, one] = y[:, one] * turn.cos() - y[:, other] * turn.sin()
        z[:, other] = y[:, one] * turn.sin() + y[:, other] * turn.cos()
        return z

    k, v = s["k"].double(), s["v"].double()
    page, at = s["slots"].long() // P, s["slots"].long() % P
    for h in range(H):
        a, b = head(Hq + h, s["wk"]), x[:, Hq + H + h]
        if s["k_scale"] is not None:
            a = (a / s["k_scale"][h].double()).clamp(-_E4M3_MAX, _E4M3_MAX)
            b = (b / s["v_scale"][h].double()).clamp(-_E4M3_MAX, _E4M3_MAX)
        k[page, at, h], v[page, at, h] = a, b
    return {"q": torch.stack([head(h, s["wq"]) for h in range(Hq)], 1), "k": k, "v": v}


def _pages(cache, pages, h):
    """The rows of one head in some pages, [rows, D] in 64 bits."""
    raw = cache.view(torch.uint8 if cache.element_size() == 1 else torch.int16)[pages][:, :, h]
    return raw.contiguous().view(cache.dtype).double().flatten(0, 1)


def _exact_attn(s):
    H, P, G = s["H"], s["P"], s["Hq"] // s["H"]
    cu, lens = s["cu"].tolist(), s["kv_lens"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    for r in range(s["R"]):
        n, L = cu[r + 1] - cu[r], lens[r]
        pages = s["table"][r, :-(-L // P)].long()
        sees = torch.ones((n, L), dtype=torch.bool, device=out.device)
        if s["mask"] is None:
            sees[:, L - n:] = torch.ones((n, n), dtype=torch.bool, device=out.device).tril()
        else:
            bits = np.unpackbits(s["mask"][cu[r]:cu[r + 1]].cpu().numpy().view(np.uint8), axis=1, bitorder="little")
            sees[:, L - n:] = torch.from_numpy(bits[:, :n].astype(bool)).to(out.device)
        for h in range(H):
            k, v = _pages(s["k"], pages, h)[:L], _pages(s["v"], pages, h)[:L]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][cu[r]:cu[r + 1], g].double() @ k.T) * s["scale"]
                x = x.masked_fill(~sees, -math.inf)
                lse[cu[r]:cu[r + 1], g] = torch.logsumexp(x, -1)
                out[cu[r]:cu[r + 1], g] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}


def _exact_commit(s):
    """Whole pages through the host, node by node."""
    P = s["P"]
    ctx, acc, num, table = (s[k].tolist() for k in ("ctx", "accepted", "n_accepted", "table"))
    k, v = s["k"].double(), s["v"].double()
    src, dst = [], []
    for r in range(s["R"]):
        for i in range(num[r]):
            a, b = ctx[r] + acc[r][i], ctx[r] + i
            src.append(table[r][a // P] * P + a % P)
            dst.append(table[r][b // P] * P + b % P)
    src, dst = (torch.tensor(x, device=k.device) for x in (src, dst))
    for x in (k, v):
        x[:, dst // P, dst % P] = x[:, src // P, src % P]
    return {"k": k, "v": v, "ctx": np.array([c + n for c, n in zip(ctx, num)], np.int32)}
