"""Plain references of the windowed attention and of the cache with exponents,
in 64-bit floats and sequential integers, and their input makers. The bounds
are those of tests/_kv.py."""
import math

import numpy as np

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests.test_gpu_kv import attn_case


def case(ctx, new, H, G, D, dt, cache, P, seed, window, sinks, trees=False, **kw):
    """attn_case with a window; cache "blocks": e4m3 with an exponent for each page and head."""
    import torch
    s = attn_case(ctx, new, H, G, D, dt, "e4m3" if cache == "blocks" else cache, P, seed, trees=trees, **kw)
    s |= {"window": window, "sinks": sinks, "k_exp": None, "v_exp": None}
    if cache == "blocks":
        g = torch.Generator(device="cuda").manual_seed(seed)
        s["ks"] = s["vs"] = None
        for name, at in (("k", 0), ("v", 1)):
            e = torch.randint(119, 123, (s["pages"], H), generator=g, device="cuda")
            s[name + "_exp"] = e.to(torch.uint8)
        s["clean"] = tuple(R_.wide(s[n + "c"]) * torch.exp2(s[n + "_exp"].cpu().double() - 127)[:, None, :, None]
                           for n in "kv")
    return s


def call(s, q=None, out=None, lse=True, ws=None, stream=None):
    """The call that the case is for; out and lse."""
    import torch
    q = s["q"] if q is None else q
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda") if out is None else out
    l = torch.full((T, Hq), 7.0, device="cuda") if lse else None
    ws = ws if ws is not None else torch.full((K.k3_tree_attention_workspace_bytes(T, Hq, s["H"], D),), 0xff,
                                              dtype=torch.uint8, device="cuda")
    c = K.k3_kv_cache_of(s["kc"], s["vc"], s["ks"], s["vs"])
    mask = None if s["mask"] is None else R_.i32(s["mask"])
    rest = (R_.i32(s["table"]), s["table"].shape[1], R_.i32(s["cu"]), R_.i32(s["lens"]), len(s["lens"]))
    if s["k_exp"] is not None:
        K.k3_block_attention(q, T, Hq, c, s["k_exp"], s["v_exp"], *rest, s["window"], s["sinks"], s["scale"], out, ws,
                             lse=l, stream=stream)
    else:
        K.k3_window_attention(q, T, Hq, c, *rest, mask, s["words"], s["window"], s["sinks"], s["scale"], out, ws,
                              lse=l, stream=stream)
    return out, l


def run(s, **kw):
    import torch
    got = call(s, **kw)
    torch.cuda.synchronize()
    return got


def sees(s, r):
    """[n, L] truth values of request r."""
    import torch
    n, L = int(s["cu"][r + 1] - s["cu"][r]), int(s["lens"][r])
    rows = slice(int(s["cu"][r]), int(s["cu"][r + 1]))
    m = None if s["mask"] is None else np.ascontiguousarray(s["mask"][rows])
    vis = R_.sees(n, L, m)
    at = torch.arange(L - n, L)
    if m is not None:
        bits = np.unpackbits(m.view(np.uint8), axis=1, bitorder="little")[:, :n]
        at = L - n + torch.from_numpy(bits.sum(1, dtype=np.int64)) - 1
    p = torch.arange(L)
    if s["window"]:
        near = (p < s["sinks"]) | (p > at[:, None] - s["window"])
        if m is not None:  # a node's ancestors are at most `window` away
            near |= p >= L - n
        vis = vis & near
    page = torch.from_numpy(s["table"][r][np.arange(L) // s["P"]].astype(np.int64))
    return vis & (page >= 0) & (page < s["pages"])


def reference(s):
    """out, lse and the bound's parts, as tests/_kv.py has them."""
    import torch
    q, (kc, vc) = s["q"].cpu().double(), s["clean"]
    (T, Hq, D), H, P = q.shape, s["H"], s["P"]
    G = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mean_abs = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    spread, most = torch.zeros(T, Hq, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    for r, L in enumerate(np.asarray(s["lens"])):
        L, rows = int(L), slice(int(s["cu"][r]), int(s["cu"][r + 1]))
        n = rows.stop - rows.start
        if n == 0 or L <= 0 or L > s["table"].shape[1] * P:
            continue
        vis = sees(s, r)
        p = np.arange(L)
        page = s["table"][r][p // P]
        page = np.where((page >= 0) & (page < s["pages"]), page, 0).astype(np.int64)
        page, at = torch.from_numpy(page), torch.from_numpy(p % P)
        for h in range(H):
            k, v = kc[page, at, h], vc[page, at, h]
            if s["ks"] is not None:
                k, v = k * float(s["ks"][h]), v * float(s["vs"][h])
            hs = slice(h * G, (h + 1) * G)
            x = torch.einsum("ngd,ld->ngl", q[rows, hs], k) * s["scale"]
            x = x.masked_fill(~vis[:, None], -math.inf)
            lse[rows, hs] = torch.logsumexp(x, -1)
            w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
            out[rows, hs], mean_abs[rows, hs] = w @ v, w @ v.abs()
            size = torch.einsum("ngd,ld->ngl", q[rows, hs].abs(), k.abs()) * abs(s["scale"])
            spread[rows, hs] = size.masked_fill(~vis[:, None], 0).amax(-1)
            most[rows, hs] = torch.where(vis.any(1)[:, None], (v.abs().amax(-1) * vis).amax(-1)[:, None], 0)
    return out, lse, mean_abs, spread, most


def check(s):
    got, lse = run(s)
    worst = R_.check_attention(got, lse, reference(s), s["dt"], max(1, int(np.max(s["lens"]))))
    print(f"  worst at {worst:.3f} of the bound", flush=True)
    return got, lse


# ---- the append -------------------------------------------------------------------

def e4m3(x):
    """The nearest e4m3 value (ties to even) in 64 bits, saturated."""
    import torch
    return x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()


def exponent(amax):
    """The byte of the smallest 2^e with amax <= 448 2^e."""
    e = -126
    while amax > 448 * 2.0 ** e:
        e += 1
    return e + 127


def append(s):
    """k3_kv_append page by page: codes (64 bits on the CPU) and exponents of s's cache afterwards."""
    import torch
    T, H, D, P = s["T"], s["H"], s["D"], s["P"]
    out = {}
    for name in ("k", "v"):
        codes, exps = R_.wide(s[name + "c"]), s[name + "_exp"].cpu().numpy().astype(int)
        x = s[name + "_in"].cpu().float().double().reshape(s[name + "_in"].shape[0], -1)[:, :H * D].view(-1, H, D)
        for r in range(len(s["lens"])):
            t0, n, L = int(s["cu"][r]), int(s["cu"][r + 1] - s["cu"][r]), int(s["lens"][r])
            if t0 < 0 or n <= 0 or t0 + n > T or L < n or L > s["table"].shape[1] * P:
                continue
            ctx = L - n
            for b in range(ctx // P, (L - 1) // P + 1):
                page, first, last = int(s["table"][r, b]), max(ctx, b * P), min(L, b * P + P)
                if not 0 <= page < s["pages"]:
                    continue
                new = x[t0 + first - ctx:t0 + last - ctx]
                for h in range(H):
                    size = new[:, h].abs()
                    size = size[size < math.inf]
                    e = exponent(float(size.max()) if len(size) else 0.0)
                    if first > b * P:
                        was = min(max(int(exps[page, h]), 1), 254)
                        if e > was:
                            codes[page, :first - b * P, h] = e4m3(codes[page, :first - b * P, h] * 2.0 ** (was - e))
                        e = max(e, was)
                    exps[page, h] = e
                    y = new[:, h].clamp(-61440, 61440) if s["dt"] == "f16" else new[:, h]
                    codes[page, first - b * P:last - b * P, h] = e4m3(y * 2.0 ** (127 - e))
        out[name], out[name + "_exp"] = codes, exps
    return out
