"""Plain references of the paged key/value cache calls (sequential integers,
64-bit floats), written from their definitions, and input makers."""
import math

import numpy as np

E4M3_MAX = 448.0
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[name]


def i32(a):
    import torch
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


def tree(n, rng):
    """Parents of a random tree, the root first."""
    return np.array([-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, n)], np.int32)[:n]


# ---- plan -----------------------------------------------------------------------

def plan(ctx, new, parents, T, n_pages, P, blocks, held, ring, state, table, words):
    """k3_kv_plan request by request."""
    R = len(ctx)
    ring, table = ring.copy(), table.copy()
    head, count = int(state[0]), min(max(int(state[1]), 0), n_pages)
    if not 0 <= head < n_pages:
        head = 0
    held_out, kv_lens = held.copy(), np.zeros(R, np.int64)
    cu = np.concatenate([[0], np.cumsum(np.maximum(new, 0).astype(np.int64))])
    wanted = given_want = taken = given = missed = 0
    old_ring, old_table = ring.copy(), table.copy()
    served = np.zeros(R, bool)
    for r in range(R):
        c, n, h = int(ctx[r]), int(new[r]), int(held[r])
        sound = c >= 0 and n >= 0 and c + n <= blocks * P and 0 <= h <= blocks
        sound = sound and not (parents is not None and n > 32 * words)
        need = -(-(c + n) // P) if sound else 0
        pops, push = (max(0, need - h), max(0, h - need)) if sound else (0, 0)
        ok = sound and (pops == 0 or wanted + pops <= count)
        ok = ok and (push == 0 or count + given_want + push <= n_pages)
        if ok:
            for j in range(pops):
                table[r, h + j] = old_ring[(head + wanted + j) % n_pages]
            for j in range(push):
                ring[(head + count + given_want + j) % n_pages] = old_table[r, need + j]
            taken, given = taken + pops, given + push
            held_out[r], kv_lens[r] = need, c + n
        else:
            missed += 1
        wanted, given_want = wanted + pops, given_want + push
        served[r] = ok
    slots, positions = np.full(T, -1, np.int64), np.zeros(T, np.int64)
    mask = np.zeros((T, 32 * words), np.uint8) if parents is not None else None
    for r in range(R):
        n = int(cu[r + 1] - cu[r])
        for i in range(n):
            t = int(cu[r]) + i
            if t >= T:
                break
            p = int(ctx[r]) + i
            if served[r]:
                page = int(table[r, p // P])
                if 0 <= page < n_pages:
                    slots[t] = page * P + p % P
            depth = i
            if parents is not None:
                depth = 0
                if n <= 32 * words:
                    a, depth = i, -1
                    while 0 <= a < n and not mask[t, a]:
                        mask[t, a] = 1
                        depth += 1
                        a = int(parents[cu[r] + a]) if cu[r] + a < T else -1
            positions[t] = min(int(ctx[r]) + depth, 2 ** 31 - 1)
    out = {"table": table, "ring": ring, "held_out": held_out, "kv_lens": kv_lens, "cu": cu,
           "ring_out": np.array([(head + taken) % n_pages, count - taken + given]), "slots": slots,
           "positions": positions, "status": np.array([missed, max(0, int(cu[R]) - T)])}
    if mask is not None:
        out["mask"] = np.packbits(mask, axis=1, bitorder="little").view(np.int32)
    return {k: np.asarray(v).astype(np.int32) for k, v in out.items()}


def pool(R, ctx, held, new, P, blocks, rng, spare):
    """A table, a ring and its state in which request r holds held[r] pages of its own."""
    need = np.maximum(held, 0)
    n_pages = int(need.sum()) + spare
    ids = rng.permutation(n_pages)
    table = np.full((R, blocks), -7, np.int32)
    at = 0
    for r in range(R):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    ring = np.full(n_pages, -9, np.int32)
    head = int(rng.integers(n_pages))
    ring[(head + np.arange(spare)) % n_pages] = ids[at:]
    return n_pages, table, ring, np.array([head, spare], np.int32)


# ---- cache ------------------------------------------------------------------------

def cache(pages, P, H, D, kind, g, order="heads first", scale=None, std=1.0):
    """[pages, P, H, D] keys or values on the GPU, in one of two memory orders."""
    import torch
    shape = (pages, H, P, D) if order == "heads first" else (pages, P, H, D)
    x = torch.randn(shape, generator=g, device="cuda") * std
    if kind == "e4m3":
        s = 1.0 if scale is None else (scale[:, None, None] if order == "heads first"
                                       else scale[:, None])
        x = (x / s).clamp(-E4M3_MAX, E4M3_MAX)
    x = x.to(torch_type(kind))
    return x.permute(0, 2, 1, 3) if order == "heads first" else x


def wide(x):
    """A cache or rows in 64 bits on the CPU."""
    return x.cpu().float().double()


# ---- norm, rotation ---------------------------------------------------------------

def norm_rotate(x, w, eps, inv_freq, rot, inter, positions):
    """[T, heads, D] in 64 bits."""
    import torch
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    a = (positions.double()[:, None] * inv_freq.double()[:rot // 2])[:, None]
    c, s = torch.cos(a), torch.sin(a)
    z = y.clone()
    i = torch.arange(rot // 2)
    one, other = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    z[..., one] = y[..., one] * c - y[..., other] * s
    z[..., other] = y[..., other] * c + y[..., one] * s
    return z


# ---- attention ----------------------------------------------------------------------

def sees(n, L, mask_rows):
    """[n, L] truth values."""
    import torch
    v = torch.ones((n, L), dtype=torch.bool)
    i, node = torch.arange(n)[:, None], torch.arange(L)[None] - (L - n)
    if mask_rows is None:
        return v & (node <= i)
    bits = torch.from_numpy(np.unpackbits(mask_rows.view(np.uint8), axis=1, bitorder="little").astype(bool))
    drafted = torch.zeros((n, L), dtype=torch.bool)
    ok = (node >= 0) & (node < bits.shape[1])
    drafted = torch.where(ok, bits.gather(1, node.clamp(0, bits.shape[1] - 1).expand(n, L)), drafted)
    return (node < 0) | drafted


def attention(q, k, v, table, cu, kv_lens, mask, scale, P, n_pages, k_scale=None, v_scale=None):
    """out, lse and the elementwise bound's parts: q [T, Hq, D], k and v
    [pages, P, H, D] in 64 bits on the CPU; the rest numpy. Places not seen
    are left out, not weighted with zero."""
    import torch
    T, Hq, D = q.shape
    H = k.shape[2]
    G = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mean_abs = torch.zeros_like(out)  # sum of weights times |v|
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    spread = torch.zeros(T, Hq, dtype=torch.float64)  # largest scale * sum |q k|
    most = torch.zeros(T, Hq, dtype=torch.float64)  # largest |v|
    for r in range(len(kv_lens)):
        n, L = int(cu[r + 1] - cu[r]), int(kv_lens[r])
        if n == 0 or L <= 0 or L > table.shape[1] * P:
            continue
        p = np.arange(L)
        page = table[r][p // P]
        there = torch.from_numpy((page >= 0) & (page < n_pages))
        page = torch.from_numpy(np.where(there.numpy(), page, 0).astype(np.int64))
        at = torch.from_numpy(p % P)
        rows = slice(int(cu[r]), int(cu[r + 1]))
        vis = sees(n, L, None if mask is None else np.ascontiguousarray(mask[rows])) & there
        for h in range(H):
            K, V = k[page, at, h], v[page, at, h]
            if k_scale is not None:
                K, V = K * float(k_scale[h]), V * float(v_scale[h])
            for i in range(n):
                s = vis[i].nonzero()[:, 0]
                if not len(s):
                    continue
                for hq in range(h * G, (h + 1) * G):
                    t = int(cu[r]) + i
                    x = (K[s] @ q[t, hq]) * scale
                    lse[t, hq] = torch.logsumexp(x, 0)
                    w = torch.softmax(x, 0)
                    out[t, hq] = w @ V[s]
                    mean_abs[t, hq] = w @ V[s].abs()
                    spread[t, hq] = (K[s].abs() @ q[t, hq].abs()).max() * abs(scale)
                    most[t, hq] = V[s].abs().max()
    return out, lse, mean_abs, spread, most


def check_attention(got, got_lse, ref, kind, keys):
    """The bound. A score is a sum of D <= 256 products in fp32 and one
    factor: off by at most (D + 2) 2^-24 of the sum of their sizes
    (`spread`), say e; a weight by the factor exp(2 e) (its own score's and
    the maximum's), 2^-21 for the exponential, and half a step of its type;
    the fp32 sum over `keys` places by 2^-24 sqrt-free worst keys * 2^-24;
    the output is rounded once more. fp16 weights are at least 2^6 at the
    largest and off by 2^-25 where they are subnormal."""
    import torch
    out, lse, mean_abs, spread, most = ref
    h = HALF_STEP[kind]
    e = (258 * 2.0 ** -24 * spread)[..., None]
    f = h + 2 * e + 2.0 ** -21 + keys * 2.0 ** -24
    small = keys * 2.0 ** -31 * most[..., None] if kind == "f16" else 0.0
    tiny = 2.0 ** -24 if kind == "f16" else 2.0 ** -126  # a subnormal's step
    bound = (1 + h) * (2 * f * mean_abs + small) + h * out.abs() + tiny
    got = got.cpu().double()
    off = (got - out).abs()
    bad = off > bound
    assert not bad.any() and not got.isnan().any(), (
        f"{int(bad.sum())} of {bad.numel()} past the bound, worst {float((off / bound).max()):.3g} of it")
    if got_lse is not None:
        g = got_lse.cpu().double()
        empty = lse == -math.inf
        assert torch.equal(g == -math.inf, empty)
        d = (g - lse)[~empty].abs()
        lim = (2 * e[..., 0] + 2.0 ** -21 + keys * 2.0 ** -24 + 2.0 ** -22 * lse.abs())[~empty]
        assert (d <= lim).all(), float((d / lim).max())
    return float((off / bound).max())
