"""Plain references of the step's calls beside the cache in 64 bits, and the
bounds that the GPU's results are held to."""
import math

import numpy as np

U = 2.0 ** -24  # half a step of fp32
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4, "f32": U}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # a subnormal's step


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


# ---- norm ---------------------------------------------------------------------

def norm(x, residual, w, eps):
    """s and y in 64 bits on the CPU."""
    import torch
    s = x.cpu().double()
    if residual is not None:
        s = s + residual.cpu().double()
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * w.cpu().double()
    return s, y


# Relative error of y before its rounding: s has one rounding, each square two
# more and two of s; a sum of them passes at most 16 (a thread's) + 6 (lanes) +
# 15 (waves) additions, all of one sign; division, eps, rsqrt (at most 2 half
# steps each) and the products with w and r one each. Half of the squares'
# relative error goes on: (4 + 37 + 6) / 2 + 2 + 3 < 32.
NORM = 32 * U


def check_norm(out, s, y, kind, group):
    h, tiny = HALF_STEP[kind], TINY[kind]
    if out.get("sum") is not None:
        off = (out["sum"].cpu().double() - s).abs()
        assert (off <= (h + 2 * U) * s.abs() + tiny).all(), float((off / s.abs()).max())
    if out.get("y") is not None:
        off = (out["y"].cpu().double() - y).abs()
        assert (off <= (h + 2 * NORM) * y.abs() + tiny).all(), float((off / y.abs()).max())
    if out.get("y8") is not None:
        g = y.unflatten(1, (-1, group))
        want = g.abs().amax(-1) / 448
        got = out["scales"].cpu().double()
        assert got.shape == want.shape
        assert ((got - want).abs() <= (NORM + 3 * U) * want).all(), float(((got - want).abs() / want).max())
        codes = out["y8"].cpu().float().double().unflatten(1, (-1, group))
        # off by half a step of the code (subnormal ones are 2^-9 apart), and
        # y / scale, in three operations, by its own error
        off = (codes * got[..., None] - g).abs()
        lim = (HALF_STEP["e4m3"] + 4 * NORM) * g.abs() + 2.0 ** -10 * got[..., None]
        assert (off <= lim).all(), float((off / g.abs()).max())
        assert (codes.abs().amax(-1)[got > 0] == 448).all()


# ---- log probabilities ----------------------------------------------------------

def logprobs(logits, beta, tokens, k):
    """Rows one by one in 64 bits, on the CPU."""
    T, V = logits.shape
    x = logits.cpu().double().numpy()
    beta = float(np.float32(beta))
    out = {"logprob": np.full(T, -math.inf), "entropy": np.zeros(T), "lse": np.full(T, -math.inf),
           "top": np.full((T, k), -1), "top_logprob": np.full((T, k), math.nan)}
    for t in range(T):
        row, token = x[t], int(tokens[t])
        bad = np.isnan(row).any() or (row == math.inf).any()
        z = np.where(np.isnan(row), -math.inf, row) * beta
        z[np.isnan(z)] = -math.inf
        with np.errstate(all="ignore"):
            m = z.max()
            log_s = np.log(np.exp(z - m).sum()) if m > -math.inf and not bad else 0.0
            lse = m + log_s
            lp = (z - m) - log_s if m > -math.inf else np.full(V, -math.inf)  # (not z - lse: of the lowest numbers)
        if bad:
            out["lse"][t] = out["entropy"][t] = math.nan
            lp = np.full(V, math.nan)
        else:
            out["lse"][t] = lse
            some = lp > -math.inf
            out["entropy"][t] = -(np.exp(lp[some]) * lp[some]).sum()
        if 0 <= token < V:
            out["logprob"][t] = lp[token]
        order = np.argsort(-np.where(np.isnan(row), 0, row), kind="stable")
        order = [i for i in order if not np.isnan(row[i])][:k]
        out["top"][t, :len(order)] = order
        out["top_logprob"][t, :len(order)] = lp[order]
    return out


def check_logprobs(got, want, V):
    """Differences to the reference are off by U of theirs, and twice more by
    the factor (rounded itself); exponentials by a step. A sum over V values
    passes at most V / 256 + 16 additions of a lane (256 lanes at least have a
    row between them, each a run of 16 more than its share), 6 + 3 of lanes and
    waves and 2048 / 64 + 6 of parts. Where a distribution over V values has
    its differences' mean: at most log V + 1 <= 18 (weights above a share 1 /
    V e of the largest cannot be further)."""
    sums = (V / 256 + 64) * U + 2 * U + 4 * U * 18
    assert np.array_equal(got["top"], want["top"]), np.argwhere(got["top"] != want["top"])[:5]
    lim = {"logprob": lambda w: sums + 8 * U * (np.abs(w) + 18), "top_logprob": lambda w: sums + 8 * U * (np.abs(w) + 18),
           "lse": lambda w: sums + 8 * U * (np.abs(w) + 18), "entropy": lambda w: 2 * sums * (1 + 18)}
    for name, bound in lim.items():
        g, w = got[name].astype(np.float64), want[name]
        odd = ~np.isfinite(w)
        assert np.array_equal(g[odd], w[odd], equal_nan=True), (name, g[odd], w[odd])
        off = np.abs(g - w)[~odd]
        assert np.isfinite(g[~odd]).all() and (off <= bound(w[~odd])).all(), (name, off.max(), g, w)
