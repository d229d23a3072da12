"""A bound on the attention's error as a whole, beside the one for each element.

An output is the rounding of sum_i w_i (1 + d_i) v_i / sum_i w_i: each weight
and the output itself are rounded once to the rows' type, by at most half a
step h. Mantissas spread evenly over their logarithm make the root mean square
of such a rounding h / sqrt(3) * sqrt(3 / (8 ln 2)) = 0.425 h of the value.
Over values of zero mean the weights' roundings, which are independent, leave
0.425 h of the output's size as well, and the two together 0.60 h. Held to
0.75 h over all the rows that read one key head of a request (hundreds of
outputs, dozens of weights that count); the fp32 sums and exponentials are far
below. The elementwise bound counts every rounding at its worst and in one
direction, which over tens of thousands of places is a third of the output
itself: wrong values in a block of places, or one row of them misplaced, are
seen by this bound alone."""
import numpy as np

from tests import _kv as R_

PART = 0.75


def exact(s, k=None, v=None):
    """[T, Hq, D] in 64 bits, all rows of a key head at once; k, v: other
    contents of the cache."""
    import torch
    q, (kc, vc) = s["q"].cpu().double(), s["clean"]
    k, v = kc if k is None else k, vc if v is None else v
    (T, Hq, D), H, P = q.shape, s["H"], s["P"]
    G, out = Hq // H, torch.zeros(q.shape, dtype=torch.float64)
    for r, L in enumerate(np.asarray(s["lens"])):
        L, rows = int(L), slice(int(s["cu"][r]), int(s["cu"][r + 1]))
        n, p = rows.stop - rows.start, np.arange(int(L))
        page = s["table"][r][p // P]
        there = torch.from_numpy((page >= 0) & (page < s["pages"]))
        page, at = torch.from_numpy(np.where(there.numpy(), page, 0).astype(np.int64)), torch.from_numpy(p % P)
        vis = R_.sees(n, L, None if s["mask"] is None else np.ascontiguousarray(s["mask"][rows])) & there
        for h in range(H):
            K, V = k[page, at, h], v[page, at, h]
            if s["ks"] is not None:
                K, V = K * float(s["ks"][h]), V * float(s["vs"][h])
            x = (q[rows, h * G:(h + 1) * G].reshape(n * G, D) @ K.T).view(n, G, L) * s["scale"]
            x = x.masked_fill(~vis[:, None], -np.inf).softmax(-1)
            out[rows, h * G:(h + 1) * G] = (x.view(n * G, L) @ V).view(n, G, D)
    return out


def parts(got, want, s):
    """The error of each request's key heads, in half steps of the output's size."""
    H, e = s["H"], []
    G = want.shape[1] // H
    for r in range(len(s["lens"])):
        for h in range(H):
            at = slice(int(s["cu"][r]), int(s["cu"][r + 1])), slice(h * G, (h + 1) * G)
            e.append(float((got[at] - want[at]).norm() / want[at].norm()) / R_.HALF_STEP[s["dt"]])
    return e


def check(got, want, s):
    e = parts(got.cpu().double(), want, s)
    assert max(e) <= PART, [round(x, 3) for x in e]
    return max(e)
