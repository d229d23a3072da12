"""The paged key/value cache calls on the GPU against plain references in
sequential integers and 64-bit floats (tests/_kv.py)."""
import math

import numpy as np
import pytest

import mxfp4_packed_weight_amd as K
from tests import _kv as R_
from tests._gpu import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ptr_aligned(n, dtype):
    import torch
    return torch.empty(n, dtype=dtype, device="cuda")


# ---- plan -------------------------------------------------------------------------

def run_plan(ctx, new, parents, T, n_pages, P, blocks, held, ring, state, table, words):
    import torch
    i32 = R_.i32
    R = len(ctx)
    junk = lambda *s: torch.full(s, -12345, dtype=torch.int32, device="cuda")  # noqa: E731
    o = {"table": i32(table), "ring": i32(ring), "held_out": junk(R), "ring_out": junk(2), "cu": junk(R + 1),
         "kv_lens": junk(R), "slots": junk(T), "positions": junk(T), "status": junk(2)}
    if parents is not None:
        o["mask"] = junk(T, words)
    K.k3_kv_plan(i32(ctx), i32(new), None if parents is None else i32(parents), R, T, n_pages, P, blocks,
                 i32(held), o["ring"], i32(state), o["table"], o["held_out"], o["ring_out"], o["cu"],
                 o["kv_lens"], o["slots"], o["positions"], o.get("mask"), words, o["status"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in o.items()}


def same_plan(*args):
    got, want = run_plan(*args), R_.plan(*args)
    assert got.keys() == want.keys()
    for k in want:
        bad = np.argwhere(np.atleast_1d(got[k] != want[k]))
        assert not len(bad), (k, bad[:5].tolist(), got[k].reshape(-1)[:8], want[k].reshape(-1)[:8])
    return want


def plan_case(R, ctx_max, n_max, trees, P, seed, spare=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_max + 1, R)
    new = rng.integers(0, n_max + 1, R)
    done = rng.random(R) < 0.15
    ctx, new = np.where(done, 0, ctx), np.where(done, 0, new)
    held = np.maximum(0, -(-ctx // P) + rng.integers(-1, 4, R))
    blocks = -(-(ctx_max + n_max) // P) + 4
    want = int(np.maximum(0, -(-(ctx + new) // P) - held).sum())
    n_pages, table, ring, state = R_.pool(R, ctx, held, new, P, blocks, rng, want if spare is None else spare)
    parents = np.concatenate([R_.tree(int(n), rng) for n in new]) if trees else None
    if n_pages < 1:
        n_pages, ring = 1, np.zeros(1, np.int32)
    return [ctx, new, parents, int(new.sum()), n_pages, P, blocks, held, ring, state, table,
            max(1, -(-n_max // 32))]


@pytest.mark.parametrize("R,ctx,n,trees,P", [
    (1, 0, 1, False, 16), (1, 100, 1, True, 1), (16, 500, 1, False, 16), (37, 300, 7, True, 24),
    (64, 200, 32, True, 16), (130, 100, 64, True, 8), (33, 200, 200, True, 7), (5, 50, 1024, True, 16),
    (3, 4000, 3000, False, 64), (1024, 90, 3, False, 16), (1025, 60, 5, True, 16), (4096, 40, 2, True, 16)])
def test_plan(R, ctx, n, trees, P):
    say(f"plan R={R} ctx={ctx} n={n} trees={trees} P={P}")
    c = plan_case(R, ctx, n, trees, P, R + n)
    if c[3] == 0:
        c[1] = c[1] + 1
        c[3] = R
        c[2] = np.full(R, -1) if trees else None
    same_plan(*c)


@pytest.mark.parametrize("spare", [0, 1, 7, 20])
def test_plan_out_of_pages(spare):
    """Requests past the free pages are not served; those that need none are."""
    say(f"plan with {spare} free pages")
    want = same_plan(*plan_case(60, 300, 20, True, 16, 5, spare))
    assert 0 < want["status"][0] < 60


def test_plan_unsound_requests():
    """Lengths, held pages and node counts out of range, and a ring that
    would overflow: not served, and the others as without them."""
    say("plan with unsound requests")
    c = plan_case(40, 200, 40, True, 16, 8, 60)
    ctx, new, held, blocks = c[0], c[1], c[7], c[6]
    ctx[3], ctx[5], held[7], held[9] = -4, 1 << 30, -2, blocks + 1
    ctx[11] = 2 ** 31 - 1
    ctx[13] = blocks * 16 - int(new[13]) + 1
    words = c[11] = 1  # some requests have more than 32 nodes
    assert (new > 32 * words).any()
    want = same_plan(*c)
    assert want["status"][0] >= 6
    c[1][15] = -3
    c[3] = int(np.maximum(c[1], 0).sum())
    c[2] = np.concatenate([R_.tree(max(0, int(n)), np.random.default_rng(1)) for n in c[1]])
    same_plan(*c)
    # a ring that says it is full has no room for what comes back
    c = plan_case(20, 100, 3, False, 16, 9)
    c[9] = np.array([3, c[4]], np.int32)
    assert same_plan(*c)["status"][0] > 0


@pytest.mark.parametrize("head,count", [(-5, 3), (10 ** 6, 4), (0, -2), (2, 10 ** 9)])
def test_plan_unsound_ring_state(head, count):
    """A head outside the ring counts as 0, a count is held to the ring's size."""
    say(f"plan with ring state {head}, {count}")
    c = plan_case(6, 60, 2, False, 16, 4)
    c[9] = np.array([head, count], np.int32)
    same_plan(*c)


@pytest.mark.parametrize("off", [-9, -1, 1, 3000])
def test_plan_token_count(off):
    """T is the caller's: a padded step fills the rest, a short one says how many are missing."""
    say(f"plan with T off by {off}")
    c = plan_case(20, 100, 30, True, 16, 11)
    T = c[3]
    c[3] = T + off
    c[2] = np.concatenate([c[2], np.full(max(off, 0), -1)])[:c[3]]
    want = same_plan(*c)
    assert want["status"][1] == max(0, -off)


def test_plan_without_tokens():
    """All requests have ended: T = 0, every page goes back."""
    import torch
    say("plan T=0")
    c = plan_case(9, 100, 5, False, 16, 12)
    c[0], c[1], c[3] = np.zeros(9, np.int64), np.zeros(9, np.int64), 0
    want = same_plan(*c)
    assert not want["held_out"].any() and want["ring_out"][1] == c[4]
    i32 = R_.i32
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (9, 2, 10, 9, 2)]
    K.k3_kv_plan(i32(c[0]), i32(c[1]), None, 9, 0, c[4], 16, c[6], i32(c[7]), i32(c[8]), i32(c[9]), i32(c[10]),
                 out[0], out[1], out[2], out[3], None, None, None, 0, out[4])
    torch.cuda.synchronize()
    assert out[1].cpu().tolist() == want["ring_out"].tolist()


@pytest.mark.parametrize("n", [5, 64, 300])
def test_plan_parents_in_any_order(n):
    """A parent may come after its child; indices outside the request end the walk; so does a cycle."""
    say(f"plan with {n} shuffled parents")
    rng = np.random.default_rng(n)
    p = R_.tree(n, rng)
    order = rng.permutation(n)
    shuffled = np.full(n, -1)
    for i in range(n):
        shuffled[order[i]] = order[p[i]] if p[i] >= 0 else -1
    wild = shuffled.copy()
    wild[rng.integers(0, n, 2)] = [n + 3, -7]
    loop = shuffled.copy()
    loop[order[0]] = order[n - 1]
    loop2 = np.arange(n)  # each its own parent
    for parents in (shuffled, wild, loop, loop2):
        c = [np.array([30, 4]), np.array([2, n]), np.concatenate([[-1, 0], parents]), n + 2, 64, 16, 40,
             np.array([2, 1]), np.arange(64), np.array([0, 60]), np.zeros((2, 40), np.int64), max(1, -(-n // 32))]
        same_plan(*c)


def test_plan_page_ids_out_of_range():
    """Slots of places in a page that does not exist are -1."""
    say("plan with bad page ids")
    c = plan_case(8, 100, 10, False, 16, 21)
    c[10][:, :3] = [[-1, 10 ** 6, 2 ** 31 - 1]]
    want = same_plan(*c)
    assert (want["slots"] == -1).any()


# ---- norm, rotation, append ---------------------------------------------------------

def qk_case(T, H, G, D, rot, inter, dt, cache, P, seed, order="heads first", gap=0, first=1000, wide_rows=True):
    import torch
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    Hq, t16 = H * G, R_.torch_type(dt)
    cols = (Hq + 2 * H) * D + gap
    x = (torch.randn((T, cols), generator=g, device="cuda") * 1.5).to(t16)
    pages = -(-T // P) + 3
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (0.01 + 0.02 * torch.rand((2, H), generator=g, device="cuda")).unbind(0)
        ks, vs = ks.contiguous(), vs.contiguous()
    return {"x": x, "q": x[:, :Hq * D], "k": x[:, Hq * D:(Hq + H) * D], "v": x[:, (Hq + H) * D:(Hq + 2 * H) * D],
            "T": T, "Hq": Hq, "H": H, "D": D, "P": P, "pages": pages, "dt": dt, "cache": cache, "ks": ks, "vs": vs,
            "wq": (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(t16),
            "wk": (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(t16), "eps": 1e-6,
            "freq": torch.tensor(10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2)), dtype=torch.float32,
                                 device="cuda"), "rot": rot, "inter": inter,
            "pos": rng.integers(0, first, T), "slots": rng.permutation(pages * P)[:T],
            "out": torch.full((T, Hq, D), 7.0, dtype=t16, device="cuda"),
            "kc": R_.cache(pages, P, H, D, cache, g, order, ks), "vc": R_.cache(pages, P, H, D, cache, g, order, vs)}


def check_qk(s):
    """The norm sums D <= 256 squares and the rest is a handful of fp32
    steps: off by at most (D + 16) 2^-24 of the sizes that are added, the
    angle (64-bit) by nothing beside it; then one rounding."""
    import torch
    T, Hq, H, D, P = s["T"], s["Hq"], s["H"], s["D"], s["P"]
    before = R_.wide(s["kc"]), R_.wide(s["vc"])
    c = K.k3_kv_cache_of(s["kc"], s["vc"], s["ks"], s["vs"])
    slots, pos = R_.i32(s["slots"]), R_.i32(s["pos"])
    K.k3_qk_norm_rope(s["q"], s["k"], s["v"], T, Hq, s["wq"], s["wk"], s["eps"], s["freq"] if s["rot"] else None,
                      s["rot"], s["inter"], pos, s["out"], c, slots)
    torch.cuda.synchronize()
    p = torch.tensor(np.asarray(s["pos"], np.int64))
    f = s["freq"].cpu()

    def turned(x, w):
        x = x.cpu().double().reshape(T, -1, D)
        y = R_.norm_rotate(x, w.cpu().double(), s["eps"], f, s["rot"], s["inter"], p)
        size = R_.norm_rotate(x.abs(), w.cpu().double().abs(), s["eps"], f, 0, False, p)
        return y, size.amax(-1, keepdim=True) * 2  # a pair's sum is at most this

    def near(got, want, size, kind, what):
        h = R_.HALF_STEP[kind]
        tiny = {"bf16": 2.0 ** -126, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}[kind]
        e = (D + 16) * 2.0 ** -24 * size
        bound = (1 + h) * e + h * want.abs() + tiny
        off = (got - want).abs()
        bad = ~(off <= bound)
        assert not bad.any(), (what, int(bad.sum()), float((off / bound).max()))

    want, size = turned(s["q"], s["wq"])
    near(s["out"].cpu().double(), want, size, s["dt"], "q")
    k, ksize = turned(s["k"], s["wk"])
    v = s["v"].cpu().double().reshape(T, H, D)
    for name, cache, old, rows, size, scale in (("k", s["kc"], before[0], k, ksize, s["ks"]),
                                               ("v", s["vc"], before[1], v, v.abs() * 0, s["vs"])):
        new = R_.wide(cache)
        ok = [(t, int(x)) for t, x in enumerate(s["slots"]) if 0 <= x < s["pages"] * P]
        t = torch.tensor([a for a, _ in ok], dtype=torch.long)
        at = torch.tensor([b for _, b in ok], dtype=torch.long)
        got = new[at // P, at % P]
        rows, size = rows[t], size[t]
        if scale is not None:
            sc = scale.cpu().double()[:, None]
            rows, size = rows / sc, size / sc
            size = size + rows.abs()  # the division
            low = rows.clamp(-448, 448)
            near(got, low, size, "e4m3", name)
        else:
            near(got, rows, size, s["cache"], name)
        new[at // P, at % P] = old[at // P, at % P]
        assert torch.equal(new.nan_to_num(1e9), old.nan_to_num(1e9)), f"{name}: other rows were written"


@pytest.mark.parametrize("T,H,G,D,rot,inter,dt,cache,P", [
    (1, 8, 8, 128, 128, False, "bf16", "bf16", 16), (1, 1, 1, 64, 64, True, "f16", "f16", 1),
    (3, 2, 5, 64, 32, False, "f16", "e4m3", 24), (7, 4, 4, 128, 64, True, "bf16", "e4m3", 64),
    (65, 8, 1, 256, 256, False, "bf16", "bf16", 7), (33, 1, 8, 256, 128, True, "f16", "f16", 32),
    (130, 4, 8, 128, 16, False, "bf16", "bf16", 16), (50, 2, 4, 128, 0, False, "f16", "f16", 16),
    (2000, 8, 2, 64, 64, False, "bf16", "e4m3", 16), (5000, 1, 1, 128, 112, False, "bf16", "bf16", 16),
    (300, 3, 3, 256, 240, True, "bf16", "e4m3", 16)])
def test_qk(T, H, G, D, rot, inter, dt, cache, P):
    say(f"qk T={T} H={H} G={G} D={D} rot={rot} inter={inter} {dt} {cache} P={P}")
    for order, gap in (("heads first", 0), ("slots first", 24)):
        check_qk(qk_case(T, H, G, D, rot, inter, dt, cache, P, T + D, order, gap))


def test_qk_slots_out_of_range():
    """Rows without a slot are not written, their queries are."""
    say("qk with slots out of range")
    s = qk_case(40, 2, 4, 128, 128, False, "bf16", "bf16", 16, 3)
    s["slots"][[0, 7, 20, 39]] = [-1, s["pages"] * 16, 2 ** 31 - 1, -(2 ** 31)]
    check_qk(s)


def test_qk_far_positions():
    """Positions up to 2^31 - 1, and below zero: the angle's fraction counts."""
    say("qk at far positions")
    s = qk_case(64, 2, 2, 128, 128, False, "f16", "f16", 16, 4, first=2 ** 31 - 1)
    s["pos"][:3] = [2 ** 31 - 1, -(2 ** 31), -5]
    check_qk(s)


def test_qk_rows_of_zeros_and_large_values():
    """A row of zeros stays zero; e4m3 saturates; rows of equal large values are normed."""
    import torch
    say("qk with extreme rows")
    s = qk_case(8, 2, 2, 128, 128, True, "bf16", "e4m3", 16, 5)
    s["x"][0] = 0
    s["x"][1] = 2.0 ** 40
    s["x"][2] = -1e30 * torch.sign(s["x"][2])
    s["x"][3] *= 1e-20
    s["v"][4] = 3e38
    # 1e30 squared is past fp32, the norm of it is 0 (as the definition has in fp32): keep it off
    s["x"][2] = s["x"][5]
    check_qk(s)


def test_qk_not_finite_rows_keep_to_themselves():
    """NaN and infinities in one head leave the other heads and tokens alone; in the values they go through."""
    import torch
    say("qk with NaN")
    s = qk_case(9, 2, 3, 64, 32, False, "bf16", "bf16", 16, 6)
    clean = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in s.items()}
    s["q"][4, 64] = float("nan")  # token 4, head 1
    s["k"][2, 3] = float("inf")   # token 2, head 0
    s["v"][5, 64 + 7] = float("nan")
    for c in (clean, s):
        if c is clean:
            x = c["x"]
            Hq, H, D = c["Hq"], c["H"], c["D"]
            c["q"], c["k"], c["v"] = x[:, :Hq * D], x[:, Hq * D:(Hq + H) * D], x[:, (Hq + H) * D:(Hq + 2 * H) * D]
        K.k3_qk_norm_rope(c["q"], c["k"], c["v"], 9, c["Hq"], c["wq"], c["wk"], c["eps"], c["freq"], c["rot"],
                          False, R_.i32(c["pos"]), c["out"], K.k3_kv_cache_of(c["kc"], c["vc"]), R_.i32(c["slots"]))
    torch.cuda.synchronize()
    differ = (s["out"] != clean["out"]).any(-1).nonzero().tolist()
    assert differ == [[4, 1]] and s["out"][4, 1].isnan().any()
    at = int(s["slots"][2])
    dk = (s["kc"] != clean["kc"]).any(-1).nonzero().tolist()
    assert dk == [[at // 16, at % 16, 0]]
    at = int(s["slots"][5])
    assert s["vc"][at // 16, at % 16, 1].isnan().nonzero().tolist() == [[7]]


# ---- attention ----------------------------------------------------------------------

def attn_case(ctx, new, H, G, D, dt, cache, P, seed, trees=True, order="heads first", words=None, q_std=1.5,
              bad_pages=0, spare=2):
    import torch
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx), np.asarray(new)
    lens = ctx + new
    T, R, Hq = int(new.sum()), len(ctx), H * G
    need = -(-lens // P)
    pages = int(need.sum()) + spare
    ids, off = rng.permutation(pages), np.concatenate([[0], np.cumsum(need)])
    blocks = max(1, int(need.max()) + 1)
    table = np.full((R, blocks), -1)
    for r in range(R):
        table[r, :need[r]] = ids[off[r]:off[r + 1]]
    for b in range(bad_pages):
        r = b % R
        table[r, int(rng.integers(max(1, need[r])))] = [-1, pages, 2 ** 31 - 1, -2 ** 31][b % 4]
    mask = None
    if trees:
        words = words or max(1, -(-int(new.max()) // 32))
        bits = np.zeros((T, 32 * words), np.uint8)
        row = 0
        for n in new:
            p = R_.tree(int(n), rng)
            for i in range(int(n)):
                if i:
                    bits[row + i] = bits[row + p[i]]
                if i < 32 * words:
                    bits[row + i, i] = 1
            row += int(n)
        mask = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (0.01 + 0.02 * torch.rand((2, H), generator=g, device="cuda")).unbind(0)
        ks, vs = ks.contiguous(), vs.contiguous()
    kc, vc = (R_.cache(pages, P, H, D, cache, g, order, s) for s in (ks, vs))
    return {"q": (torch.randn((T, Hq, D), generator=g, device="cuda") * q_std).to(R_.torch_type(dt)), "kc": kc,
            "vc": vc, "ks": ks, "vs": vs, "table": table, "cu": np.concatenate([[0], np.cumsum(new)]), "lens": lens,
            "mask": mask, "words": words or 1, "scale": D ** -0.5, "P": P, "pages": pages, "H": H, "dt": dt,
            "clean": (R_.wide(kc), R_.wide(vc))}


def run_attn(s, lse=True, stream=None, out=None, ws=None):
    import torch
    T, Hq, D = s["q"].shape
    out = torch.full((T, Hq, D), 7.0, dtype=s["q"].dtype, device="cuda") if out is None else out
    l = torch.full((T, Hq), 7.0, device="cuda") if lse else None
    ws = ws if ws is not None else torch.full((K.k3_tree_attention_workspace_bytes(T, Hq, s["H"], D),), 0xff,
                                              dtype=torch.uint8, device="cuda")
    c = K.k3_kv_cache_of(s["kc"], s["vc"], s["ks"], s["vs"])
    mask = None if s["mask"] is None else R_.i32(s["mask"])
    K.k3_tree_attention(s["q"], T, Hq, c, R_.i32(s["table"]), s["table"].shape[1], R_.i32(s["cu"]),
                        R_.i32(s["lens"]), len(s["lens"]), mask, s["words"], s["scale"], out, ws, lse=l,
                        stream=stream)
    torch.cuda.synchronize()
    return out, l


def reference(s):
    k, v = s["clean"]
    f = lambda x: None if x is None else x.cpu().double()  # noqa: E731
    return R_.attention(s["q"].cpu().double(), k, v, s["table"], s["cu"], s["lens"], s["mask"], s["scale"], s["P"],
                        s["pages"], f(s["ks"]), f(s["vs"]))


def check_attn(s):
    got, lse = run_attn(s)
    worst = R_.check_attention(got, lse, reference(s), s["dt"], max(1, int(np.max(s["lens"]))))
    say(f"  worst at {worst:.3f} of the bound")
    return got, lse


RAGGED = ([0, 1, 15, 16, 17, 31, 100, 257], [1, 1, 1, 1, 1, 1, 1, 1])
TREES = ([0, 1, 30, 127, 128, 500, 64, 3], [1, 2, 3, 33, 5, 64, 32, 17])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("lens,H,G,P", [(RAGGED, 2, 8, 16), (RAGGED, 3, 5, 7), (RAGGED, 1, 1, 24),
                                        (TREES, 2, 4, 16), (TREES, 1, 5, 24)])
def test_attention(D, dt, cache, lens, H, G, P):
    say(f"attention D={D} {dt} {cache} lens={lens} H={H} G={G} P={P}")
    order = "slots first" if P == 7 else "heads first"
    check_attn(attn_case(*lens, H, G, D, dt, cache, P, D + G, order=order))


@pytest.mark.parametrize("ctx,new,H,G,D,P", [
    ([5000], [1], 1, 8, 128, 16), ([20000], [2], 1, 4, 64, 32), ([4096], [1], 2, 1, 256, 64),
    ([3001, 7, 12000], [1, 1, 1], 2, 2, 128, 24), ([9000, 2], [24, 30], 1, 4, 128, 16),
    ([6000], [64], 1, 8, 128, 16)])
def test_attention_split(ctx, new, H, G, D, P):
    """Long rows, shared out to many workgroups and joined."""
    say(f"attention split ctx={ctx} new={new} H={H} G={G} D={D}")
    check_attn(attn_case(ctx, new, H, G, D, "bf16", "bf16", P, D + G))


@pytest.mark.parametrize("ctx,new,H,G,D,dt,cache", [
    ([0], [200], 2, 1, 64, "f16", "f16"), ([77, 0], [130, 65], 1, 3, 128, "bf16", "bf16"),
    ([300, 5, 0], [1, 150, 20], 1, 2, 128, "bf16", "e4m3"), ([10], [300], 1, 1, 256, "bf16", "bf16")])
def test_attention_of_prompts(ctx, new, H, G, D, dt, cache):
    """No trees: causal within the step."""
    say(f"attention of prompts ctx={ctx} new={new} H={H} G={G} D={D}")
    check_attn(attn_case(ctx, new, H, G, D, dt, cache, 16, D + G, trees=False))


def test_attention_rows_that_see_nothing():
    """Empty requests, nodes without bits over an empty context, and requests that were not served."""
    say("attention with empty rows")
    for D, G in ((64, 8), (128, 1), (256, 4)):
        s = attn_case([0, 0, 40, 10, 0, 9], [3, 1, 2, 5, 0, 4], 2, G, D, "bf16", "bf16", 16, 1)
        s["mask"][0] = 0
        s["mask"][2] = 0
        s["mask"][3] = 0   # request 1's only row
        s["mask"][4] = 0   # over a context: sees that
        s["lens"][3] = 0   # not served
        s["lens"][5] = 10 ** 6  # past the table's row
        got, lse = check_attn(s)
        empty = [0, 2, 3, 6, 7, 8, 9, 10, 11, 12, 13, 14]
        assert not got[empty].any() and (lse[empty] == -math.inf).all()
        s["lens"][2] = -1
        got, lse = check_attn(s)
        assert not got[4:6].any()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_bad_pages(cache):
    """Places in pages that do not exist are not seen."""
    say(f"attention with bad pages, {cache}")
    s = attn_case([100, 300, 0, 17, 60], [5, 40, 3, 1, 64], 2, 4, 128, "bf16", cache, 16, 2, bad_pages=12)
    check_attn(s)
    s["table"][:] = -1
    got, lse = check_attn(s)
    assert not got.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("D,dt,cache", [(64, "f16", "f16"), (128, "bf16", "bf16"), (256, "bf16", "bf16"),
                                        (128, "bf16", "e4m3"), (64, "f16", "e4m3")])
@pytest.mark.parametrize("trees,ctx,new,G", [(True, [70, 0, 33], [20, 40, 3], 4), (True, [70, 5], [2, 1], 3),
                                             (False, [20, 0], [150, 70], 1), (True, [100, 31], [64, 60], 8)])
def test_attention_not_finite_where_not_seen(D, dt, cache, trees, ctx, new, G):
    """NaN and infinities past the requests' ends, in pages of nobody, and at
    drafted places that some rows see: rows that do not see them stay as they
    were, to the bit; rows that see a NaN value have NaN there alone."""
    import torch
    say(f"attention with NaN D={D} {dt} {cache} trees={trees} new={new}")
    P, H = 16, 2
    s = attn_case(ctx, new, H, G, D, dt, cache, P, 3, trees=trees)
    want, want_lse = run_attn(s)
    used = np.zeros((s["pages"], P), bool)
    for r, L in enumerate(s["lens"]):
        for p in range(int(L)):
            used[s["table"][r, p // P], p % P] = True
    junk = torch.from_numpy(~used).cuda()
    raw = torch.uint8 if cache == "e4m3" else torch.int16
    nan = {"e4m3": 0x7f, "bf16": 0x7fc0, "f16": 0x7e00}[cache]
    inf = {"e4m3": 0xff, "bf16": 0xff80 - 0x10000, "f16": 0xfc00 - 0x10000}[cache]
    for x, bits in ((s["kc"], nan), (s["vc"], inf)):
        x.view(raw)[junk] = bits
    got, lse = run_attn(s)
    assert torch.equal(got, want) and torch.equal(lse, want_lse), "places past the ends were read"
    # the last node of request 0: its value of head 1, dimension 5
    place = int(s["lens"][0]) - 1
    page, at = int(s["table"][0, place // P]), place % P
    s["vc"].view(raw)[page, at, 1, 5] = nan
    s["kc"].view(raw)[page, at, 0, 3] = nan
    got, lse = run_attn(s)
    n = int(s["cu"][1])
    vis = R_.sees(n, int(s["lens"][0]), None if s["mask"] is None else np.ascontiguousarray(s["mask"][:n]))
    sees = vis[:, place].tolist()
    assert any(sees) and not all(sees)
    for t in range(s["q"].shape[0]):
        if t < n and sees[t]:
            assert got[t, :G].isnan().all() and lse[t, :G].isnan().all()  # a NaN score
            assert got[t, G:, 5].isnan().all()                            # a NaN value
            rest = [d for d in range(D) if d != 5]
            assert torch.equal(got[t, G:][:, rest], want[t, G:][:, rest])
            assert torch.equal(lse[t, G:], want_lse[t, G:])
        else:
            assert torch.equal(got[t], want[t]) and torch.equal(lse[t], want_lse[t]), t


def test_attention_infinite_value_that_is_seen():
    """An infinity in V at a committed place: infinite in that dimension for every row, finite elsewhere."""
    import torch
    say("attention with a seen infinity")
    s = attn_case([50], [6], 1, 2, 64, "bf16", "bf16", 16, 5)
    want, _ = run_attn(s)
    page = int(s["table"][0, 0])
    s["vc"][page, 3, 0, 9] = float("inf")
    got, _ = run_attn(s)
    assert (got[:, :, 9] == math.inf).all()
    rest = [d for d in range(64) if d != 9]
    assert torch.equal(got[..., rest], want[..., rest])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("G,new", [(8, [1, 1]), (4, [40, 20]), (2, [150, 1])])
def test_attention_sharp_and_rising_scores(dt, G, new):
    """Scores in the hundreds that rise along the cache: the running maximum
    moves often, and the first weights vanish."""
    import torch
    say(f"attention with rising scores {dt} G={G}")
    s = attn_case([700, 300], new, 1, G, 64, dt, dt, 16, 6, q_std=0.0, trees=False)
    s["q"][:] = 4.0
    s["kc"].zero_()
    for r, L in enumerate(s["lens"]):
        for p in range(int(L)):
            s["kc"][int(s["table"][r, p // 16]), p % 16, 0] = (p % 97) / 16.0 if r else p / 64.0
    s["clean"] = R_.wide(s["kc"]), R_.wide(s["vc"])
    check_attn(s)
    s["scale"] = -s["scale"]
    check_attn(s)
    s["scale"] = 0.0
    check_attn(s)


def test_attention_strides_and_no_lse():
    """Rows of q and out inside wider ones; a cache of other strides; lse left out."""
    import torch
    say("attention strides")
    s = attn_case([90, 3], [3, 20], 2, 4, 128, "bf16", "bf16", 16, 7)
    want, _ = run_attn(s)
    T, Hq, D = s["q"].shape
    wide = torch.zeros((T, Hq * D + 40), dtype=s["q"].dtype, device="cuda")
    wide[:, :Hq * D] = s["q"].reshape(T, Hq * D)
    out = torch.full((T, Hq * D + 72), 5.0, dtype=s["q"].dtype, device="cuda")
    s["q"] = wide[:, :Hq * D].view(T, Hq, D) if False else wide.as_strided((T, Hq, D), (Hq * D + 40, D, 1))
    for name in ("kc", "vc"):
        big = torch.zeros((s["pages"] + 1, 2, 16 + 3, D + 8), dtype=torch.bfloat16, device="cuda")
        view = big[:s["pages"], :, :16, :D].permute(0, 2, 1, 3)
        view.copy_(s[name])
        s[name] = view
    got, _ = run_attn(s, lse=False, out=out.as_strided((T, Hq, D), (Hq * D + 72, D, 1)))
    assert torch.equal(got.reshape(T, -1), want.reshape(T, -1))
    assert (out[:, Hq * D:] == 5.0).all()


def test_attention_offsets_past_32_bits():
    """Pages whose rows lie more than 4 GiB apart."""
    import torch
    say("attention and append past 4 GiB")
    P, H, D, pages = 16, 1, 64, 5
    stride = (1 << 31) + 1024  # elements: 4 GiB and a little
    kv = []
    for _ in range(2):
        buf = torch.empty(stride * (pages - 1) + P * D, dtype=torch.bfloat16, device="cuda")
        kv.append(buf.as_strided((pages, P, H, D), (stride, D, P * D, 1)))
    s = attn_case([50], [9], H, 4, D, "bf16", "bf16", P, 8, spare=1)
    assert s["pages"] == pages
    want, _ = run_attn(s)
    kv[0].copy_(s["kc"])
    kv[1].copy_(s["vc"])
    s["kc"], s["vc"] = kv
    got, _ = run_attn(s)
    assert torch.equal(got, want)
    # the append and the commit at the same offsets
    c = K.k3_kv_cache_of(*kv)
    x = torch.randn((2, 3 * D), device="cuda").to(torch.bfloat16)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    K.k3_qk_norm_rope(x[:, :D], x[:, D:2 * D], x[:, 2 * D:], 2, 1, w, w, 0.0, None, 0, False, R_.i32([0, 0]),
                      torch.empty((2, 1, D), dtype=torch.bfloat16, device="cuda"), c, R_.i32([4 * P + 3, 2]))
    assert torch.equal(kv[1][4, 3, 0], x[0, 2 * D:]) and torch.equal(kv[1][0, 2, 0], x[1, 2 * D:])
    out = torch.empty(1, dtype=torch.int32, device="cuda")
    K.k3_kv_commit(c, 1, 0, R_.i32([[4, 3]]), 2, R_.i32([1]), R_.i32([[2, 17]]), R_.i32([2]), 2, 1, out)
    assert out.item() == 3 and torch.equal(kv[1][4, 1, 0], x[0, 2 * D:])


def test_attention_request_left_out():
    """cu that is not ascending within [0, T]: those requests' rows stay as they were."""
    import torch
    say("attention with unsound cu")
    s = attn_case([30, 20, 10], [4, 5, 3], 1, 4, 64, "bf16", "bf16", 16, 9)
    want, _ = run_attn(s)
    s["cu"] = np.array([0, 4, 10 ** 9, 12])
    got, lse = run_attn(s)
    assert torch.equal(got[:4], want[:4]) and (got[4:] == 7).all() and (lse[4:] == 7).all()
    s["cu"] = np.array([-4, 4, 9, 5])
    got, _ = run_attn(s)
    assert torch.equal(got[4:9], want[4:9]) and (got[:4] == 7).all() and (got[9:] == 7).all()


def test_attention_same_bits_again_and_on_another_stream():
    import torch
    say("attention again, on a side stream")
    s = attn_case([3000, 40, 900], [1, 30, 7], 2, 4, 128, "bf16", "bf16", 16, 10)
    want, lse = run_attn(s)
    side = torch.cuda.Stream()
    for _ in range(3):
        got, l2 = run_attn(s)
        assert torch.equal(got, want) and torch.equal(l2, lse)
        torch.cuda.synchronize()
        got, l2 = run_attn(s, stream=side)
        assert torch.equal(got, want) and torch.equal(l2, lse)


# ---- commit -------------------------------------------------------------------------

def commit_ref(k, table, ctx, acc, num, most, n_pages, P, blocks):
    k, out = k.clone(), np.array(ctx).copy()
    for r in range(len(ctx)):
        n = int(num[r])
        if n < 0 or n > most or ctx[r] < 0:
            continue
        a = [int(x) for x in acc[r][:n]]
        if any(a[i] <= (a[i - 1] if i else -1) for i in range(n)):
            continue
        moves = []
        ok = True
        for i in range(n):
            if a[i] == i:
                continue
            at = []
            for p in (int(ctx[r]) + a[i], int(ctx[r]) + i):
                page = int(table[r][p // P]) if p // P < blocks else -1
                ok = ok and 0 <= page < n_pages
                at.append((page, p % P))
            moves.append(at)
        if not ok:
            continue
        rows = [k[:, x[0][0], x[0][1]].clone() for x in moves]
        for row, x in zip(rows, moves):
            k[:, x[1][0], x[1][1]] = row
        out[r] = ctx[r] + n
    return k, out


@pytest.mark.parametrize("R,layers,most,n_max,H,D,kind,P", [
    (1, 1, 1, 5, 1, 64, "bf16", 16), (9, 3, 6, 30, 4, 128, "bf16", 16), (33, 2, 20, 64, 8, 64, "e4m3", 24),
    (5, 4, 64, 64, 2, 256, "f16", 7), (3, 1, 1000, 1024, 1, 64, "f16", 64)])
def test_commit(R, layers, most, n_max, H, D, kind, P):
    import torch
    say(f"commit R={R} layers={layers} most={most} H={H} D={D} {kind} P={P}")
    rng = np.random.default_rng(R + most)
    g = _gen(R)
    ctx = rng.integers(0, 60, R)
    blocks = -(-(60 + n_max) // P) + 1
    pages = R * blocks
    table = rng.permutation(pages).reshape(R, blocks)
    num = rng.integers(0, most + 1, R)
    acc = np.stack([np.sort(rng.permutation(max(n_max, most))[:most]) for _ in range(R)])
    acc[0] = np.arange(most)  # a path that lies there already
    if R > 8:  # unsound ones
        num[1], num[2] = -1, most + 1
        acc[3] = acc[3][::-1]
        num[3] = most
        acc[4][0] = -2
        num[4] = 1
        table[5] = -1
        num[5] = most
        acc[5] = np.arange(most) + 3
        table[6][-1] = pages
        ctx[7] = 2 ** 31 - 1
    full = [R_.cache(layers * pages, P, H, D, kind, g).unflatten(0, (layers, pages)) for _ in range(2)]
    raw = torch.uint8 if kind == "e4m3" else torch.int16
    want = [commit_ref(x.view(raw).cpu(), table, ctx, acc, num, most, pages, P, blocks) for x in full]
    out = torch.full((R,), -5, dtype=torch.int32, device="cuda")
    K.k3_kv_commit(K.k3_kv_cache_of(full[0][0], full[1][0]), layers, full[0].stride(0), R_.i32(table), blocks,
                   R_.i32(ctx), R_.i32(acc), R_.i32(num), most, R, out)
    torch.cuda.synchronize()
    for x, (w, o) in zip(full, want):
        assert torch.equal(x.view(raw).cpu(), w)
        assert out.cpu().tolist() == o.tolist()


# ---- together ---------------------------------------------------------------------

def test_graph_of_a_step():
    """Plan, append, attention and commit captured into one graph, replayed
    with new lengths and rows between eager runs: the same bits as eager."""
    import torch
    say("graph of a step")
    R, n, H, G, D, P, layers = 6, 8, 2, 4, 64, 16, 2
    T, Hq, blocks = R * n, H * G, 12
    n_pages = R * blocks
    rng = np.random.default_rng(4)
    i32 = R_.i32
    ctx0 = [rng.integers(0, 120, R) for _ in range(4)]
    held0 = [-(-c // P) for c in ctx0]
    st = {k: i32(np.zeros(s)) for k, s in dict(ctx=R, new=R, parents=T, held=R, ring=n_pages, state=2,
                                               table=(R, blocks), held_out=R, ring_out=2, cu=R + 1, kv=R, slots=T,
                                               pos=T, mask=(T, 1), status=2, acc=(R, 3), num=R, ctx_out=R).items()}
    g = _gen(1)
    x = torch.zeros((T, (Hq + 2 * H) * D), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    freq = torch.tensor(100.0 ** (-np.arange(32) / 32), dtype=torch.float32, device="cuda")
    kc, vc = (R_.cache(layers * n_pages, P, H, D, "bf16", g).unflatten(0, (layers, n_pages)) for _ in range(2))
    q = torch.zeros((layers, T, Hq, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((layers, T, Hq), device="cuda")
    ws = torch.empty(K.k3_tree_attention_workspace_bytes(T, Hq, H, D), dtype=torch.uint8, device="cuda")
    caches = [K.k3_kv_cache_of(kc[i], vc[i]) for i in range(layers)]
    base = kc.clone(), vc.clone()

    def step():
        K.k3_kv_plan(st["ctx"], st["new"], st["parents"], R, T, n_pages, P, blocks, st["held"], st["ring"],
                     st["state"], st["table"], st["held_out"], st["ring_out"], st["cu"], st["kv"], st["slots"],
                     st["pos"], st["mask"], 1, st["status"])
        for i in range(layers):
            K.k3_qk_norm_rope(x[:, :Hq * D], x[:, Hq * D:(Hq + H) * D], x[:, (Hq + H) * D:], T, Hq, w, w, 1e-6, freq,
                              64, False, st["pos"], q[i], caches[i], st["slots"])
            K.k3_tree_attention(q[i], T, Hq, caches[i], st["table"], blocks, st["cu"], st["kv"], R, st["mask"], 1,
                                D ** -0.5, out[i], ws, lse=lse[i])
        K.k3_kv_commit(caches[0], layers, kc.stride(0), st["table"], blocks, st["ctx"], st["acc"], st["num"], 3, R,
                       st["ctx_out"])

    def load(k):
        r = np.random.default_rng(k)
        c, h = ctx0[k], held0[k]
        table = np.full((R, blocks), -1)
        ids = r.permutation(n_pages)
        off = np.concatenate([[0], np.cumsum(h)])
        for i in range(R):
            table[i, :h[i]] = ids[off[i]:off[i + 1]]
        ring = np.full(n_pages, -1)
        free = ids[off[R]:]
        ring[:len(free)] = free
        values = dict(ctx=c, new=np.full(R, n), parents=np.concatenate([R_.tree(n, r) for _ in range(R)]), held=h,
                      ring=ring, state=[0, len(free)], table=table, acc=np.tile([0, 2, 5], (R, 1)),
                      num=r.integers(0, 4, R))
        for name, v in values.items():
            st[name].copy_(i32(v).view(st[name].shape))
        gg = _gen(k)
        x.copy_(torch.randn(x.shape, generator=gg, device="cuda").to(x.dtype))
        kc.copy_(base[0])
        vc.copy_(base[1])
        torch.cuda.synchronize()

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (out, lse, q, kc, vc, *st.values())]

    load(0)
    step()  # the first call loads the kernels
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in (1, 2, 3, 1, 2):
        load(k)
        step()
        want = result()
        assert not want[0].isnan().any()
        load(k)
        graph.replay()
        for a, b in zip(result(), want):
            assert torch.equal(a, b)
