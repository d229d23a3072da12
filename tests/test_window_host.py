"""Refusals of the windowed attention and of the cache with exponents before
any launch, and of their binding before the C call (no GPU needed)."""
import ctypes
import os

import pytest
import torch

import mxfp4_packed_weight_amd as K
from tests.test_kv_binding_host import BLOCKS, D, H, HQ, P, PAGES, R, T, WORDS, _Stream, ints, rows
from tests.test_kv_binding_host import cache as cache_of_rows
from tests.test_kv_host import ATTN, _cache, _p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return K.lib()


def _ordered(a, names):
    return [a[n] for n in names]


WINDOW = {**ATTN, "window": 64, "sinks": 4}
WINDOW_ORDER = ("q", "qs", "dt", "T", "Hq", "cache", "table", "blocks", "cu", "kv", "R", "mask", "words", "window",
                "sinks", "scale", "out", "os", "ws", "nb", "lse", "s")


@pytest.mark.parametrize("change,status,says", [
    (dict(q=None), 1, "q is NULL"), (dict(ws=None), 1, "ws is NULL"), (dict(mask=_p(7) + 1), 1, "mask is not"),
    (dict(window=-1), 2, "window=-1"), (dict(window=(1 << 30) + 1), 2, "window="), (dict(sinks=-1), 2, "sinks=-1"),
    (dict(sinks=(1 << 30) + 1), 2, "sinks="), (dict(window=31), 2, "window=31"), (dict(words=3), 2, "96 nodes"),
    (dict(words=33), 2, "words=33"), (dict(T=-3), 2, "T=-3"), (dict(R=0), 2, "R=0"), (dict(qs=100), 2, "q_stride"),
    (dict(scale=float("nan")), 2, "scale"), (dict(nb=16), 3, "is below the"), (dict(out=_p(3)), 2, "out is q")])
def test_window_refusals(L, change, status, says):
    a = {**WINDOW, **change, "cache": ctypes.byref(_cache())}
    assert L.k3_window_attention(*_ordered(a, WINDOW_ORDER)) == status
    assert says in K.last_error() and "k3_window_attention" in K.last_error()


def _cache8(**kw):
    return _cache(**{**dict(dtype=K.K3_E4M3), **kw})


BLOCK = {**ATTN, "ke": _p(11), "ve": _p(12), "window": 0, "sinks": 0}
BLOCK_ORDER = ("q", "qs", "dt", "T", "Hq", "cache", "ke", "ve", "table", "blocks", "cu", "kv", "R", "window", "sinks",
               "scale", "out", "os", "ws", "nb", "lse", "s")
APPEND = dict(k=_p(1), ks=8 * 128, v=_p(2), vs=8 * 128, dt=K.K3_BF16, T=3, cache=None, ke=_p(3), ve=_p(4), table=_p(5),
              blocks=8, cu=_p(6), kv=_p(7), R=2, s=None)
CACHES = [(dict(dtype=K.K3_BF16), 2, "cache dtype=0"), (dict(k_scale=_p(9)), 2, "without scales"),
          (dict(v_scale=_p(9)), 2, "without scales"), (dict(page_size=18, page_stride=18 * 8 * 128), 2, "multiple of 4"),
          (dict(head_dim=96), 2, "head_dim=96"), (dict(k=None), 1, "c->k is NULL")]


@pytest.mark.parametrize("change,cache,status,says", [
    (dict(ke=None), {}, 1, "k_exp is NULL"), (dict(ve=None), {}, 1, "v_exp is NULL"), (dict(ve=_p(11)), {}, 2, "k_exp is v_exp"),
    (dict(window=-1), {}, 2, "window=-1"), (dict(sinks=-2), {}, 2, "sinks=-2"), (dict(dt=K.K3_E4M3), {}, 2, "dtype=2"),
    (dict(cu=None), {}, 1, "cu is NULL"), (dict(nb=16), {}, 3, "is below the"), (dict(Hq=63), {}, 2, "Hq=63")]
    + [({}, *c) for c in CACHES])
def test_block_attention_refusals(L, change, cache, status, says):
    a = {**BLOCK, **change, "cache": ctypes.byref(_cache8(**cache))}
    assert L.k3_block_attention(*_ordered(a, BLOCK_ORDER)) == status
    assert says in K.last_error() and "k3_block_attention" in K.last_error()


@pytest.mark.parametrize("change,cache,status,says", [
    (dict(k=None), {}, 1, "k_in is NULL"), (dict(v=_p(2) + 8), {}, 1, "v_in is not 16-byte"),
    (dict(ke=None), {}, 1, "k_exp is NULL"), (dict(ve=_p(3)), {}, 2, "k_exp is v_exp"), (dict(table=None), {}, 1, "table is NULL"),
    (dict(cu=_p(6) + 2), {}, 1, "cu is not"), (dict(kv=None), {}, 1, "kv_lens is NULL"), (dict(dt=K.K3_F32), {}, 2, "dtype=3"),
    (dict(T=-1), {}, 2, "T=-1"), (dict(T=(1 << 20) + 1), {}, 2, "T="), (dict(R=4097), {}, 2, "R=4097"),
    (dict(blocks=0), {}, 2, "blocks=0"), (dict(ks=8 * 128 - 8), {}, 2, "k_stride"), (dict(vs=8 * 128 + 4), {}, 2, "v_stride")]
    + [({}, *c) for c in CACHES])
def test_append_refusals(L, change, cache, status, says):
    a = {**APPEND, **change, "cache": ctypes.byref(_cache8(**cache))}
    assert L.k3_kv_append(*a.values()) == status
    assert says in K.last_error() and "k3_kv_append" in K.last_error()


def test_calls_without_tokens(L):
    none = {"T": 0, "q": None, "out": None}
    assert L.k3_window_attention(*_ordered({**WINDOW, **none, "cache": ctypes.byref(_cache())}, WINDOW_ORDER)) == K.K3_OK
    c = ctypes.byref(_cache8())
    assert L.k3_block_attention(*_ordered({**BLOCK, **none, "cache": c}, BLOCK_ORDER)) == K.K3_OK
    assert L.k3_kv_append(*{**APPEND, "T": 0, "k": None, "v": None, "cache": c}.values()) == K.K3_OK


# ---- the binding ------------------------------------------------------------------

NAMES = ("k3_window_attention", "k3_kv_append", "k3_block_attention")


@pytest.fixture
def calls(monkeypatch):
    """The C calls' arguments, in place of the calls."""
    seen = []
    monkeypatch.setattr(K, "_functions", {n: (lambda *a, n=n: seen.append((n, a)) or K.K3_OK) for n in NAMES})
    return seen


def cache8():
    k = torch.zeros(PAGES, H, P, D).to(torch.float8_e4m3fn).permute(0, 2, 1, 3)
    return K.k3_kv_cache_of(k, k.clone())


def arguments(name):
    lens = dict(table=ints(R, BLOCKS), blocks=BLOCKS, cu=ints(R + 1), kv_lens=ints(R), R=R)
    attn = dict(scale=0.1, out=rows(HQ), ws=torch.zeros(64, dtype=torch.uint8), lse=torch.zeros(T, HQ))
    if name == "k3_window_attention":
        return dict(q=rows(HQ), T=T, Hq=HQ, cache=cache_of_rows(), **lens, mask=ints(T, WORDS), words=WORDS, window=64,
                    sinks=1, **attn)
    e = lambda: torch.zeros(PAGES, H, dtype=torch.uint8)  # noqa: E731
    if name == "k3_kv_append":
        return dict(k_in=rows(H), v_in=rows(H), T=T, cache=cache8(), k_exp=e(), v_exp=e(), **lens)
    return dict(q=rows(HQ), T=T, Hq=HQ, cache=cache8(), k_exp=e(), v_exp=e(), **lens, window=0, sinks=0, **attn)


def call(name, **change):
    return getattr(K, name)(**{**arguments(name), **change}, stream=_Stream())


@pytest.mark.parametrize("name", NAMES)
def test_sound_arguments_reach_the_call(calls, name):
    a = arguments(name)
    getattr(K, name)(**a, stream=_Stream())
    (got, args), = calls
    assert got == name
    for k, v in a.items():
        if torch.is_tensor(v):
            assert v.data_ptr() in args, k


@pytest.mark.parametrize("name,arg", [(n, k) for n in NAMES for k, v in arguments(n).items()
                                      if torch.is_tensor(v) and k != "ws"])
def test_types_and_sizes(calls, name, arg):
    t = arguments(name)[arg]
    first = arg in ("q", "k_in")
    with pytest.raises(TypeError, match=None if first else arg):
        call(name, **{arg: t.double()})
    with pytest.raises(ValueError, match=arg):
        call(name, **{arg: torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]})
    short = t[:-1] if t.dim() == 3 else t.reshape(-1)[:-1]
    with pytest.raises(ValueError, match=arg):
        call(name, **{arg: short})
    assert not calls


def test_arrays_that_may_be_left_out(calls):
    call("k3_window_attention", mask=None, words=0, lse=None)
    call("k3_block_attention", lse=None)
    for name in ("k3_window_attention", "k3_block_attention"):
        with pytest.raises(ValueError, match="ws"):
            call(name, ws=torch.zeros(64, dtype=torch.uint8)[::2])
    assert len(calls) == 2
