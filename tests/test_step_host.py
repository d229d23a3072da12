"""Refusals of the norm and the log probabilities before any launch, and of
their binding before the C call (no GPU needed): the addresses given are
never touched."""
import os

import pytest
import torch

import mxfp4_packed_weight_amd as K
from tests.test_kv_host import _p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return K.lib()


NORM = dict(x=_p(1), xs=256, r=_p(2), rs=256, dt=K.K3_BF16, T=3, n=256, w=_p(3), eps=1e-6, sum=_p(4), ss=256,
            y=_p(5), ys=256, y8=_p(6), y8s=256, sc=_p(7), group=64, s=None)


@pytest.mark.parametrize("change,status,says", [
    (dict(x=None), 1, "x is NULL"), (dict(w=None), 1, "w is NULL"), (dict(x=_p(1) + 8), 1, "x is not 16-byte"),
    (dict(r=_p(2) + 2), 1, "residual is not 16-byte"), (dict(sum=_p(4) + 2), 1, "sum is not"),
    (dict(y8=_p(6) + 4), 1, "y8 is not 8-byte"), (dict(sc=None), 1, "scales is NULL"),
    (dict(y=None, y8=None), 1, "both y and y8"), (dict(dt=K.K3_E4M3), 2, "dtype=2"), (dict(dt=K.K3_F32), 2, "dtype=3"),
    (dict(T=-1), 2, "T=-1"), (dict(T=(1 << 20) + 1), 2, "T="), (dict(n=0), 2, "hidden=0"), (dict(n=252), 2, "hidden=252"),
    (dict(n=16392), 2, "hidden=16392"), (dict(eps=-1.0), 2, "eps"), (dict(eps=float("nan")), 2, "eps"),
    (dict(group=0), 2, "group=0"), (dict(group=48), 2, "group=48"), (dict(group=512), 2, "group=512"),
    (dict(group=96, n=288), 2, "group=96"), (dict(group=64, n=224), 2, "group=64"), (dict(group=-64), 2, "group=-64"),
    (dict(xs=248), 2, "x_stride"), (dict(rs=260), 2, "residual_stride"), (dict(ss=-256), 2, "sum_stride"),
    (dict(ys=8), 2, "y_stride"), (dict(y8s=252), 2, "y8_stride"), (dict(sum=_p(2), ss=512), 2, "sum is an input"),
    (dict(y=_p(1), ys=512), 2, "y is an input"), (dict(y8=_p(1)), 2, "y8 is an input"),
    (dict(sum=_p(5)), 2, "another output"), (dict(y=_p(6)), 2, "y is y8")])
def test_norm_refusals(L, change, status, says):
    assert L.k3_add_rms_norm(*{**NORM, **change}.values()) == status
    assert says in K.last_error() and "k3_add_rms_norm" in K.last_error()


LOGP = dict(x=_p(1), stride=1000, dt=K.K3_BF16, T=3, V=1000, beta=1.0, tok=_p(2), k=4, lp=_p(3), ent=_p(4), lse=_p(5),
            top=_p(6), tlp=_p(7), ws=_p(8), nb=1 << 40, s=None)


@pytest.mark.parametrize("change,status,says", [
    (dict(x=None), 1, "logits is NULL"), (dict(x=_p(1) + 1), 1, "2-byte"), (dict(x=_p(1) + 2, dt=K.K3_F32), 1, "4-byte"),
    (dict(tok=None), 1, "go together"), (dict(lp=None), 1, "go together"), (dict(ent=_p(4) + 2), 1, "entropy is not"),
    (dict(top=None), 1, "top is NULL"), (dict(tlp=None), 1, "top_logprob is NULL"), (dict(dt=K.K3_E4M3), 2, "dtype=2"),
    (dict(T=-1), 2, "T=-1"), (dict(V=0), 2, "V=0"), (dict(V=(1 << 24) + 1), 2, "2^24"), (dict(k=-1), 2, "k=-1"),
    (dict(k=K.K3_MAX_TOPK + 1), 2, "k=65"), (dict(V=3), 2, "k=4"), (dict(stride=999), 2, "stride=999"),
    (dict(beta=0.0), 2, "beta=0"), (dict(beta=-1.0), 2, "beta=-1"), (dict(beta=float("nan")), 2, "beta"),
    (dict(beta=float("inf")), 2, "beta")])
def test_logprobs_refusals(L, change, status, says):
    assert L.k3_token_logprobs(*{**LOGP, **change}.values()) == status
    assert says in K.last_error() and "k3_token_logprobs" in K.last_error()


def test_calls_without_rows(L):
    """T = 0 enqueues nothing and needs no rows."""
    none = {k: None for k in ("x", "r", "sum", "y", "y8", "sc")}
    assert L.k3_add_rms_norm(*{**NORM, **none, "T": 0}.values()) == K.K3_OK
    none = {k: None for k in ("x", "tok", "lp", "ent", "lse", "top", "tlp", "ws")}
    assert L.k3_token_logprobs(*{**LOGP, **none, "T": 0}.values()) == K.K3_OK


def test_workspace_bytes(L):
    assert K.k3_token_logprobs_workspace_bytes(0, 1000, 4) == 0
    for bad in ((-1, 1000, 4), (1, 0, 0), (1, 10, 11), (1, 1000, 65)):
        assert K.k3_token_logprobs_workspace_bytes(*bad) == 0 and K.last_error()


class _Stream:
    cuda_stream = 0


@pytest.fixture
def calls(monkeypatch):
    """The C calls' arguments, in place of the calls."""
    seen = []
    names = ("k3_add_rms_norm", "k3_token_logprobs")
    monkeypatch.setattr(K, "_functions", {n: (lambda *a, n=n: seen.append((n, a)) or K.K3_OK) for n in names})
    return seen


T, N, V, TOP = 4, 64, 100, 3


def arguments(name):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    if name == "k3_add_rms_norm":
        return dict(x=z(T, N), residual=z(T, N), T=T, hidden=N, w=z(N), eps=1e-6, sum_out=z(T, N), y=z(T, N),
                    y8=z(T, N, dtype=torch.float8_e4m3fn), scales=z(T, N // 32, dtype=torch.float32), group=32)
    f = torch.float32
    return dict(logits=z(T, V), T=T, V=V, beta=1.0, tokens=z(T, dtype=torch.int32), k=TOP, logprob=z(T, dtype=f),
                entropy=z(T, dtype=f), lse=z(T, dtype=f), top=z(T, TOP, dtype=torch.int32),
                top_logprob=z(T, TOP, dtype=f), ws=z(64, dtype=torch.uint8))


def call(name, **change):
    return getattr(K, name)(**{**arguments(name), **change}, stream=_Stream())


@pytest.mark.parametrize("name", ["k3_add_rms_norm", "k3_token_logprobs"])
def test_sound_arguments_reach_the_call(calls, name):
    a = arguments(name)
    getattr(K, name)(**a, stream=_Stream())
    (got, args), = calls
    assert got == name
    for k, v in a.items():
        if torch.is_tensor(v):
            assert v.data_ptr() in args, k


@pytest.mark.parametrize("name,arg", [(n, k) for n in ("k3_add_rms_norm", "k3_token_logprobs")
                                      for k, v in arguments(n).items() if torch.is_tensor(v)])
def test_types_and_sizes(calls, name, arg):
    t = arguments(name)[arg]
    if arg not in ("x", "logits", "ws"):
        with pytest.raises(TypeError, match=arg):
            call(name, **{arg: t.double()})
    elif arg != "ws":
        with pytest.raises(TypeError):
            call(name, **{arg: t.double()})
    strided = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
    with pytest.raises(ValueError, match=arg):
        call(name, **{arg: strided})
    if arg != "ws":
        short = t[:-1] if t.dim() == 2 else t.reshape(-1)[:-1]
        with pytest.raises(ValueError, match=arg):
            call(name, **{arg: short})
    assert not calls


def test_rows_in_wider_ones(calls):
    call("k3_add_rms_norm", x=torch.zeros(T + 1, 3 * N, dtype=torch.bfloat16)[:, :N + 8])
    call("k3_token_logprobs", logits=torch.zeros(T + 1, V + 3, dtype=torch.float32))
    assert calls[0][1][1] == 3 * N and calls[1][1][1] == V + 3 and calls[1][1][2] == K.K3_F32
    for wrong in (torch.zeros(T, N - 8, dtype=torch.bfloat16), torch.zeros(T * N, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="x"):
            call("k3_add_rms_norm", x=wrong)


def test_arrays_that_may_be_left_out(calls):
    call("k3_add_rms_norm", residual=None, sum_out=None, y8=None, scales=None, group=0)
    call("k3_token_logprobs", tokens=None, logprob=None, entropy=None, lse=None, top=None, top_logprob=None, k=0,
         ws=None)
    assert len(calls) == 2
