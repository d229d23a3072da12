"""What the binding of the paged key/value cache calls refuses before the C
call (no GPU needed): arrays of another type, strided or too short ones, rows
of fewer tokens or heads than the call's."""
import pytest
import torch

import mxfp4_packed_weight_amd as K

R, T, BLOCKS, WORDS, PAGES, P, H, HQ, D, MOST = 3, 5, 4, 2, 7, 16, 2, 4, 64, 2


class _Stream:
    cuda_stream = 0


@pytest.fixture
def calls(monkeypatch):
    """The C calls' arguments, in place of the calls."""
    seen = []
    names = ("k3_kv_plan", "k3_qk_norm_rope", "k3_tree_attention", "k3_kv_commit", "k3_kv_commit_ex")
    monkeypatch.setattr(K, "_functions", {n: (lambda *a, n=n: seen.append((n, a)) or K.K3_OK) for n in names})
    return seen


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def rows(heads, n=T):
    return torch.zeros(n, heads, D, dtype=torch.bfloat16)


def cache():
    k = torch.zeros(PAGES, H, P, D, dtype=torch.bfloat16).permute(0, 2, 1, 3)
    return K.k3_kv_cache_of(k, torch.zeros_like(k))


def arguments(name):
    ones = torch.ones(D, dtype=torch.bfloat16)
    if name == "k3_kv_plan":
        return dict(ctx=ints(R), new=ints(R), parents=ints(T), R=R, T=T, n_pages=PAGES, page_size=P, blocks=BLOCKS,
                    held=ints(R), ring=ints(PAGES), ring_state=ints(2), table=ints(R, BLOCKS), held_out=ints(R),
                    ring_out=ints(2), cu=ints(R + 1), kv_lens=ints(R), slots=ints(T), positions=ints(T),
                    mask=ints(T, WORDS), words=WORDS, status=ints(2))
    if name == "k3_qk_norm_rope":
        return dict(q_in=rows(HQ), k_in=rows(H), v_in=rows(H), T=T, Hq=HQ, wq=ones, wk=ones.clone(), eps=1e-6,
                    inv_freq=torch.zeros(D // 2), rot=D, interleaved=False, positions=ints(T), q_out=rows(HQ),
                    cache=cache(), slots=ints(T))
    if name == "k3_tree_attention":
        return dict(q=rows(HQ), T=T, Hq=HQ, cache=cache(), table=ints(R, BLOCKS), blocks=BLOCKS, cu=ints(R + 1),
                    kv_lens=ints(R), R=R, mask=ints(T, WORDS), words=WORDS, scale=0.1, out=rows(HQ),
                    ws=torch.zeros(64, dtype=torch.uint8), lse=torch.zeros(T, HQ))
    a = dict(cache=cache(), layers=1, layer_stride=0, table=ints(R, BLOCKS), blocks=BLOCKS, ctx=ints(R),
             accepted=ints(R, MOST), n_accepted=ints(R), most=MOST, R=R, ctx_out=ints(R))
    return {**a, "kv_lens": ints(R)} if name == "k3_kv_commit_ex" else a


NAMES = ("k3_kv_plan", "k3_qk_norm_rope", "k3_tree_attention", "k3_kv_commit", "k3_kv_commit_ex")
INTS = {n: [k for k, v in arguments(n).items() if torch.is_tensor(v) and v.dtype == torch.int32] for n in NAMES}
ROWS = [("k3_qk_norm_rope", k) for k in ("q_in", "k_in", "v_in", "q_out")]
ROWS += [("k3_tree_attention", k) for k in ("q", "out")]


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


@pytest.mark.parametrize("name,arg", [(n, k) for n in NAMES for k in INTS[n]])
def test_integer_arrays(calls, name, arg):
    t = arguments(name)[arg]
    for wrong in (t.long(), t.float(), t.to(torch.int16)):
        with pytest.raises(TypeError, match=arg):
            call(name, **{arg: wrong})
    with pytest.raises(ValueError, match=arg):  # strided
        call(name, **{arg: torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=torch.int32)[..., ::2]})
    with pytest.raises(ValueError, match=arg):  # one value short
        call(name, **{arg: t.reshape(-1)[:-1]})
    assert not calls
    call(name, **{arg: torch.zeros(t.numel() + 3, dtype=torch.int32)})  # more than is needed
    assert len(calls) == 1


@pytest.mark.parametrize("name,arg", ROWS)
def test_rows(calls, name, arg):
    t = arguments(name)[arg]
    heads = t.shape[1]
    with pytest.raises(TypeError, match=arg if arg not in ("q_in", "q") else None):
        call(name, **{arg: t.half()})
    for wrong in (t[:-1], t[:, :-1], t.flatten(1)[:, :-8], t.flatten(1)[:-1], t.flatten(),
                  torch.zeros(T, heads, 2 * D, dtype=t.dtype)[..., ::2], t.transpose(0, 1),
                  torch.zeros(T, heads, 2 * D, dtype=t.dtype)[..., :D]):
        with pytest.raises(ValueError, match=arg):
            call(name, **{arg: wrong})
    assert not calls
    for right in (rows(heads, T + 2), t.flatten(1), torch.zeros(T, 3 * heads * D, dtype=t.dtype),
                  torch.zeros(T, heads + 3, D, dtype=t.dtype)[:, :heads]):
        call(name, **{arg: right})
    assert len(calls) == 4


@pytest.mark.parametrize("name,arg,dtype", [
    ("k3_qk_norm_rope", "inv_freq", torch.float32), ("k3_qk_norm_rope", "wq", torch.bfloat16),
    ("k3_qk_norm_rope", "wk", torch.bfloat16), ("k3_tree_attention", "lse", torch.float32)])
def test_other_arrays(calls, name, arg, dtype):
    t = arguments(name)[arg]
    with pytest.raises(TypeError, match=arg):
        call(name, **{arg: t.double()})
    with pytest.raises(ValueError, match=arg):
        call(name, **{arg: torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=dtype)[..., ::2]})
    with pytest.raises(ValueError, match=arg):
        call(name, **{arg: t.reshape(-1)[:-1]})
    assert not calls


def test_workspace_is_dense(calls):
    with pytest.raises(ValueError, match="ws"):
        call("k3_tree_attention", ws=torch.zeros(64, dtype=torch.uint8)[::2])
    assert not calls


def test_arrays_that_may_be_left_out(calls):
    call("k3_kv_plan", parents=None, mask=None, words=0)
    call("k3_kv_plan", parents=None, mask=None, words=0, slots=None, positions=None, T=0)
    call("k3_qk_norm_rope", inv_freq=None, rot=0)
    call("k3_tree_attention", mask=None, words=1, lse=None)
    assert len(calls) == 4
