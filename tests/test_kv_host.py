"""Refusals of the paged key/value cache calls, before any launch (no GPU
needed): the addresses given are never touched."""
import ctypes
import os

import pytest
import torch

import mxfp4_packed_weight_amd as K

P16 = 0x10000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return K.lib()


def _p(n):
    return P16 * n


def _cache(**kw):
    c = K.k3_kv_cache(_p(1), _p(2), None, None, 16 * 8 * 128, 8 * 128, 128, 10, 16, 8, 128, K.K3_BF16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


PLAN = dict(ctx=_p(1), new=_p(2), parents=_p(3), R=4, T=9, n_pages=10, page=16, blocks=8, held=_p(4),
            ring=_p(5), state=_p(6), table=_p(7), held_out=_p(8), ring_out=_p(9), cu=_p(10), kv=_p(11),
            slots=_p(12), pos=_p(13), mask=_p(14), words=2, status=_p(15), s=None)


@pytest.mark.parametrize("change,status,says", [
    (dict(ctx=None), 1, "ctx is NULL"), (dict(new=_p(2) + 2), 1, "4-byte aligned"),
    (dict(held=None), 1, "held is NULL"), (dict(status=None), 1, "status is NULL"),
    (dict(slots=None), 1, "slots is NULL"), (dict(mask=None), 1, "mask is NULL"),
    (dict(R=0), 2, "R=0"), (dict(R=K.K3_MAX_REQUESTS + 1), 2, "R=4097"), (dict(T=-1), 2, "T=-1"),
    (dict(T=(1 << 20) + 1), 2, "T="), (dict(n_pages=0), 2, "n_pages=0"), (dict(page=0), 2, "page_size=0"),
    (dict(n_pages=1 << 27, page=16), 2, "below 2^31"), (dict(blocks=0), 2, "blocks=0"),
    (dict(blocks=1 << 27), 2, "2^30 places"), (dict(words=0), 2, "words=0"),
    (dict(words=K.K3_MAX_TREE_WORDS + 1), 2, "words=33"), (dict(held_out=_p(4)), 2, "same array"),
    (dict(ring_out=_p(6)), 2, "same array"), (dict(kv=_p(1)), 2, "same array"),
    (dict(pos=_p(3)), 2, "same array")])
def test_plan_refusals(L, change, status, says):
    assert L.k3_kv_plan(*{**PLAN, **change}.values()) == status
    assert says in K.last_error()


QK = dict(q=_p(3), qs=64 * 128, k=_p(4), ks=8 * 128, v=_p(5), vs=8 * 128, dt=K.K3_BF16, T=3, Hq=64, wq=_p(6),
          wk=_p(7), eps=1e-6, freq=_p(8), rot=128, inter=0, pos=_p(9), out=_p(10), os=64 * 128, cache=None,
          slots=_p(11), s=None)


@pytest.mark.parametrize("change,cache,status,says", [
    (dict(q=None), {}, 1, "q_in is NULL"), (dict(k=_p(4) + 8), {}, 1, "16-byte aligned"),
    (dict(wq=None), {}, 1, "wq is NULL"), (dict(freq=None), {}, 1, "inv_freq is NULL"),
    (dict(slots=None), {}, 1, "slots is NULL"), (dict(out=None), {}, 1, "q_out is NULL"),
    (dict(dt=K.K3_E4M3), {}, 2, "dtype=2"), (dict(dt=K.K3_F16), {}, 2, "cache of dtype=0"),
    (dict(T=-1), {}, 2, "T=-1"), (dict(Hq=12), {}, 2, "Hq=12"), (dict(Hq=0), {}, 2, "Hq=0"),
    (dict(rot=136), {}, 2, "rot=136"), (dict(rot=8), {}, 2, "rot=8"), (dict(eps=-1.0), {}, 2, "eps"),
    (dict(eps=float("nan")), {}, 2, "eps"), (dict(qs=64 * 128 + 4), {}, 2, "q_stride"),
    (dict(vs=8 * 128 - 8), {}, 2, "v_stride"), (dict(out=_p(4)), {}, 2, "q_out is k_in"),
    ({}, dict(k=None), 1, "c->k is NULL"), ({}, dict(v=_p(2) + 8), 1, "16-byte aligned"),
    ({}, dict(head_dim=96), 2, "head_dim=96"), ({}, dict(dtype=7), 2, "dtype=7"),
    ({}, dict(k_scale=_p(12)), 2, "only an e4m3 cache"), ({}, dict(n_heads=0), 2, "n_heads=0"),
    ({}, dict(n_pages=0), 2, "n_pages=0"), ({}, dict(n_pages=1 << 27), 2, "below 2^31"),
    ({}, dict(slot_stride=8 * 128 + 4), 2, "strides"), ({}, dict(head_stride=64), 2, "at least a row"),
    ({}, dict(page_stride=-16), 2, "strides")])
def test_qk_refusals(L, change, cache, status, says):
    a = {**QK, **change, "cache": ctypes.byref(_cache(**cache))}
    assert L.k3_qk_norm_rope(*a.values()) == status
    assert says in K.last_error()


ATTN = dict(q=_p(3), qs=64 * 128, dt=K.K3_BF16, T=3, Hq=64, cache=None, table=_p(4), blocks=8, cu=_p(5),
            kv=_p(6), R=2, mask=_p(7), words=1, scale=0.1, out=_p(8), os=64 * 128, ws=_p(9), nb=1 << 40,
            lse=_p(10), s=None)


@pytest.mark.parametrize("change,status,says", [
    (dict(q=None), 1, "q is NULL"), (dict(out=_p(8) + 2), 1, "16-byte aligned"), (dict(ws=None), 1, "ws is NULL"),
    (dict(cu=None), 1, "cu is NULL"), (dict(kv=None), 1, "kv_lens is NULL"), (dict(table=None), 1, "table is NULL"),
    (dict(mask=_p(7) + 1), 1, "mask is not"), (dict(lse=_p(7) + 2), 1, "lse is not"), (dict(dt=K.K3_E4M3), 2, "dtype=2"),
    (dict(T=-3), 2, "T=-3"), (dict(Hq=63), 2, "Hq=63"), (dict(R=0), 2, "R=0"), (dict(blocks=0), 2, "blocks=0"),
    (dict(words=0), 2, "words=0"), (dict(words=33), 2, "words=33"), (dict(scale=float("inf")), 2, "scale"),
    (dict(qs=100), 2, "q_stride"), (dict(os=8), 2, "out_stride"), (dict(out=_p(3)), 2, "out is q"),
    (dict(nb=16), 3, "is below the")])
def test_attention_refusals(L, change, status, says):
    a = {**ATTN, **change, "cache": ctypes.byref(_cache())}
    assert L.k3_tree_attention(*a.values()) == status
    assert says in K.last_error()


COMMIT = dict(cache=None, layers=2, ls=1 << 20, table=_p(4), blocks=8, ctx=_p(5), acc=_p(6), n=_p(7), most=3, R=2,
              out=_p(8), s=None)


@pytest.mark.parametrize("change,status,says", [
    (dict(ctx=None), 1, "ctx is NULL"), (dict(acc=None), 1, "accepted is NULL"), (dict(n=None), 1, "n_accepted is NULL"),
    (dict(out=None), 1, "ctx_out is NULL"), (dict(layers=0), 2, "layers=0"), (dict(ls=100), 2, "layer_stride=100"),
    (dict(most=0), 2, "most=0"), (dict(most=1025), 2, "most=1025"), (dict(R=0), 2, "R=0"),
    (dict(out=_p(5)), 2, "same array")])
def test_commit_refusals(L, change, status, says):
    a = {**COMMIT, **change, "cache": ctypes.byref(_cache())}
    assert L.k3_kv_commit(*a.values()) == status
    assert says in K.last_error()


def test_a_step_without_tokens_is_accepted(L):
    """T = 0 enqueues nothing in the per-layer calls and needs no rows."""
    c = ctypes.byref(_cache())
    rows = {k: None for k in ("q", "k", "v", "pos", "out", "slots")}
    assert L.k3_qk_norm_rope(*{**QK, **rows, "T": 0, "cache": c}.values()) == K.K3_OK
    assert L.k3_tree_attention(*{**ATTN, "q": None, "out": None, "T": 0, "cache": c}.values()) == K.K3_OK


def test_workspace_size(L):
    for bad in ((1, 64, 0, 128), (1, 64, 8, 80), (-1, 64, 8, 128), (1, 60, 8, 128)):
        assert K.k3_tree_attention_workspace_bytes(*bad) == 0
    for T in (0, 1, 5, 100, 5000):
        assert 0 < K.k3_tree_attention_workspace_bytes(T, 64, 8, 128) < 1 << 28


def test_cache_handle():
    k = torch.zeros(5, 4, 16, 64, dtype=torch.bfloat16).permute(0, 2, 1, 3)
    c = K.k3_kv_cache_of(k, torch.zeros_like(k))
    assert (c.n_pages, c.page_size, c.n_heads, c.head_dim) == (5, 16, 4, 64)
    assert (c.page_stride, c.slot_stride, c.head_stride) == (4 * 16 * 64, 64, 16 * 64)
    with pytest.raises(ValueError):
        K.k3_kv_cache_of(k, k.contiguous())
    with pytest.raises(ValueError):
        K.k3_kv_cache_of(k[..., ::2], k[..., ::2])
    with pytest.raises(ValueError):
        K.k3_kv_cache_of(k[0], k[0])
    with pytest.raises(TypeError):
        K.k3_kv_cache_of(k.float(), k.float())
    f8 = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        K.k3_kv_cache_of(f8, f8, torch.ones(3), torch.ones(4))
    assert K.k3_kv_cache_of(f8, f8, torch.ones(4), torch.ones(4)).dtype == K.K3_E4M3
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):  # rows of two types
        K.k3_qk_norm_rope(q, q.half(), q, 3, 8, w, w, 1e-6, None, 0, False, i, q, c, i, stream=_NoStream())
    with pytest.raises(TypeError):
        K.k3_qk_norm_rope(q, q, q, 3, 8, w.float(), w, 1e-6, None, 0, False, i, q, c, i, stream=_NoStream())
    with pytest.raises(ValueError):  # heads that are not dense
        K.k3_tree_attention(q.transpose(0, 1), 8, 3, c, i, 1, i, i, 1, None, 1, 1.0, q, w, stream=_NoStream())


class _NoStream:
    cuda_stream = 0
