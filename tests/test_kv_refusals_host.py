"""Refusals of the commit with the step's lengths, and of queries in place at
another stride, before any launch (no GPU needed): the addresses given are
never touched."""
import ctypes
import os

import pytest

import mxfp4_packed_weight_amd as K
from tests.test_kv_host import COMMIT, QK, _cache, _p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return K.lib()


ORDER = ("cache", "layers", "ls", "table", "blocks", "ctx", "lens", "acc", "n", "most", "R", "out", "s")


@pytest.mark.parametrize("change,status,says", [
    (dict(lens=None), 1, "kv_lens is NULL"), (dict(lens=_p(9) + 1), 1, "kv_lens is not 4-byte"),
    (dict(ctx=None), 1, "ctx is NULL"), (dict(most=1025), 2, "most=1025"), (dict(R=0), 2, "R=0"),
    (dict(out=_p(9)), 2, "same array"), (dict(out=_p(5)), 2, "same array")])
def test_commit_ex_refusals(L, change, status, says):
    a = {**COMMIT, "lens": _p(9), **change, "cache": ctypes.byref(_cache())}
    assert L.k3_kv_commit_ex(*(a[k] for k in ORDER)) == status
    assert says in K.last_error() and "k3_kv_commit_ex" in K.last_error()


@pytest.mark.parametrize("change,status", [
    (dict(out=_p(3), os=66 * 128), 2), (dict(out=_p(3), qs=66 * 128), 2), (dict(out=_p(3), T=0, os=66 * 128), 0)])
def test_queries_in_place_keep_their_stride(L, change, status):
    """Rows written at another stride would land on rows that are still to be read."""
    a = {**QK, **change, "cache": ctypes.byref(_cache())}
    assert L.k3_qk_norm_rope(*a.values()) == status
    assert status == 0 or "q_out is q_in" in K.last_error()
