"""The workspace that k3_token_logprobs asks for: one for the largest step
does for every smaller one (no GPU needed)."""
import os

import pytest

import mxfp4_packed_weight_amd as K
from tests.test_kv_host import _p
from tests.test_step_host import LOGP


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return K.lib()


@pytest.mark.parametrize("V", [1, 4095, 8192, 50021, 131072, 1 << 24])
def test_never_less_for_more(L, V):
    size = K.k3_token_logprobs_workspace_bytes
    for k in (0, 1):
        last = 0
        for T in [*range(0, 1100), 5000, 1 << 20]:
            now = size(T, V, k)
            assert now >= last and now >= size(T, max(1, V // 2), k), (T, k)
            last = now
    assert size(300, V, 1) >= size(300, V, 0)


def test_calls_take_what_they_need(L):
    """A call of one part to a row works without a workspace; one of several refuses too small a one."""
    long = {**LOGP, "V": 131072, "stride": 131072, "T": 3}
    assert L.k3_token_logprobs(*{**long, "nb": 1024}.values()) == K.K3_ERR_MEMORY
    assert L.k3_token_logprobs(*{**long, "ws": None}.values()) == K.K3_ERR_ARG
    # (T = 1000: one part; only its other arguments are looked at: `top` is refused last)
    assert L.k3_token_logprobs(*{**long, "T": 1000, "ws": None, "top": _p(6) + 2}.values()) == K.K3_ERR_ARG
    assert "top is not 4-byte" in K.last_error()
