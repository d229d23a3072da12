"""Queries normed and rotated in place, inside the rows that hold keys and
values too."""
import pytest

import mxfp4_packed_weight_amd as K
from tests import test_gpu_kv as kv
from tests import _kv as R_
from tests._gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,G,D,rot,inter,dt", [
    (1, 8, 8, 128, 128, False, "bf16"), (40, 2, 5, 64, 32, False, "f16"), (700, 4, 8, 256, 256, True, "bf16"),
    (5000, 1, 3, 64, 64, False, "bf16")])
def test_queries_in_place(T, H, G, D, rot, inter, dt):
    """The same bits as into rows of their own; keys and values stay."""
    import torch
    say(f"qk in place T={T} H={H} G={G} D={D}")
    s = kv.qk_case(T, H, G, D, rot, inter, dt, dt, 16, 7)
    c, pos, slots = K.k3_kv_cache_of(s["kc"], s["vc"]), R_.i32(s["pos"]), R_.i32(s["slots"])
    x, n = s["x"].clone(), H * G * D

    def call(out):
        K.k3_qk_norm_rope(s["q"], s["k"], s["v"], T, H * G, s["wq"], s["wk"], s["eps"], s["freq"], rot, inter, pos,
                          out, c, slots)
        torch.cuda.synchronize()

    call(s["out"])
    cached = s["kc"].clone(), s["vc"].clone()
    call(s["q"])
    assert torch.equal(s["x"][:, :n], s["out"].view(T, n)) and torch.equal(s["x"][:, n:], x[:, n:])
    assert torch.equal(s["kc"], cached[0]) and torch.equal(s["vc"], cached[1])
