"""k3_token_logprobs where some lanes of a wave have read nothing but -inf (masks
that leave a few tokens, rows shorter than a wave's run) and the others large
products of logit and inverse temperature: one row has one reference."""
import math

import numpy as np
import pytest

from tests.test_gpu_logprobs import check, logits
from tests._gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [97, 200, 1003, 5000, 70001])
@pytest.mark.parametrize("size,beta", [(25.3, 100.0), (7100.0, 1.0), (7100.0, 50.0), (20.0, 1000.0), (300.0, 1000.0),
                                       (30000.0, 30.0)])
def test_few_tokens_of_large_products(size, beta, V, kind):
    """The products beta x / ln 2 are between 3600 and 2^20 to 2^21, on both sides of where the differences change."""
    import torch
    say(f"logprobs of masked rows size={size} beta={beta} V={V} {kind}")
    near = size + logits(8, V, "f32", V, std=3 / beta)
    x = torch.full((8, V), -math.inf, device="cuda")
    x[0, V // 3] = size
    x[1, [5, V - 2]] = torch.tensor([size, size * (1 - 1 / 14200)], device="cuda")
    some = [1, V // 4, V // 2, V - 9, V - 1]
    x[2, some] = near[2, some]
    x[3] = near[3]
    x[4, some] = -near[4, some]
    x[5, V // 2:] = near[5, V // 2:]
    x[6] = -near[6]
    x[7, :64] = near[7, :64] - 40 / beta  # the largest come last
    x[7, V - 1] = size
    tokens = [V // 3, V - 2, V // 2, 7, 1, V - 3, 0, 9]
    for k in (0, 5):
        check(x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[kind]), beta, tokens, k)


@pytest.mark.parametrize("k", [0, 3])
def test_a_row_that_grows(k):
    """A lane's reference passes 2^20 on its way: what was summed against the smaller one joins the larger."""
    import torch
    say(f"logprobs of growing rows k={k}")
    V, beta = 60000, 64.0
    x = torch.linspace(0, 20000, V, device="cuda")[None].repeat(4, 1)
    x[1] = x[1].flip(0)
    x[2, ::2] = -math.inf
    x[3] = 11357 + x[3] * 1e-6  # about 2^20 all the way
    check(x, beta, np.array([V - 1, 0, V - 1, V // 2]), k)
