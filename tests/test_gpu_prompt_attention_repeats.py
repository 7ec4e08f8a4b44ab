"""moe_prompt_attention again and again on the same prompts: the same bits every time."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


@pytest.mark.parametrize("low,high,n,H,K,D", [(0, 21, 4096, 32, 4, 128), (0, 21, 4096, 32, 4, 64),
                                              (1, 400, 300, 32, 8, 128), (100, 1200, 11, 64, 4, 128)])
def test_the_same_bits(moe, low, high, n, H, K, D):
    lens = np.random.RandomState(n).randint(low, high, n)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn((int(lens.sum()), h, D), generator=g, device="cuda").to(torch.bfloat16)
               for h in (H, K, K))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out, lse = moe.moe_prompt_attention(q, k, v, off, ws=ws)
    for _ in range(30):
        again = moe.moe_prompt_attention(q, k, v, off, ws=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
