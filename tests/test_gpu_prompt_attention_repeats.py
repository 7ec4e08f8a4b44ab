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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [3, 5, 7, 40, 100, 8, 128])
def test_each_sequence_by_itself(moe, G, D):
    """A sequence's bits do not depend on the other sequences, nor on what was computed before: also
    where a group does not fill its rows of a tile."""
    lens = [137, 1, 387, 558, 280, 3, 278]
    g = torch.Generator(device="cuda").manual_seed(G + D)
    q, k, v = ((2.5 * torch.randn((sum(lens), h, D), generator=g, device="cuda")).to(torch.bfloat16)
               for h in (G, 1, 1))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(i, j):
        a, b = sum(lens[:i]), sum(lens[:j])
        off = torch.tensor(np.cumsum([0] + lens[i:j]), dtype=torch.int32, device="cuda")
        return moe.moe_prompt_attention(q[a:b], k[a:b], v[a:b], off, ws=ws)

    out, lse = run(0, len(lens))
    for _ in range(5):
        again = run(0, len(lens))
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    for i, n in enumerate(lens):
        a = sum(lens[:i])
        alone = run(i, i + 1)
        assert torch.equal(alone[0], out[a:a + n]) and torch.equal(alone[1], lse[a:a + n])
