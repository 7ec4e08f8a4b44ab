"""moe_kv_attention again and again on one cache: the results are the same bits every time.  The cache
fits L2, so that data arrive early and what is read late in a slot of a ring would be the next load's."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,length,H,K,D,page,new", [
    (16, 8192, 48, 2, 128, 128, 1), (64, 4096, 32, 1, 128, 16, 1), (16, 8192, 64, 4, 128, 32, 3),  # 32 rows
    (16, 8192, 32, 2, 128, 64, 1), (64, 2048, 16, 2, 128, 16, 2),                                  # 16
    (16, 8192, 16, 2, 128, 128, 1), (64, 2048, 8, 2, 128, 16, 1),                                  # 8
    (16, 8192, 64, 2, 64, 64, 1), (16, 8192, 32, 2, 64, 16, 1), (64, 2048, 8, 2, 64, 32, 1),
    (4, 1024, 64, 2, 64, 16, 1), (4, 1500, 8, 1, 128, 16, 1)])                                     # a CTA a unit
def test_the_same_bits(moe, n, length, H, K, D, page, new):
    g = torch.Generator(device="cuda").manual_seed(n + H)
    width = -(-length // page)
    codes = torch.randint(0, 120, (1, n * width, 2, K, page, D), generator=g, dtype=torch.uint8,
                          device="cuda")
    scales = torch.randint(117, 120, (1, n * width, 2, K, page // 16), generator=g,
                           dtype=torch.uint8, device="cuda")
    cache = moe.KvCache(codes, scales)
    q = (0.1 * torch.randn((n * new, H, D), generator=g, device="cuda")).to(torch.bfloat16)
    table = torch.arange(n * width, dtype=torch.int32, device="cuda").view(n, -1)
    args = (q, cache, 0, _i32([new * i for i in range(n + 1)]), _i32([length] * n), table)
    ws = moe.new_kv_attention_workspace(q, cache, table)
    runs = [moe.moe_kv_attention(*args, ws=ws) for _ in range(25)]
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
