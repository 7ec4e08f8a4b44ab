"""Index tensors of a wrong rank are refused by the binding of the serving calls."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("offsets", [[[0, 5]], [[0], [5]], [[0, 2, 5], [0, 3, 5]], 5, []])
def test_offsets_of_a_wrong_rank(moe, offsets):
    q, k = (torch.zeros((5, h, 64), dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    with pytest.raises(ValueError, match="seq_offsets"):
        moe.moe_prompt_attention(q, k, k, _i32(offsets))
    cache = moe.new_kv_cache(2, 1, 16, 64)
    for call, x in ((moe.moe_kv_append, (cache, 0, k, k)), (moe.moe_kv_attention, (q, cache, 0))):
        with pytest.raises(ValueError, match="seq_offsets"):
            call(*x, _i32(offsets), _i32([5]), _i32([[0]]))


@pytest.mark.parametrize("lens,table", [([[5]], [[0]]), ([5], [0]), ([5], [[[0]]]), ([5, 5], [[0]])])
def test_lengths_and_tables_of_a_wrong_shape(moe, lens, table):
    q, k = (torch.zeros((5, h, 64), dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    cache = moe.new_kv_cache(2, 1, 16, 64)
    for call, x in ((moe.moe_kv_append, (cache, 0, k, k)), (moe.moe_kv_attention, (q, cache, 0))):
        with pytest.raises(ValueError):
            call(*x, _i32([0, 5]), _i32(lens), _i32(table))
