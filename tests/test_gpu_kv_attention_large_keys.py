"""moe_kv_attention where a later draft's key is infinite: its block's scale is then the largest there is
and the block's earlier keys are zeros (as moe_kv_append leaves them), which rows of large queries see."""

import numpy as np
import pytest
import torch

from tests import serving_ref as R
from tests.test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


@pytest.mark.parametrize("far", [0, 30])
@pytest.mark.parametrize("power", [0, 13, 60])
@pytest.mark.parametrize("H,K,D,width", [(h, k, d, w) for h, k in ((4, 1), (16, 2), (16, 1))
                                         for d in (64, 128) for w in (0, 400)])
def test_an_infinite_key_among_the_drafts(moe, H, K, D, width, power, far):
    """Queries of 2^power; `far`: values of a block 2^far above the others'."""
    lens = [20, 50, 171, 1610]
    c = Case(moe, lens, [2] * 4, H, K, D, 16, seed=power + H, width=width)
    c.q *= 2.0 ** power
    used = c.scales[0, :, 0] < 200
    c.scales[0, :, 0] = np.where(used, np.maximum(c.scales[0, :, 0].astype(int) - power, 1), 250)
    for s, n in enumerate(lens):
        p, at = c.table[s, (n - 1) // 16], (n - 1) % 16
        c.codes[0, p, 0, :, :at] = 0
        c.codes[0, p, 0, :, at] = 0x7E
        c.scales[0, p, 0] = 247
        c.scales[0, c.table[s, 0], 1] += far
    out, lse = c.run()
    rows = {r: x for r, x in c.rows().items() if r[0] % 2 == 0}
    R.check_rows(out, lse, rows, c.scale)
