"""moe_kv_attention with index data that does not fit: flagged, and what it names takes no part.
The batch's other sequences get what they get without it."""

import numpy as np
import pytest
import torch

from tests import serving_ref as R
from tests.test_gpu_kv_attention import Case, _i32

pytestmark = pytest.mark.gpu

ways = pytest.mark.parametrize("H,K,D,width", [(h, k, d, w) for h, k in ((4, 1), (16, 2), (16, 1))
                                               for d in (64, 128) for w in (0, 400)])


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


@ways
@pytest.mark.parametrize("page", [16, 32, 128])
def test_pages_outside_the_pool(moe, H, K, D, width, page):
    """Their keys are not seen; a sequence with no other gives zeros."""
    lens, new = [700, 40, 300, 13, 1000], [2, 2, 2, 2, 2]
    c = Case(moe, lens, new, H, K, D, page, seed=page, width=width)
    rows = c.rows()
    bad = {0: [0, 3], 2: [300 // page], 3: [0], 4: [1, 2, 5]}
    for s, pages in bad.items():
        for i, p in enumerate(pages):
            c.table[s, p] = (-1, c.codes.shape[1], 10 ** 6)[i % 3]
        for r in (2 * s, 2 * s + 1):
            for h in range(H):
                q, k, v, seen = rows[r, h]
                rows[r, h] = (q, k, v, seen & ~np.isin(np.arange(len(seen)) // page, pages))
    out, lse = c.run(status=moe.MOE_ERR_DEVICE_CHECK)
    R.check_rows(out, lse, rows, c.scale)
    assert out[6:8].eq(0).all() and lse[6:8].eq(-float("inf")).all()
    for _ in range(3):  # nothing left over from other sequences or launches
        again = c.run(status=moe.MOE_ERR_DEVICE_CHECK)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@ways
@pytest.mark.parametrize("length", [-1, 1 << 30])
def test_lengths_that_do_not_fit(moe, H, K, D, width, length):
    """Negative, or past the block table: the sequence sees nothing."""
    c = Case(moe, [100, 60, 33], [2, 2, 2], H, K, D, 16, seed=1, width=width)
    rows = {r: x for r, x in c.rows().items() if r[0] not in (2, 3)}
    c.lens = [100, length, 33]
    out, lse = c.run(status=moe.MOE_ERR_DEVICE_CHECK)
    R.check_rows(out, lse, rows, c.scale)
    assert out[2:4].eq(0).all() and lse[2:4].eq(-float("inf")).all()


@ways
def test_offsets_that_do_not_fit(moe, H, K, D, width):
    """The rows of a sequence whose offsets go down or leave the batch stay as they were."""
    c = Case(moe, [100, 60, 33], [2, 2, 2], H, K, D, 16, seed=2, width=width)
    rows = {r: x for r, x in c.rows().items() if r[0] < 2}
    for off in ([0, 2, 1, 7], [0, 2, -4, -2], [0, 2, 9, 6]):
        c.off = np.array(off, np.int32)
        out = torch.full((6, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((6, H), 7.0, device="cuda")
        c.run(status=moe.MOE_ERR_DEVICE_CHECK, out=out, lse=lse)
        R.check_rows(out, lse, rows, c.scale)
        assert out[2:].eq(7).all() and lse[2:].eq(7).all()
