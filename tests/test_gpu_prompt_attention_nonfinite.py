"""moe_prompt_attention where keys and values hold NaN or infinities that rows see: these give what they
give, without the rows being computed again one by one, and what rows do not see has no effect."""

import numpy as np
import pytest
import torch

from tests import serving_ref as R
from tests.test_gpu_prompt_attention import _offsets, _qkv, _rows

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


def _run(moe, q, k, v, lens, bound_ms=20):
    """With a short bound on the kernel's waits: no warp may keep the others waiting that long."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    try:
        moe.moe_set_wait_timeout_ns(bound_ms * 1000000)
        out, lse = moe.moe_prompt_attention(q.cuda(), k.cuda(), v.cuda(),
                                            torch.from_numpy(_offsets(lens)).cuda(), ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_OK
    finally:
        moe.moe_set_wait_timeout_ns(0)
    return out, lse


def _check(moe, q, k, v, lens, keep):
    out, lse = _run(moe, q, k, v, lens)
    with np.errstate(invalid="ignore", over="ignore"):
        R.check_rows(out, lse, _rows(q, k, v, lens, lambda s, i: i in keep), q.shape[2] ** -0.5)
    return out, lse


def _keep(n, *at):
    near = {a + d for a in at for d in (-129, -128, -127, -65, -2, -1, 0, 1, 2, 64, 127, 128)}
    return {i for i in near | {0, 1, n - 2, n - 1} if 0 <= i < n}


@pytest.mark.parametrize("H,K,D", [(8, 1, 128), (2, 2, 64), (3, 1, 128)])
def test_a_nan_that_all_rows_see(moe, H, K, D):
    n = 4000
    q, k, v = _qkv(n, H, K, D, seed=D)
    v[0, 0, 5] = NAN
    out, _ = _check(moe, q, k, v, [n], _keep(n, 0, 2000))
    bad = torch.isnan(out.float()).cpu()
    assert bad[:, :H // K, 5].all() and int(bad.sum()) == n * (H // K)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_all_values_the_same(moe, D, value):
    """Each row's result is that value, also where later ones meet it with a weight of zero."""
    n = 3000
    q, k, v = _qkv(n, 8, 1, D, seed=1)
    v[:] = value
    out, lse = _run(moe, q, k, v, [n])
    assert (out.float().isnan() if value != value else out.float() == value).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,K", [(8, 1), (2, 2), (7, 1)])
def test_here_and_there(moe, H, K, D):
    """Columns that hold a NaN or an infinity from some key on, infinities of both signs, and a NaN
    that rows do not see in a column where they see an infinity."""
    n = 1500
    at = {0: (700, NAN), 3: (701, INF), 9: (130, -INF), 17: (1499, NAN), 20: (0, INF), 21: (640, NAN)}
    q, k, v = _qkv(n, H, K, D, seed=H + D)
    for c, (t, x) in at.items():
        v[t, :, c] = x
    v[100, :, 30], v[710, :, 30] = INF, -INF
    v[660, :, 31], v[700, :, 31] = INF, NAN
    v[1000:, 0, 40] = INF
    _check(moe, q, k, v, [n], _keep(n, 0, 100, 130, 640, 660, 700, 710, 1000))


def test_the_next_sequence(moe):
    """A sequence is what it is without the next one, whose values are all NaN."""
    lens = [3001, 500, 77]
    q, k, v = _qkv(sum(lens), 8, 1, 128, seed=3)
    ref, _ = _run(moe, q[:3001], k[:3001], v[:3001], [3001])
    v[3001:3501] = NAN
    out, lse = _run(moe, q, k, v, lens)
    R.check_rows(out, lse, _rows(q, k, v, lens, lambda s, i: s != 1 and (s == 2 or i > 2940)),
                 128 ** -0.5)
    assert torch.equal(out[:2800], ref[:2800])
    assert out[3001:3501].float().isnan().all()


def test_scores_that_are_not_finite(moe):
    """A NaN key reaches every row that sees it, whole."""
    n = 2000
    q, k, v = _qkv(n, 8, 1, 128, seed=4)
    k[300, 0, 3] = NAN
    out, lse = _check(moe, q, k, v, [n], _keep(n, 300))
    assert out[300:].float().isnan().all() and lse[300:].isnan().all()
    assert torch.isfinite(out[:300].float()).all()


def test_a_long_prompt_of_nan(moe):
    """Every value NaN, 8192 tokens of 64 heads: a few times the usual time, not thousands."""
    n = 8192
    q, k, v = [t.cuda() for t in _qkv(n, 64, 8, 128, seed=5)]
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def time():
        moe.moe_prompt_attention(q, k, v, off, ws=ws)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out, _ = moe.moe_prompt_attention(q, k, v, off, ws=ws)
        b.record()
        b.synchronize()
        return a.elapsed_time(b), out

    usual, _ = time()
    v[0] = NAN
    one, out = time()
    assert out.float().isnan().all()
    v[:] = NAN
    every, out = time()
    assert out.float().isnan().all()
    print(f"usual {usual:.3f} ms, NaN in the first token {one:.3f} ms, everywhere {every:.3f} ms")
    assert one < 3 * usual and every < 30 * usual
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
