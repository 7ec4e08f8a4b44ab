"""moe_kv_append with index data that does not fit: flagged and skipped, the rest written."""

import numpy as np
import pytest
import torch

from tests import serving_ref as R
from tests.test_gpu_kv_append import _i32, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


def _append(moe, T, off, lens, table, good, pages=40):
    """The cache after a call of which the sequences `good` alone fit, compared with the rule."""
    g = torch.Generator().manual_seed(T)
    k, v = _rows((T, 2, 64), g), _rows((T, 2, 64), g)
    cache = moe.new_kv_cache(pages, 2, 16, 64)
    cache.codes.copy_(torch.randint(0, 127, cache.codes.shape, generator=g, dtype=torch.uint8))
    cache.scales.copy_(torch.randint(118, 132, cache.scales.shape, generator=g, dtype=torch.uint8))
    codes, scales = cache.codes[0].cpu().numpy().copy(), cache.scales[0].cpu().numpy().copy()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_kv_append(cache, 0, k.cuda(), v.cuda(), _i32(off), _i32(lens), _i32(table), ws=ws)
    status = moe.moe_get_device_status(ws)
    for s in good:
        R.append(codes, scales, k.double().numpy(), v.double().numpy(), off[s:s + 2], lens[s:s + 1],
                 np.asarray(table)[s:s + 1])
    assert np.array_equal(cache.codes[0].cpu().numpy(), codes)
    assert np.array_equal(cache.scales[0].cpu().numpy(), scales)
    return status


def _table(n, width=10):
    return np.arange(n * width).reshape(n, width)


def test_what_fits_is_not_flagged(moe):
    assert _append(moe, 60, [0, 20, 60], [25, 40], _table(2), [0, 1]) == moe.MOE_OK


@pytest.mark.parametrize("page", [-1, 40, 1 << 30])
def test_a_page_outside_the_pool(moe, page):
    """Skipped with its tokens; the sequence's other pages are written."""
    table = _table(2)
    table[1] = page
    assert _append(moe, 60, [0, 20, 60], [25, 40], table, [0]) == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("length", [-5, 39, 161, 1 << 30])
def test_a_length_that_does_not_fit(moe, length):
    """Shorter than the new tokens, negative, or past the table."""
    assert _append(moe, 60, [0, 20, 60], [25, length], _table(2), [0]) == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("T,off", [
    (60, [0, 20, 61]),                 # past T
    (60, [0, 20, 5]),                  # down
    (60, [0, 20, 1 << 30, 60]),
    (60, [0, 20, -60, -20]),
    (300, [0, 100, 4, 20]),            # far down: the next sequence starts before this one
    (300, [0, 150, 2, 160, 300]),
])
def test_offsets_that_do_not_fit(moe, T, off):
    """Flagged; nothing is written outside the pages of the sequences."""
    n = len(off) - 1
    g = torch.Generator().manual_seed(T)
    k, v = _rows((T, 2, 64), g), _rows((T, 2, 64), g)
    cache = moe.new_kv_cache(16 * n + 8, 2, 16, 64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = [max(1, b - a) + 3 if abs(b - a) <= T else 40 for a, b in zip(off, off[1:])]
    moe.moe_kv_append(cache, 0, k.cuda(), v.cuda(), _i32(off), _i32(lens),
                      _i32(4 + _table(n, 16)), ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert cache.codes[0, :4].eq(0).all() and cache.codes[0, 16 * n + 4:].eq(0).all()


@pytest.mark.parametrize("new", [1, 5])
def test_the_last_positions_there_are(moe, new):
    """A table of 2^31 positions (pages shared by many entries), written at its end."""
    last = (1 << 31) - 1
    g = torch.Generator().manual_seed(9)
    k, v = _rows((new, 1, 64), g), _rows((new, 1, 64), g)
    cache = moe.new_kv_cache(3, 1, 128, 64)
    table = torch.full((1, 1 << 24), 1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_kv_append(cache, 0, k.cuda(), v.cuda(), _i32([0, new]), _i32([last]), table, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    codes = np.zeros((3, 2, 1, 128, 64), np.uint8)
    scales = np.zeros((3, 2, 1, 8), np.uint8)
    R.append(codes, scales, k.double().numpy(), v.double().numpy(), [0, new], [127], np.array([[1]]))
    assert np.array_equal(cache.codes[0].cpu().numpy(), codes)
    assert np.array_equal(cache.scales[0].cpu().numpy(), scales)
