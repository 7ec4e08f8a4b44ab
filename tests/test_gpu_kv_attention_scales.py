"""moe_kv_attention over value blocks whose scales lie far apart: no block's scale takes bits from
another block's weights, least of all that of a block which a row does not see.

Blocks are 16 keys.  The cases are given by the query rows that a sequence and KV head have: 8, 16
and 32 of them go different ways, as does a wide block table (the work dealt out over the grid) from
a narrow one (few units: a CTA each)."""

import numpy as np
import pytest
import torch

from tests import serving_ref as R
from tests.test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu

# (heads, KV heads): with the 2 new tokens of most cases 8, 16 and 32 rows
GROUPS = [(4, 1), (16, 2), (16, 1)]
ways = pytest.mark.parametrize("H,K,D,width", [(h, k, d, w) for h, k in GROUPS for d in (64, 128)
                                               for w in (0, 400)])
LENS = [17, 49, 33, 161, 1601, 2305]     # the second of two new tokens begins a block


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_20_gb300 import binding
    return binding


def _place(c, s, block):
    page = c.codes.shape[4]
    return c.table[s, block * 16 // page], block * 16 % page


def _value_scale(c, s, block, byte):
    p, at = _place(c, s, block)
    c.scales[c.layer, p, 1, :, at // 16] = byte


def _values(c, s, block):
    """The codes [heads, 16, dim] of a block's values."""
    p, at = _place(c, s, block)
    return c.codes[c.layer, p, 1, :, at:at + 16]


def _score(c, s, block, below):
    """Every key of the block scores `below` under zero (and no more than that)."""
    p, at = _place(c, s, block)
    c.q[:, :, 0] = 8.0
    c.codes[c.layer, p, 0, :, at:at + 16] = 0
    code = int(R.encode(np.array([-below / (8.0 * c.scale)]))[0])
    c.codes[c.layer, p, 0, :, at:at + 16, 0] = code
    c.scales[c.layer, p, 0, :, at // 16] = 127


def _level(c):
    """Keys that do not look at the column that _score uses."""
    c.codes[c.layer, :, 0, :, :, 0] = 0


def _check(c, pick=lambda r: True):
    """Rows against 64 bits, to 11 bits of the weights.  An f16 weight is off by 2^-11 of itself, or
    by 2^-25 in units where the row's largest is at least 2^2 (2^6, less 4 binary orders between
    blocks that share a unit): 2^-27 of the largest for each key.  The result is rounded to bf16,
    off by 2^-8 of itself."""
    out, lse = c.run()
    out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    n = 0
    for (r, h), (q, k, v, seen) in c.rows().items():
        if not pick(r):
            continue
        n += 1
        o, z = R.attention(q, k, v, seen, c.scale)
        eo, ez = R.attention_bounds(q, k, v, seen, c.scale)
        kk, vv = k[seen], v[seen]
        s = (kk @ q) * c.scale
        e = np.exp(s - s.max())
        p = e / e.sum()
        eo = eo - (2.0 ** -8 - 2.0 ** -11) * (p @ np.abs(vv)) + 2.0 ** -27 * np.abs(vv).sum(0) / e.sum()
        bound = 1.02 * eo + 2.0 ** -8 * (np.abs(o) + eo) + 1e-36
        bad = ~(np.abs(out[r, h] - o) <= bound)
        assert not bad.any(), (f"row {r} head {h}: {out[r, h][bad][:4]} != {o[bad][:4]} "
                               f"+- {bound[bad][:4]}")
        assert abs(lse[r, h] - z) <= ez, f"row {r} head {h}: lse {lse[r, h]} != {z} +- {ez}"
    assert n


@ways
@pytest.mark.parametrize("up", [5, 24, 40, 126])
def test_a_later_draft_with_large_values(moe, H, K, D, width, up):
    """The second draft lies alone in a block, its values 2^up above the others' (126: what an
    infinity is stored as).  The first does not see it."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=up, width=width)
    for s, n in enumerate(LENS):
        _value_scale(c, s, n // 16, 121 + up)
        _values(c, s, n // 16)[:, 0] = 0x7E
    _check(c, lambda r: up < 126 or r % 2 == 0)


@ways
@pytest.mark.parametrize("below,up", [(200.0, 40), (200.0, 100), (28.0, 40), (28.0, 20), (90.0, 110)])
def test_large_values_of_little_weight(moe, H, K, D, width, below, up):
    """A block that all rows see, at the start, in the middle or near the end, whose values are large
    and whose weight is next to nothing (e^-28 2^40 is the size of the rest)."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=int(below) + up, width=width)
    _level(c)
    for s, n in enumerate(LENS):
        at = (0, n // 32, max(0, n // 16 - 2))[s % 3]
        _value_scale(c, s, at, 121 + up)
        _score(c, s, at, below)
    _check(c)


@ways
@pytest.mark.parametrize("up", [8, 30, 60])
def test_large_values_in_some_columns(moe, H, K, D, width, up):
    """Blocks of ordinary weight with large values in two columns, zeros in the others: these keep
    what the ordinary blocks give them."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=up, width=width)
    for s, n in enumerate(LENS):
        for at in range(s % 2, n // 16, 5):
            _value_scale(c, s, at, 121 + up)
            v = _values(c, s, at)
            keep = v[..., [3, D - 2]].copy()
            v[:] = 0
            v[..., [3, D - 2]] = keep
    _check(c)


@ways
@pytest.mark.parametrize("low,high", [(112, 124), (60, 190), (1, 110), (0, 120)])
def test_each_block_its_scale_and_columns(moe, H, K, D, width, low, high):
    """Every block's scale is drawn by itself; the columns belong to four kinds of block."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=low + high, width=width)
    rng = np.random.RandomState(low)
    kinds = np.linspace(low, high, 4).astype(int)
    for s, n in enumerate(LENS):
        for at in range(-(-n // 16)):
            kind = rng.randint(4)
            _value_scale(c, s, at, kinds[kind])
            v = _values(c, s, at)
            v[..., np.arange(D) % 4 != kind] = 0
    _check(c)


@ways
@pytest.mark.parametrize("step", [1, -1, 9, -9])
def test_scales_that_drift(moe, H, K, D, width, step):
    """Scales that rise or fall all along the keys."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=step + 10, width=width)
    for s, n in enumerate(LENS):
        blocks = -(-n // 16)
        for at in range(blocks):
            _value_scale(c, s, at, int(np.clip(121 + step * (at - blocks // 2), 1, 230)))
    _check(c)


@ways
def test_blocks_of_zeros(moe, H, K, D, width):
    """Zero values have the smallest scale byte there is."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=2, width=width)
    for s, n in enumerate(LENS):
        for at in range(s % 3, -(-n // 16), 3):
            _value_scale(c, s, at, 0)
            _values(c, s, at)[:] = 0
    _check(c)


@ways
def test_not_a_number_beside_large_values(moe, H, K, D, width):
    """The second draft's values are NaN in some columns and large in others."""
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=3, width=width)
    for s, n in enumerate(LENS):
        _value_scale(c, s, n // 16, 170)
        _values(c, s, n // 16)[:, 0, 1::7] = 0x7F
    _check(c, lambda r: r % 2 == 0)
    out, _ = c.run()
    bad = torch.isnan(out.float()).cpu().numpy()
    assert not bad[0::2].any() and bad[1::2, :, 1::7].all()
    assert bad[1::2].sum() == bad[1::2, :, 1::7].size


@ways
def test_results_repeat(moe, H, K, D, width):
    c = Case(moe, LENS, [2] * len(LENS), H, K, D, 16, seed=4, width=width, spread=14)
    one = c.run()
    for _ in range(3):
        two = c.run()
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("H", [8, 32, 48])
def test_a_wait_that_gives_up(moe, H):
    """With scales far apart and a bound of 1 ns: the call ends, the next one is as before."""
    n, length, page = 16, 1 << 15, 128
    g = torch.Generator(device="cuda").manual_seed(H)
    pages = n * length // page
    codes = torch.randint(0, 120, (1, pages, 2, 2, page, 128), generator=g, dtype=torch.uint8,
                          device="cuda")
    scales = torch.full((1, pages, 2, 2, page // 16), 118, dtype=torch.uint8, device="cuda")
    scales[:, :, 1] += 12 * torch.randint(0, 2, scales[:, :, 1].shape, generator=g, dtype=torch.uint8,
                                          device="cuda")
    cache = moe.KvCache(codes, scales)
    q = (0.1 * torch.randn((n, H, 128), generator=g, device="cuda")).to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(n, -1)
    off, lens = (torch.tensor(v, dtype=torch.int32, device="cuda")
                 for v in (list(range(n + 1)), [length] * n))
    ws = moe.new_kv_attention_workspace(q, cache, table)
    ref = moe.moe_kv_attention(q, cache, 0, off, lens, table, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    try:
        moe.moe_set_wait_timeout_ns(1)
        moe.moe_kv_attention(q, cache, 0, off, lens, table, ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_TIMEOUT
    finally:
        moe.moe_set_wait_timeout_ns(0)
    again = moe.moe_kv_attention(q, cache, 0, off, lens, table, ws=ws)
    assert torch.equal(ref[0], again[0]) and torch.equal(ref[1], again[1])
