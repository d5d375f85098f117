"""GPU parity of the append into pages whose scales the caller chose, no powers of two:
conversion is to the nearest code of value / scale, ties to even, and a row fits a page
where its largest value is at most 448 * scale -- both of the exact quotient and product,
not of a rounded one."""
import numpy as np
import pytest

import q8_ref as R
from test_parity_q8 import as_dtype, pool, run_append, same_pools

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", range(6))
def test_rows_next_to_ties(medusa, seed, dtype):
    """Values that lie next to the middle of two codes, times the page's scale."""
    rng = np.random.default_rng(seed)
    Hkv, D, P = 4, 64, 32
    pools = list(pool(rng, 2, Hkv, P, D))
    for i in (2, 3):
        pools[i] = rng.uniform(0.3, 3.0, pools[i].shape).astype(np.float32)
    grid = np.unique(R.VALUES[np.isfinite(R.VALUES) & (R.VALUES >= 0)])
    middle = (grid[1:] + grid[:-1]) / 2
    x = []
    for s in pools[2:]:
        t = rng.choice(middle, (Hkv, D)) * rng.choice([-1.0, 1.0], (Hkv, D)) * s[1].astype(np.float64)[:, None]
        x.append(as_dtype(t[None, None], dtype))
    table, kv_len = np.array([[1]], np.int32), np.array([7], np.int32)
    got, _, _, _ = run_append(medusa, pools, *x, dtype, table, kv_len)
    *want, _, _ = R.append(*x, *pools, table, kv_len)
    same_pools(got, want)


@pytest.mark.parametrize("seed", range(4))
def test_rows_that_just_fit_or_just_do_not(medusa, seed):
    rng = np.random.default_rng(seed)
    Hkv, D, P = 16, 64, 16
    pools = list(pool(rng, 2, Hkv, P, D))
    for i in (2, 3):
        pools[i] = rng.uniform(0.3, 3.0, pools[i].shape).astype(np.float32)
    x = []
    for s in pools[2:]:
        y = rng.normal(0, 1, (Hkv, D)).astype(np.float32)
        y[:, 9] = np.float32(448) * s[1]  # the product, rounded: above or below the exact one
        x.append(y.astype(np.float64)[None, None])
    table, kv_len = np.array([[1]], np.int32), np.array([5], np.int32)
    got, _, _, _ = run_append(medusa, pools, *x, "f32", table, kv_len)
    *want, _, _ = R.append(*x, *pools, table, kv_len)
    same_pools(got, want)


@pytest.mark.parametrize("seed", range(4))
def test_earlier_codes_move_to_the_new_grid(medusa, seed):
    """The new scale is a power of two, the old one was chosen so that codes times it lie
    next to the middle of two codes of the new grid."""
    rng = np.random.default_rng(seed)
    Hkv, D, P = 16, 128, 32
    pools = list(pool(rng, 2, Hkv, P, D))
    for i in (2, 3):  # c * s next to an odd number of sixteenths for a code c = 8..15
        c = rng.integers(8, 16, pools[i].shape)
        pools[i] = ((2 * rng.integers(8, 16, pools[i].shape) + 1) / 16.0 / c).astype(np.float32)
    x = [np.full((1, 1, Hkv, D), 2000.0) for _ in "kv"]
    table, kv_len = np.array([[1]], np.int32), np.array([30], np.int32)
    got, _, _, _ = run_append(medusa, pools, *x, "f32", table, kv_len)
    *want, _, _ = R.append(*x, *pools, table, kv_len)
    same_pools(got, want)
