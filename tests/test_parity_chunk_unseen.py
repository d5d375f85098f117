"""GPU parity of the chunk attention of rows that see no key although pages behind them are there: zero,
whatever the query holds."""
import numpy as np
import pytest

import chunk_ref as K
from test_parity_chunk import NAMES, attend, case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,P", [
    (24, 4, 2, 64, 16),    # one tile, two streams of which one has it
    (300, 4, 2, 128, 32),  # blocks of 256 rows, the streams share tiles
    (60, 34, 2, 64, 16),   # 17 query heads a KV head
])
def test_rows_in_front_of_the_first_page_that_is_there(medusa, T, Hq, Hkv, D, P, dtype):
    """The first page of all is absent: the rows of its slots see nothing, those behind it see their own
    page on; the keys of the pages that are there lie in the same tile."""
    c = case(T, 2, T, Hq, Hkv, D, P, [0, 3], None, dtype)
    c["table"][:, 0] = -1
    good = c["q"].copy()
    c["q"][:, :P - 4] = np.nan
    c["q"][1, T - 1, 2] = np.inf
    ref = K.attention(good, *(c[n] for n in NAMES), c["table"], c["kv_len"], None, c["scale"])
    tol = K.attention_tolerance(good, c["k_pages"], c["table"], c["kv_len"], c["v_scale"], ref, dtype == "bf16")
    got = attend(medusa, c)
    bad = np.zeros(got.shape, bool)
    bad[1, T - 1, 2] = True
    assert not got[0, :P].any() and not got[1, :P - 3].any() and got[0, P].any()
    assert np.array_equal(np.isnan(got), bad)
    assert (bad | (np.abs(np.nan_to_num(got) - ref[0]) <= tol)).all()
    c["q"] = good
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_units_cut_over_many_blocks(medusa, dtype):
    """No page is there, then a far one alone: rows that are not finite are zero, then NaN."""
    c = case(9, 1, 6, 8, 2, 128, 16, [7000], None, dtype)
    page = c["table"][0, 200]
    c["table"][:] = -1
    good = c["q"].copy()
    c["q"][0, 2, 3, 0], c["q"][0, 5, 7, 9] = np.nan, -np.inf
    assert not attend(medusa, c).any()
    c["table"][0, 200] = page
    bad = np.zeros(good.shape, bool)
    bad[0, 2, 3] = bad[0, 5, 7] = True
    assert np.array_equal(np.isnan(attend(medusa, c)), bad)
    c["q"] = good
    check(c, attend(medusa, c))
