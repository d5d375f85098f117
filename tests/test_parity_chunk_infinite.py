"""GPU parity of the chunk attention of queries with an infinity: a row that sees a key is NaN, whatever the
signs of its scores."""
import numpy as np
import pytest

from test_parity_chunk import attend, case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,prefix", [
    (1, 1, 2, 1, 64, 16, [0]), (2, 2, 4, 2, 128, 16, [5, 0]), (2, 1, 4, 4, 64, 16, [900, 30]), (1, 70, 4, 1, 128, 32, [1500]),
])
@pytest.mark.filterwarnings("ignore:invalid value")
def test_scores_that_are_all_minus_infinity(medusa, B, T, Hq, Hkv, D, P, prefix, dtype):
    c = case(B + T, B, T, Hq, Hkv, D, P, prefix, None, dtype)
    c["k_pages"] |= 0x80           # every code of K negative,
    c["k_pages"][c["k_pages"] == 0x80] = 0x81  # none of them zero
    c["q"] = np.abs(c["q"])
    c["q"][0, T - 1, 1, 3], c["q"][0, 0, 0, 5] = np.inf, np.inf
    got = attend(medusa, c)
    assert np.isnan(got[0, T - 1, 1]).all() and np.isnan(got[0, 0, 0]).all()
    check(c, got)
