"""GPU tests of the paged tree attention: a row that sees a tree row whose V is not finite
is NaN, wherever that row stands in the tree and whatever the scores behind it."""
import numpy as np
import pytest

import q8_ref as R
from test_parity_q8 import as_dtype, attend, attention_case, reference, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["chain", "random"])
@pytest.mark.parametrize("N,D,L,bad,high", [(150, 64, 40, 0, 130), (150, 128, 300, 100, 129), (341, 64, 0, 5, 200),
                                            (341, 128, 700, 140, 300), (512, 64, 100, 0, 511)])
def test_a_bad_tree_row_marks_the_rows_that_see_it(medusa, N, D, L, bad, high, kind, dtype):
    """V of node `bad` holds an infinity, and the key of a node in a later tile scores about
    130 above the others: rows that see both are NaN all the same."""
    c = attention_case(N + L, 2, N, 2, 2, D, 32, [L, L // 2], dtype, kind)
    base = np.ones(D)
    c["q"] = as_dtype(base + 0.1 * c["q"], dtype)
    c["k_tree"][:, high] = 130 / (D * c["scale"])
    c["k_tree"] = as_dtype(c["k_tree"], dtype)
    ref = reference(c)
    c["v_tree"][0, bad, 1, 3] = -np.inf
    hurt = R.sees(c["mask"], N)[:, bad]
    got = attend(medusa, c)
    assert np.isnan(got[0, hurt, 1]).all()
    got[0, hurt, 1] = ref[0][0, hurt, 1]
    tol = tolerance(c, ref)
    assert (np.abs(got - ref[0]) <= tol).all()
