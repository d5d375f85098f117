"""Which random number a node's draw takes: that of its steps from the root, whatever way the rows are
drawn from and whatever the depth array holds."""
import numpy as np
import pytest

from test_parity_draw import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wrong", ["zero", "reversed", "far", "none"])
@pytest.mark.parametrize("B,N,V,kind", [
    (6, 30, 500, "dense"), (4, 64, 700, "chain"), (3, 512, 40, "chain"),  # drawn from all rows at once
    (3, 60, 32001, "dense"), (2, 50, 64000, "random"),                    # walked: 22 MB and more
])
def test_the_depth_array_does_not_choose_the_number(medusa, B, N, V, kind, wrong):
    c = case(B + N, B, N, V, kind, peak=9.0)
    d = c["depth"]
    c["depth"] = {"zero": np.zeros_like(d), "reversed": d[::-1].copy(), "far": d + 1000, "none": -1 - d}[wrong]
    got = run(medusa, c)
    assert got["accept_len"].max() > 0
    check(c, got)


def test_numbers_of_every_step_count(medusa):
    """A chain of which each row has weight on two tokens, its child's and another: u[b, d] alone says how
    far a walk gets, at every depth up to the last, and max_depth may cut the tree short."""
    N, V, B = 512, 16, 512
    p = np.zeros((B, N, V), np.float32)
    p[:, :, 3], p[:, :, 9] = 0.5, 0.5
    u = np.full((B, N), 0.25, np.float32)
    u[np.arange(B), np.arange(B)] = 0.75  # the number at which sequence b leaves the chain
    c = dict(probs=p, cand=np.full((B, N), 3, np.int32), parent=np.arange(N, dtype=np.int32) - 1, depth=np.arange(N, dtype=np.int32), u=u,
             max_depth=N - 1)
    got = run(medusa, c)
    assert np.array_equal(got["accept_len"], np.arange(B)) and (got["next_tok"] == 9).all()
    c.update(u=np.ascontiguousarray(u[:, :101]), max_depth=100)
    got = run(medusa, c)
    assert np.array_equal(got["accept_len"], np.minimum(np.arange(B), 100))
    assert np.array_equal(got["next_tok"], np.where(np.arange(B) <= 100, 9, 3))
