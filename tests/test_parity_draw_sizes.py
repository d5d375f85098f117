"""GPU parity of drawn tokens where the way of drawing changes: on both sides of 20 MB of rows and of 1024
blocks for them, many nodes on a small vocabulary among them."""
import pytest

from test_parity_draw import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,V,kind", [
    (1, 40, 131072, "random"), (1, 41, 128256, "random"),    # 20 MB exactly; a little more
    (4, 9, 128256, "dense"), (2, 21, 128256, "dense"),       # 18 MB; 21 MB
    (16, 64, 40, "random"), (41, 25, 41, "random"),          # 1024 blocks; 1025
    (2, 341, 700, "dense"), (1, 341, 10000, "dense"), (3, 342, 500, "dense"),
    (2, 128, 20000, "random"), (1, 512, 10239, "random"), (1, 512, 10241, "random"),
    (300, 1, 1000, "chain"), (2, 1, 200001, "chain"),        # no tree: never walked
])
def test_tokens_and_paths(medusa, B, N, V, kind):
    c = case(B * 3 + N + V, B, N, V, kind, peak=6.0)
    check(c, run(medusa, c))
