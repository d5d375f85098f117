"""The plain definitions of tests/chunk_ref.py against what their rules fix."""
import numpy as np
import pytest

import chunk_ref as K
import q8_ref as R


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_differences_of_positions(interleaved):
    rng = np.random.default_rng(1)
    f = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    q, k = rng.normal(size=(1, 2, 24)), rng.normal(size=(1, 2, 24))
    a, b = K.turned(q, [7], f, interleaved), K.turned(k, [3], f, interleaved)
    c, d = K.turned(q, [1007], f, interleaved), K.turned(k, [1003], f, interleaved)
    assert np.allclose((a * b).sum(-1), (c * d).sum(-1))  # the product depends on 7 - 3
    assert np.allclose((a ** 2).sum(-1), (q ** 2).sum(-1)) and np.array_equal(a[..., 16:], q[..., 16:])
    assert np.array_equal(K.turned(q, [0], f, interleaved), q)


def test_draws_follow_the_row():
    p = np.array([0.0, 0.25, 0.0, 0.5, 0.125, 0.125, 0.0], np.float32)
    grid = (np.arange(4096) + 0.5) / 4096
    got = np.bincount([K.draw(p, u) for u in grid], minlength=7) / 4096
    assert np.allclose(got, p, atol=1e-3)
    assert K.draw(p, 0.0) == 1 and K.draw(p, 0.25) == 3 and K.draw(p, np.nextafter(0.25, 0)) == 1
    assert K.draw(p, 1.0) == 5 and K.draw(p, 2.0) == 5 and K.draw(p, -1.0) == 1 and K.draw(p, float("nan")) == 1
    assert K.draw(np.zeros(4), 0.5) == -1 and K.draw([-1.0, np.nan, 1.0], 0.3) == 2 and K.draw([2.0, 1.0], 0.5) == 1
    assert K.draw(p / 3, 0.26) == K.draw(p, 0.26)


def test_drawn_tokens_of_a_tree_follow_the_target():
    """The first token of a round, accepted or not, has the root row's distribution."""
    rng = np.random.default_rng(3)
    p = rng.dirichlet(np.ones(6), (1, 4)).astype(np.float32)
    cand, parent = np.array([[5, 2, 4, 1]], np.int32), np.array([-1, 0, 0, 1])
    first = np.zeros(6)
    for _ in range(4000):
        u = rng.random((1, 3)).astype(np.float32)
        r = K.verify(p, cand, parent, u, 2)
        first[cand[0, r["path_nodes"][0, 1]] if r["accept_len"][0] else r["next_tok"][0]] += 1
    assert np.abs(first / 4000 - p[0, 0]).max() < 0.035  # 4 deviations of at most 0.5 / sqrt(4000)


def test_an_appended_page_holds_the_turned_rows():
    rng = np.random.default_rng(5)
    Hkv, P, D = 2, 16, 64
    f = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    z = np.zeros((4, Hkv, P, D), np.uint8), np.zeros((4, Hkv), np.float32)
    k, v = rng.normal(size=(1, 20, Hkv, D)), rng.normal(size=(1, 20, Hkv, D))
    kc, vc, ks, vs, L, n, slack, _ = K.append(k, v, z[0], z[0], z[1], z[1], np.array([[2, 0, -1]]), np.array([3], np.int32) * 0, f, False)
    assert L[0] == 20 and n[0] == 20
    got = np.concatenate([R.decode(kc[2]) * ks[2][:, None, None], R.decode(kc[0])[:, :4] * ks[0][:, None, None]], 1)
    want = K.turned(k[0], np.arange(20), f, False).transpose(1, 0, 2)
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + 2.0 ** -10 * ks.max()).all()
    assert slack[2].max() > 0 and slack[1].max() == 0


def test_chunk_rows_see_up_to_their_own_slot():
    rng = np.random.default_rng(7)
    P, D = 16, 64
    kp, vp = rng.integers(0, 120, (3, 1, P, D)).astype(np.uint8), rng.integers(0, 120, (3, 1, P, D)).astype(np.uint8)
    one = np.ones((3, 1), np.float32)
    q = rng.normal(size=(1, 4, 2, D)) * 0.01
    out, _, _ = K.attention(q, kp, vp, one, one, np.array([[0, 2]]), np.array([18]), np.array([2]), 0.01)
    v = np.concatenate([R.decode(vp[0, 0]), R.decode(vp[2, 0])])
    assert np.array_equal(out[0, 3], np.zeros((2, D)))
    z = np.concatenate([R.decode(kp[0, 0]), R.decode(kp[2, 0])]) @ q[0, 1, 0] * 0.01
    w = np.exp(z[:17] - z[:17].max())
    assert np.allclose(out[0, 1, 0], w @ v[:17] / w.sum())
