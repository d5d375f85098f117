"""GPU parity of the rotation of tree and chunk rows against its definition in float64."""
import numpy as np
import pytest
import torch

import chunk_ref as K
from test_parity_q8 import as_dtype, dev
from util import to_dev

pytestmark = pytest.mark.gpu


def freqs(n, base=10000.0):
    return (base ** (-np.arange(n) / n)).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,n,lens,depth", [
    (1, 1, 1, 1, 64, 32, [0], None),
    (2, 9, 4, 2, 64, 16, [1048576, 5], "tree"),
    (3, 64, 5, 5, 128, 64, [100, 0, 70001], "tree"),
    (1, 341, 40, 40, 128, 32, [999999], "tree"),
    (2, 300, 7, 1, 128, 64, [17, 4000], None),
    (2, 33, 3, 0, 80, 40, [17, 4000], None),
    (1, 5, 2, 1, 512, 256, [2 ** 29 - 10], None),
    (64, 3, 2, 2, 16, 8, list(range(64)), None),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_turn_by_their_positions(medusa, B, T, Hq, Hkv, D, n, lens, depth, interleaved, dtype):
    rng = np.random.default_rng(B * 1000 + T)
    f = freqs(n)
    q, k = (as_dtype(rng.normal(0, 1, (B, T, h, D)), dtype) for h in (Hq, Hkv))
    d = np.minimum(rng.integers(0, 6, T), np.arange(T)).astype(np.int32) if depth else None
    out = medusa.rope_rows(dev(q, dtype), dev(k, dtype) if Hkv else None, to_dev(np.array(lens, np.int32)), to_dev(f),
                           depth=to_dev(d) if depth else None, interleaved=interleaved)
    torch.cuda.synchronize()
    for x, got in ((q, out[0]), (k, out[1])):
        if not x.shape[2]:
            assert got is None
            continue
        got = got.double().cpu().numpy()
        for b in range(B):
            want = K.turned(x[b], lens[b] + (d if depth else np.arange(T)), f, interleaved)
            # the rounding to the type, and float32's own; an angle is off by another 2^-30 at a million tokens and by
            # 2 pi * 2^29 * 2^-53 = 2^-21.3 at half a billion
            far = (np.abs(x[b]).max() * 2 * 2.0 ** -21) if max(lens) > 2 ** 24 else 0
            tol = K.turn_error(x[b], n, interleaved) + far
            tol = tol * (1 + 2.0 ** -8) + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 0)
            assert (np.abs(got[b] - want) <= tol).all()
            assert np.array_equal(got[b][..., 2 * n:], x[b][..., 2 * n:])


def test_in_place_and_given_outputs_are_the_same_bits(medusa):
    rng = np.random.default_rng(3)
    q, k, f, L = dev(rng.normal(0, 1, (2, 40, 8, 128)), "bf16"), dev(rng.normal(0, 1, (2, 40, 2, 128)), "bf16"), to_dev(freqs(64)), to_dev(np.array([5, 900], np.int32))
    a, b = medusa.rope_rows(q, k, L, f)
    o = torch.zeros_like(q), torch.zeros_like(k)
    assert medusa.rope_rows(q, k, L, f, out=o)[0] is o[0]
    assert torch.equal(a, o[0]) and torch.equal(b, o[1])
    medusa.rope_rows(q, k, L, f, out=(q, k))
    assert torch.equal(a, q) and torch.equal(b, k)


def test_frequencies_of_any_size_and_sign(medusa):
    """Whole turns per position do not matter, however many."""
    f = np.array([6.2, 100.0, -0.3, 1e-7, 0.0, 1000.5, -7.0, 3.14159], np.float32)
    x = np.random.default_rng(4).normal(0, 1, (1, 50, 2, 16)).astype(np.float32).astype(np.float64)
    got, _ = medusa.rope_rows(dev(x, "f32"), None, to_dev(np.array([1000], np.int32)), to_dev(f))
    want = K.turned(x[0], 1000 + np.arange(50), f, False)
    # 2 pi * 1050 * 1000.5 / 2 pi * 2^-53 of a turn is below 2^-30
    assert (np.abs(got[0].double().cpu().numpy() - want) <= K.turn_error(x[0], 8, False) + 2.0 ** -28).all()


def test_values_that_are_not_finite_stay_in_their_pair(medusa):
    x = np.ones((1, 1, 1, 64), np.float32)
    x[..., 3], x[..., 40] = np.inf, np.nan
    got, _ = medusa.rope_rows(to_dev(x), None, to_dev(np.array([2], np.int32)), to_dev(freqs(32)))
    g = got.cpu().numpy()[0, 0, 0]
    assert np.isinf(g[3]) and np.isinf(g[35]) and np.isnan(g[8]) and np.isnan(g[40])
    assert np.isfinite(np.delete(g, [3, 35, 8, 40])).all()
