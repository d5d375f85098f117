"""GPU parity of the rotation's angles, where a sine is small enough for float32 to show them: to the
bound that include/medusa.h, part 6e, gives."""
import numpy as np
import pytest
import torch

from util import to_dev

pytestmark = pytest.mark.gpu

INV_2PI = np.longdouble("0.159154943091895335768883763372514362034459645740456448747667")


@pytest.mark.parametrize("start", [0, 900_000, -300_000, 2 ** 29])
def test_sines_near_zero(medusa, start):
    """(1, 0) turns to (cos, sin).  Below 2^-10 a sine's own roundings (of the angle to float32 twice, of the
    series' products and sums: at most 6 of 2^-24) are below 2^-31; a cut angle would be off by 2^-29.3."""
    T = 1 << 17
    f = np.array([1.0, 0.731, 3.3e-2, 5.9, 1e-3, 2.6, 0.25, 1.7], np.float32)
    x = np.zeros((1, T, 1, 16), np.float32)
    x[..., :8] = 1
    got, _ = medusa.rope_rows(to_dev(x), None, to_dev(np.array([start], np.int32)), to_dev(f))
    got = got.cpu().numpy()[0, :, 0].astype(np.float64)
    p = np.arange(start, start + T, dtype=np.int64)
    # (products with 24 bits are exact in 64; turns are then off by 2^-64 of themselves: 2^-36 at the far end)
    t = p.astype(np.longdouble)[:, None] * f.astype(np.longdouble) * INV_2PI
    angle = (t - np.round(t)).astype(np.float64) * 2 * np.pi
    bound = 2.0 ** -30 + np.abs(p)[:, None] * (2.0 ** -52 * f.astype(np.float64) + 2.0 ** -62)
    small = np.abs(np.sin(angle)) < 2.0 ** -10
    assert small.sum() > 300
    err = np.abs(got[:, 8:] - np.sin(angle))
    assert (err <= bound + 2.0 ** -31)[small].all()
    assert (np.abs(got[:, :8] - np.cos(angle)) <= bound + 4 * 2.0 ** -24).all()


def test_positions_wrap_as_int32(medusa):
    """kv_len + depth beyond 2^31 is the negative number that int32 makes of it."""
    x = torch.randn(1, 4, 2, 32, device="cuda")
    f = to_dev(np.linspace(0.1, 1, 16).astype(np.float32))
    a, _ = medusa.rope_rows(x, None, to_dev(np.array([2 ** 31 - 2], np.int32)), f)
    b, _ = medusa.rope_rows(x, None, to_dev(np.array([0], np.int32)), f, depth=to_dev(np.array([2 ** 31 - 2, 2 ** 31 - 1, -2 ** 31, 1 - 2 ** 31], np.int64).astype(np.int32)))
    assert torch.equal(a, b)
