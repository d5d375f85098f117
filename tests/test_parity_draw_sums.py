"""GPU parity of drawn tokens where a row's sums need more than float32's bits: entries that repeat (so
that roundings do not cancel), of every size, and numbers next to the boundaries."""
import numpy as np
import pytest
import torch

from util import to_dev

pytestmark = pytest.mark.gpu

V = 128256


def two_levels(first, second, n=V):
    return np.r_[np.full(n // 2, first, np.float32), np.full(n - n // 2, second, np.float32)]


def row_of(name):
    rng = np.random.default_rng(17)
    if name == "halves beside a large token":
        r = two_levels(1.1e-6, 1.3e-6)
        r[7] = 0
        r[7] = 1 - r.astype(np.float64).sum()
        return r
    if name == "one token of 0.9, a tail of two sizes":
        return np.r_[np.float32(0.9), two_levels(6.5e-7, 9.1e-7, V - 1)]
    if name == "halves scaled by 2^-10":
        return two_levels(1.1e-6, 1.3e-6) * np.float32(2.0 ** -10)
    if name == "random scaled by 1e-3":
        return ((0.5 + rng.random(V)) / V * 1e-3).astype(np.float32)
    return np.full(V, 0.7, np.float32)  # a sum far above 1


NAMES = ["halves beside a large token", "one token of 0.9, a tail of two sizes", "halves scaled by 2^-10", "random scaled by 1e-3",
         "every entry 0.7"]


def whole(row):
    """The row's running sums as whole numbers, exactly (the least entry's last bit is 1 or more)."""
    e = int(np.frexp(row[row > 0].min())[1])
    w = np.ldexp(row.astype(np.float64), 24 - e)
    assert (w == np.floor(w)).all() and w.sum() < 2.0 ** 62
    return np.cumsum(w.astype(np.int64))


def drawn(sums, u):
    """The smallest v whose sum lies above u * total, in whole numbers."""
    total, out = int(sums[-1]), []
    for x in u:
        num, den = float(x).as_integer_ratio()
        out.append(int(np.searchsorted(sums, num * total // den, side="right")))
    return np.array(out, np.int32)


def numbers(sums, count, rng):
    """float32 numbers beside boundaries, the nearest first, but not nearer than the 2^-37 of the total
    that the sums may be off by (2^-36 here), and as many anywhere."""
    total = int(sums[-1])
    at = sums[:-1] / total
    u = np.concatenate([at.astype(np.float32), np.nextafter(at.astype(np.float32), np.float32(1)), np.nextafter(at.astype(np.float32), np.float32(0))])
    # (the distance in float64 is off by 2^-53 of a number near 1: far less than what is asked for)
    far = np.abs(u.astype(np.float64) - np.concatenate([at, at, at]))
    ok = (far > 2.0 ** -36) & (u >= 0) & (u < 1)
    near = u[ok][np.argsort(far[ok], kind="stable")[:count]]
    return np.concatenate([near, rng.random(count, dtype=np.float32)])


@pytest.mark.parametrize("name", NAMES)
def test_single_rows(medusa, name):
    row = row_of(name)
    sums = whole(row)
    u = numbers(sums, 600, np.random.default_rng(1))
    B = len(u)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = medusa.verify_accept_tree_draw(to_dev(row).expand(B, 1, V).contiguous(), zero.expand(B, 1).contiguous(), zero - 1, zero,
                                         to_dev(u[:, None]), 0)
    assert np.array_equal(got["next_tok"].cpu().numpy(), drawn(sums, u))


@pytest.mark.parametrize("name", NAMES)
def test_walks(medusa, name):
    """A root whose child holds the token for every second sequence, so that both rows of those are drawn from."""
    row = row_of(name)
    sums = whole(row)
    u = numbers(sums, 200, np.random.default_rng(2))
    want = drawn(sums, u)
    B = len(u)
    cand = np.zeros((B, 2), np.int32)
    cand[:, 1] = np.where(np.arange(B) % 2, want, -1)
    node = torch.arange(2, dtype=torch.int32, device="cuda")
    got = medusa.verify_accept_tree_draw(to_dev(row).expand(B, 2, V).contiguous(), to_dev(cand), node - 1, node,
                                         to_dev(np.stack([u, u[::-1]], 1)), 1)
    got = {k: x.cpu().numpy() for k, x in got.items()}
    assert np.array_equal(got["accept_len"], np.arange(B) % 2)
    assert np.array_equal(got["next_tok"], np.where(np.arange(B) % 2, want[::-1], want))


@pytest.mark.parametrize("n", [1 << 20, 1 << 24])
def test_large_vocabularies(medusa, n):
    row = two_levels(0.7 / n, 0.9 / n, n)
    sums = whole(row)
    u = numbers(sums, 8, np.random.default_rng(3))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    B = len(u)
    got = medusa.verify_accept_tree_draw(to_dev(row).expand(B, 1, n).contiguous(), zero.expand(B, 1).contiguous(), zero - 1, zero,
                                         to_dev(u[:, None]), 0)
    assert np.array_equal(got["next_tok"].cpu().numpy(), drawn(sums, u))


@pytest.mark.parametrize("B", [1, 64])
def test_entries_above_one_count_as_one(medusa, B):
    """What the header says of weights that are not scaled to [0, 1]: the row clipped to it is drawn from."""
    rng = np.random.default_rng(5)
    counts = rng.integers(-1, 6, (B, 2, 40000)).astype(np.float32)
    node = torch.arange(2, dtype=torch.int32, device="cuda")
    rest = to_dev(np.full((B, 2), 40001, np.int32)), node - 1, node, to_dev(rng.random((B, 2), dtype=np.float32)), 1
    a = medusa.verify_accept_tree_draw(to_dev(counts), *rest)
    b = medusa.verify_accept_tree_draw(to_dev(np.clip(counts, 0, 1)), *rest)
    for name in a:
        assert torch.equal(a[name], b[name])


@pytest.mark.parametrize("u", [1.0, 1.0000001, 3.5, float("inf")])
@pytest.mark.parametrize("B,N,V", [(400, 1, 1003), (400, 1, 44914), (40, 5, 44914)])
def test_from_one_on_the_last_token_with_weight(medusa, B, N, V, u):
    """Rows whose last weights are below what any sum of them is rounded by."""
    rng = np.random.default_rng(V)
    z = rng.normal(0, 12, (B, V)).astype(np.float32)
    p = np.exp(z - z.max(1, keepdims=True))
    p[::3, -5:] = 0
    p[1::3, -1] = np.float32(1e-44)
    last = V - 1 - np.argmax(p[:, ::-1] > 0, 1)
    node = torch.arange(N, dtype=torch.int32, device="cuda")
    got = medusa.verify_accept_tree_draw(to_dev(p).view(B, 1, V).expand(B, N, V).contiguous(), to_dev(np.full((B, N), -1, np.int32)), node - 1, node,
                                         torch.full((B, N), u, device="cuda"), N - 1)
    assert np.array_equal(got["next_tok"].cpu().numpy(), last)
