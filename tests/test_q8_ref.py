"""The plain definitions of the 8-bit paged cache (tests/q8_ref.py) against what
their formats and rules fix."""
import numpy as np
import torch

import q8_ref as R


def test_e4m3_values_are_the_format_s():
    t = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.VALUES, t, equal_nan=True)


def test_encode_is_nearest_even_and_inverts_decode():
    codes = np.array([c for c in range(256)], np.uint8)
    assert np.array_equal(R.encode(R.decode(codes))[codes != 255], codes[codes != 255])  # 0xff: NaN as 0x7f
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(0, 100, 4000), rng.normal(0, 0.01, 4000), [1e9, -1e9, 448, 464, 2.0 ** -10]])
    got = R.decode(R.encode(x))
    grid = R.VALUES[np.isfinite(R.VALUES)]
    best = np.abs(grid[None] - np.clip(x, -448, 448)[:, None]).min(1)
    assert np.array_equal(np.abs(got - np.clip(x, -448, 448)), best)
    y = x[np.abs(x) <= 448].astype(np.float32)
    assert np.array_equal(R.encode(y), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert R.encode([2.0 ** -10])[0] == 0 and R.encode([3 * 2.0 ** -10])[0] == 2  # ties to the even code


def test_page_scale_is_the_smallest_that_fits():
    for top in (1e-30, 0.1, 447.9, 448.0, 448.5, 896.0, 1e6):
        s = R.page_scale([0.0, -top, np.inf, np.nan])
        assert s == 2.0 ** -64 or (top <= 448 * s and top > 224 * s)
    assert R.page_scale([0.0]) == 2.0 ** -64 and R.page_scale([1e30]) == 2.0 ** 64


def test_fork_keeps_every_text_and_no_page_twice():
    rng = np.random.default_rng(2)
    for _ in range(200):
        B, M, P, n = int(rng.integers(1, 7)), int(rng.integers(1, 6)), 16, int(rng.integers(6, 40))
        kv_len = rng.integers(0, M * P + 1, B)
        perm, table = rng.permutation(n).tolist(), np.full((B, M), -1, np.int32)
        for b in range(B):
            k = -(-int(kv_len[b]) // P)
            if k > len(perm):
                kv_len[b] = k = 0
            for j in range(k):
                table[b, j] = perm.pop()
        src, need = rng.integers(-1, B, B), rng.integers(0, 40, B)
        t, L, refs, taken, copies = R.fork(table, kv_len, n, P, src, need)
        moved = {d: s for s, d, _ in copies}
        for b in range(B):
            if src[b] < 0:
                assert L[b] == 0 and (t[b] == -1).all()
                continue
            assert L[b] == kv_len[src[b]] or (taken[b] == -1 and L[b] == kv_len[src[b]] // P * P)
            for j in range(-(-int(L[b]) // P)):
                assert moved.get(int(t[b, j]), int(t[b, j])) == table[src[b], j]
            if taken[b] >= 0:
                assert L[b] + need[b] <= P * (t[b] >= 0).sum()
        held = np.bincount(t[t >= 0], minlength=n)
        assert np.array_equal(held, refs)
        for p in np.flatnonzero(held > 1):  # shared pages are full for all that hold them
            for b, j in zip(*np.where(t == p)):
                assert (j + 1) * P <= L[b]


def test_compact_keeps_every_page_and_leaves_no_hole():
    rng = np.random.default_rng(3)
    for _ in range(100):
        n, B, M = int(rng.integers(1, 60)), int(rng.integers(1, 5)), int(rng.integers(1, 9))
        table = rng.integers(-1, n, (B, M)).astype(np.int32)
        held = (rng.random(n) < 0.1).astype(np.int32)
        t, new, live, moves = R.compact(table, n, held)
        used = set(table[table >= 0].tolist()) | set(np.flatnonzero(held).tolist())
        assert live == len(used) and sorted(new[sorted(used)].tolist()) == list(range(live))
        assert {s for s, _ in moves} == {p for p in used if p >= live}
        assert np.array_equal(t[table >= 0], new[table[table >= 0]]) and (t[table < 0] == -1).all()
