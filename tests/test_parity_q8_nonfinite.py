"""GPU parity of the 8-bit paged cache where values are not finite: rows that are
appended in the model's type, codes that count, queries."""
import numpy as np
import pytest

import q8_ref as R
from test_parity_q8 import as_dtype, attend, attention_case, check, pool, reference, run_append, same_pools, tables, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_append_extreme_bf16_values_row_by_row(medusa, D, P):
    """Zeros, infinities, NaN, the ends of bf16 and growing rows, one token at a time, K
    and V of different rows."""
    rng = np.random.default_rng(12)
    Hkv, M = 3, 3
    pools = pool(rng, 5, Hkv, P, D)
    table, kv_len = tables(rng, [3 * P], M, P, 5), np.array([0], np.int32)
    mixed = rng.normal(0, 1, (Hkv, D))
    mixed[0, ::7], mixed[1, 1], mixed[2, :] = np.inf, np.nan, -np.inf
    rows = [np.zeros((Hkv, D)), np.full((Hkv, D), 1e-38), rng.normal(0, 1e-3, (Hkv, D)), mixed, np.full((Hkv, D), -np.inf),
            np.full((Hkv, D), np.nan), rng.normal(0, 1e6, (Hkv, D)), np.full((Hkv, D), 3.3e38), rng.normal(0, 1, (Hkv, D)),
            np.full((Hkv, D), 9.2e-41)]
    for i in range(2 * P + 5):
        k, v = (as_dtype(rows[j % len(rows)].reshape(1, 1, Hkv, D), "bf16") for j in (i, 3 * i + 1))
        got, new_len, count, _ = run_append(medusa, pools, k, v, "bf16", table, kv_len)
        *want, want_len, _ = R.append(k, v, *pools, table, kv_len)
        same_pools(got, want)
        assert new_len[0] == kv_len[0] + 1 and count[0] == 1
        pools, kv_len = want, want_len


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_prompts_with_non_finite_rows(medusa, dtype):
    rng = np.random.default_rng(13)
    B, T, Hkv, D, P = 2, 150, 2, 128, 32
    pools = pool(rng, 14, Hkv, P, D)
    table, kv_len = tables(rng, [T + 20, T], 6, P, 14), np.array([20, 0], np.int32)
    k, v = (rng.normal(0, 1, (B, T, Hkv, D)) for _ in "kv")
    for x in (k, v):
        for value in (np.inf, -np.inf, np.nan):
            x[rng.random(x.shape) < 0.01] = value
        x[1, 64:96, 0] = np.nan  # a page of nothing else
        x[1, 64:96, 1] = np.inf
    k, v = as_dtype(k, dtype), as_dtype(v, dtype)
    got, new_len, count, _ = run_append(medusa, pools, k, v, dtype, table, kv_len)
    *want, want_len, want_count = R.append(k, v, *pools, table, kv_len)
    same_pools(got, want)
    assert np.array_equal(new_len, want_len) and np.array_equal(count, want_count)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", [(1, 4, 2, 64, 16), (30, 2, 2, 128, 32), (80, 2, 2, 64, 64)])
def test_attention_nan_codes_that_count(medusa, N, Hq, Hkv, D, P, dtype):
    """A NaN in K makes every row of the head NaN; one in V the column; other heads and
    sequences are as without."""
    c = attention_case(120 + N, 3, N, Hq, Hkv, D, P, [500, 200, 300], dtype)
    G = Hq // Hkv
    ref = reference(c)
    c["k_pages"][c["table"][0, 190 // P], 0, 190 % P, 5] = 0x7f
    c["v_pages"][c["table"][1, 3], 1, 0, 7] = 0xff
    got = attend(medusa, c)
    assert np.isnan(got[0, :, :G]).all() and np.isnan(got[1, :, G:, 7]).all()
    hurt = np.isnan(got)
    assert hurt.sum() == N * G * D + N * G
    assert (np.abs(got - ref[0]) <= tolerance(c, ref))[~hurt].all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", [(2, 4, 2, 64, 16), (30, 2, 2, 128, 32), (80, 2, 2, 64, 64)])
def test_attention_queries_that_are_not_finite(medusa, N, Hq, Hkv, D, P, dtype):
    """A row of q with a NaN is NaN, the rows beside it are as without."""
    c = attention_case(130 + N, 2, N, Hq, Hkv, D, P, [300, 129], dtype)
    ref = reference(c)
    tol = tolerance(c, ref)
    c["q"][0, 1, 0, 3], c["q"][1, N - 1, Hq - 1, 0] = np.nan, np.nan
    got = attend(medusa, c)
    hurt = np.isnan(got)
    assert hurt[0, 1, 0].all() and hurt[1, N - 1, Hq - 1].all() and hurt.sum() == 2 * D
    assert (np.abs(got - ref[0]) <= tol)[~hurt].all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_infinite_queries_hurt_no_other_row(medusa, dtype):
    c = attention_case(140, 1, 30, 2, 2, 64, 32, [300], dtype)
    ref = reference(c)
    tol = tolerance(c, ref)
    c["q"][0, 7, 1, 3] = np.inf
    got = attend(medusa, c)
    hurt = np.isnan(got)
    assert hurt[0, 7, 1].all() and hurt.sum() == 64
    assert (np.abs(got - ref[0]) <= tol)[~hurt].all()
