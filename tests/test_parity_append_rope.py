"""GPU parity of the append that rotates on the way against its definition in float64."""
import numpy as np
import pytest
import torch

import chunk_ref as K
import q8_ref as R
from test_parity_q8 import NAMES, as_dtype, dev, pool, tables
from test_parity_rope import freqs
from util import to_dev

pytestmark = pytest.mark.gpu


def case(seed, B, T, Hq, Hkv, D, P, n, lens, last, dtype, interleaved=False, rows=None, size=1.0):
    rng = np.random.default_rng(seed)
    width = rows or T
    M = max(-(-(L + width) // P) for L in lens)
    n_pages = B * M + 2
    c = dict(zip(NAMES, pool(rng, n_pages, Hkv, P, D)))
    c["table"] = tables(rng, [L + width for L in lens], M, P, n_pages)
    c["kv_len"], c["last"] = np.array(lens, np.int32), None if last is None else np.array(last, np.int32)
    grow = np.exp(rng.normal(0, 0.7, (B, T, 1, 1))) * size
    c["k"], c["v"] = as_dtype(rng.normal(0, 1, (B, T, Hkv, D)) * grow, dtype), as_dtype(rng.normal(0, 1, (B, T, Hkv, D)) * grow, dtype)
    c["q"] = as_dtype(rng.normal(0, 1, (B, T, Hq, D)), dtype) if Hq else None
    c["rows"] = None
    if rows:
        c["rows"] = np.sort(rng.integers(0, T, (B, rows)), 1).astype(np.int32)
    c.update(f=freqs(n), dtype=dtype, interleaved=interleaved)
    return c


def run(M, c, **kw):
    pools = [to_dev(c[n].copy()) for n in NAMES]
    opt = lambda x: None if x is None else to_dev(x)  # noqa: E731
    r = M.kv_append_rope_q8(dev(c["k"], c["dtype"]), dev(c["v"], c["dtype"]), *pools, to_dev(c["table"]), to_dev(c["kv_len"]), to_dev(c["f"]),
                            rows=opt(c["rows"]), last=opt(c["last"]), q=None if c["q"] is None else dev(c["q"], c["dtype"]),
                            interleaved=c["interleaved"], **kw)
    torch.cuda.synchronize()
    return r, [p.cpu().numpy() for p in pools]


def check(c, r, got):
    kc, vc, ks, vs, L, n, slack, exact = K.append(c["k"], c["v"], *(c[m] for m in NAMES), c["table"], c["kv_len"], c["f"], c["interleaved"],
                                                  c["rows"], c["last"])
    assert np.array_equal(r["kv_len"].cpu().numpy(), L) and np.array_equal(r["appended"].cpu().numpy(), n)
    assert np.array_equal(got[2], ks) and np.array_equal(got[3], vs) and np.array_equal(got[1], vc)
    same = slack == 0
    assert np.array_equal(got[0][same], kc[same])
    # the nearest code of a value off by d is as near to the exact one as its own nearest, but for 2 d (slack)
    near, mine = np.abs(R.decode(kc) - exact), np.abs(R.decode(got[0]) - exact)
    ok = mine <= near + slack + 1e-12
    assert (ok | same | (np.isnan(R.decode(got[0])) & np.isnan(exact))).all()
    if c["q"] is not None:
        q = r["q"].double().cpu().numpy()
        for b in range(len(L)):
            m = c["q"].shape[1] if c["last"] is None else min(max(int(c["last"][b]), -1), c["q"].shape[1] - 1) + 1
            want = K.turned(c["q"][b, :m], int(c["kv_len"][b]) + np.arange(m), c["f"], c["interleaved"])
            tol = K.turn_error(c["q"][b, :m], len(c["f"]), c["interleaved"]) * (1 + 2.0 ** -8)
            tol = tol + np.abs(want) * (2.0 ** -8 if c["dtype"] == "bf16" else 0)
            assert (np.abs(q[b, :m] - want) <= tol).all() and not q[b, m:].any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,n,lens,last", [
    (1, 1, 4, 1, 64, 16, 32, [0], None),
    (3, 1, 8, 2, 128, 32, 64, [31, 32, 777], None),
    (2, 5, 4, 4, 64, 64, 16, [61, 100], [4, -1]),
    (3, 100, 3, 1, 128, 16, 64, [0, 15, 300], [99, 7, 50]),
    (2, 300, 10, 5, 128, 64, 32, [1000, 63], [299, 250]),
    (2, 200, 2, 2, 128, 128, 64, [5, 128], [199, 122]),
    (2, 150, 0, 40, 64, 128, 24, [5, 3], None),
    (1, 600, 24, 9, 128, 64, 64, [40], None),
])
def test_pages_hold_the_turned_rows(medusa, B, T, Hq, Hkv, D, P, n, lens, last, dtype, interleaved):
    c = case(T + P, B, T, Hq, Hkv, D, P, n, lens, last, dtype, interleaved)
    check(c, *run(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accepted_rows_turn_by_the_slots_they_go_to(medusa, dtype):
    c = case(5, 3, 64, 0, 4, 128, 16, 64, [14, 200, 0], [3, 5, 0], dtype, rows=6)
    rng = np.random.default_rng(6)
    hidden, best = dev(rng.normal(0, 1, (3, 64, 32)), dtype), to_dev(c["rows"][np.arange(3), c["last"]])
    r, got = run(medusa, c, best_node=best, hidden_rows=hidden)
    check(c, r, got)
    assert torch.equal(r["h_next"], hidden[torch.arange(3), best.long().cpu()])


def test_the_scale_does_not_depend_on_the_position(medusa):
    """The same rows at other positions of a page give the same scales, and 316 is where they change."""
    for size, want in ((316.0, 1.0), (316.25, 2.0), (158.0, 0.5)):
        for start in (0, 16, 16 * 57):
            c = case(9, 1, 16, 0, 1, 64, 16, 32, [start], None, "f32")
            c["k"] = np.clip(c["k"], -1, 1) * 0.5
            c["k"][0, 3, 0, 5] = -size
            r, got = run(medusa, c)
            check(c, r, got)
            assert got[2][c["table"][0, start // 16], 0] == want


def test_rows_under_a_caller_s_own_scale(medusa):
    """Scales that are no powers of two: codes of the exact quotient's nearest."""
    c = case(12, 2, 20, 2, 2, 64, 16, 32, [5, 20], None, "f32", size=0.01)
    c["k_scale"][:], c["v_scale"][:] = np.float32(0.37), np.float32(1.9)
    check(c, *run(medusa, c))


def test_values_that_are_not_finite(medusa):
    c = case(13, 1, 20, 2, 2, 64, 16, 32, [3], None, "f32")
    c["k"][0, 2, 0, 7], c["k"][0, 4, 1, 50], c["v"][0, 5, 0, 1] = np.inf, np.nan, -np.inf
    r, got = run(medusa, c)
    check_scales = K.append(c["k"], c["v"], *(c[m] for m in NAMES), c["table"], c["kv_len"], c["f"], False)
    assert np.array_equal(got[2], check_scales[2]) and np.array_equal(got[3], check_scales[3])
    page = int(c["table"][0, 0])
    k = R.decode(got[0])
    assert abs(k[page, 0, 5, 7]) == 448 and abs(k[page, 0, 5, 39]) == 448  # cos and sin of position 5 are not zero
    assert np.isnan(k[page, 1, 7, 50]) and np.isnan(k[page, 1, 7, 18])
    assert R.decode(got[1])[page, 0, 8, 1] == -448
    bad = np.zeros(k.shape, bool)
    bad[page, 1, 7, [18, 50]] = True
    assert np.array_equal(np.isnan(k), bad)


@pytest.mark.parametrize("what", ["last", "kv_len", "table", "rows"])
def test_a_refused_sequence_changes_nothing_and_the_others_do(medusa, what):
    c = case(15, 3, 30, 0 if what == "rows" else 2, 2, 64, 16, 32, [3, 40, 0], [29, 10, 5] if what != "rows" else [3, 3, 3], "bf16", rows=4 if what == "rows" else None)
    if what == "last":
        c["last"][1] = 30
    elif what == "kv_len":
        c["kv_len"][1] = -1
    elif what == "table":
        c["table"][1, 3] = 10 ** 6
    else:
        c["rows"][1, 2] = 30
    r, got = run(medusa, c)
    check(c, r, got)
    assert r["appended"].tolist()[1] == -2


def test_queries_in_place(medusa):
    c = case(16, 2, 50, 6, 3, 128, 32, 64, [7, 90], [49, 20], "bf16")
    r, _ = run(medusa, c)
    q = dev(c["q"], "bf16")
    out = dict(kv_len=torch.empty_like(r["kv_len"]), q=q)
    medusa.kv_append_rope_q8(dev(c["k"], "bf16"), dev(c["v"], "bf16"), *(to_dev(c[n].copy()) for n in NAMES), to_dev(c["table"]), to_dev(c["kv_len"]),
                             to_dev(c["f"]), last=to_dev(c["last"]), q=q, out=out)
    assert torch.equal(q, r["q"]) and torch.equal(out["kv_len"], r["kv_len"])
