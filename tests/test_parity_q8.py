"""GPU parity of the 8-bit paged cache's operators against their definitions in
float64 (tests/q8_ref.py): attention over the pages and the tree, append, fork,
compact, and decode rounds that use them together."""
import numpy as np
import pytest
import torch

import q8_ref as R
from util import to_dev, to_np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a unit in the last place of float32, relative


# ---------------------------------------------------------------------------
# inputs
def pool(rng, n, Hkv, P, D, fill=1.0):
    """Codes and power-of-two scales of random rows whose size varies by page."""
    out = {}
    for s in "kv":
        x = rng.standard_normal((n, Hkv, P, D), np.float32) * np.exp(rng.normal(0, 0.5, (n, Hkv, 1, 1))).astype(np.float32) * fill
        top = np.abs(x).max((2, 3), keepdims=True)
        scale = R.page_scales(top).astype(np.float32)
        # (the same codes as R.encode gives: nothing exceeds 448 under these scales)
        codes = torch.from_numpy(x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        out[s] = codes, scale
    return out["k"][0], out["v"][0], out["k"][1], out["v"][1]


def tables(rng, lens, M, P, n, spare=0):
    perm = rng.permutation(n).tolist()
    t = np.full((len(lens), M), -1, np.int32)
    for b, L in enumerate(lens):
        for j in range(min(M, -(-int(L) // P) + spare)):
            t[b, j] = perm.pop()
    return t


def tree(kind, N, rng):
    if kind == "chain":
        par = np.arange(N) - 1
    elif kind == "dense":
        par = np.where(np.arange(N) > 0, (np.arange(N) - 1) // 4, -1)
    else:
        par = np.array([-1] + [int(rng.integers(0, i)) for i in range(1, N)])
    m = np.zeros((N, (N + 63) // 64), np.uint64)
    for i in range(N):
        j = i
        while j >= 0:
            m[i, j >> 6] |= np.uint64(1) << np.uint64(j & 63)
            j = par[j]
    return m


def as_dtype(x, dtype):
    """float64 values that the type holds."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float64)).float()
    return (t.bfloat16() if dtype == "bf16" else t).double().numpy()


def dev(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x)).float()
    return (t.bfloat16() if dtype == "bf16" else t).cuda()


def attention_case(seed, B, N, Hq, Hkv, D, P, lens, dtype, kind="random", q_std=1.0, extra=3):
    rng = np.random.default_rng(seed)
    M = max(1, -(-max(lens) // P)) + 1
    n = sum(-(-L // P) for L in lens) + extra
    c = dict(zip(("k_pages", "v_pages", "k_scale", "v_scale"), pool(rng, n, Hkv, P, D)))
    c["table"], c["kv_len"] = tables(rng, lens, M, P, n), np.array(lens, np.int32)
    c["q"] = as_dtype(rng.normal(0, q_std, (B, N, Hq, D)), dtype)
    c["k_tree"] = as_dtype(rng.normal(0, 1, (B, N, Hkv, D)), dtype)
    c["v_tree"] = as_dtype(rng.normal(0, 1, (B, N, Hkv, D)), dtype)
    c["mask"], c["scale"], c["dtype"] = tree(kind, N, rng), float(np.float32(1 / np.sqrt(D))), dtype
    return c


NAMES = ("k_pages", "v_pages", "k_scale", "v_scale")


def attend(M, c, **kw):
    out = M.tree_attention_q8(dev(c["q"], c["dtype"]), dev(c["k_tree"], c["dtype"]), dev(c["v_tree"], c["dtype"]),
                              *(to_dev(c[n]) for n in NAMES), to_dev(c["table"]), to_dev(c["kv_len"]), to_dev(c["mask"]),
                              c["scale"], **kw)
    torch.cuda.synchronize()
    M.device_status()
    return out.double().cpu().numpy()


def reference(c):
    return R.attention(c["q"], c["k_tree"], c["v_tree"], *(c[n] for n in NAMES), c["table"], c["kv_len"], c["mask"],
                       c["scale"])


def tolerance(c, ref):
    """What rounding may make of each output, from the call's documentation.

    Scores: products summed in float32, D terms, relative to sum |q||k|; a score
    off by e makes its weight off by e^e - 1 <= 1.01 e for e < 0.01, and the sum it
    is divided by likewise: 2.1 e.  Sums over the keys in float32: each addition
    rounds once, relative to the sum of magnitudes.  exp2: 2 units, its argument's
    rounding is part of e (arguments stay below 2^7 in units of the score).
    bf16: q enters to 2^-17 of the largest |q| of the row block (all of q here);
    weights of tree rows are bf16, 2^-8, those of pages have 9 bits, 2^-9 (both are
    held to 2^-8 here), and half of e5m2's least step, 2^-17, in
    planes that hold at least 2^9 for a weight of 1 on the largest V scale: 2^-26,
    times a code of at most 448, for each key; the output rounds to bf16: 2^-8."""
    out, spread, bounds = ref
    keys = min(int(c["kv_len"].max()), c["table"].shape[1] * c["k_pages"].shape[2]) + c["q"].shape[1]
    D = c["q"].shape[3]
    e = (D + 8) * U * bounds[..., 0] + 8 * U * 128
    per = (2 * keys + 64) * U
    if c["dtype"] == "bf16":
        e = e + 2.0 ** -17 * np.abs(c["q"]).max() * bounds[..., 1]
        per = per + 2.0 ** -8
    tol = spread * (2.1 * e[..., None] + per)
    if c["dtype"] == "bf16":
        vs = np.where(np.isfinite(c["v_scale"]), c["v_scale"], 0).max()
        tol = tol + 2.0 ** -8 * np.abs(out) + keys * 2.0 ** -26 * 448 * max(vs, 1 / 448)
    else:
        tol = tol + U * np.abs(out)
    return tol


def worst_score(c, ref):
    """What the rounding of q may add to a weight, as a share (tolerance's e)."""
    return 2.1 * 2.0 ** -17 * np.abs(c["q"]).max() * np.nanmax(ref[2][..., 1])


def check(c, got, ref):
    assert np.array_equal(np.isnan(got), np.isnan(ref[0]))  # NaN codes in keys that count
    err, tol = (np.nan_to_num(x) for x in (np.abs(got - ref[0]), tolerance(c, ref)))
    assert (err - tol).max() <= 0, ((err - tol).max(), err.max())
    norm = np.linalg.norm(np.nan_to_num(ref[0]))
    if c["dtype"] == "bf16" and norm:
        # independent roundings of the output and the weights, at most 2^-8 each: a
        # uniform error within +-h has root mean square h / sqrt(3)
        assert np.linalg.norm(err) / norm <= np.sqrt(2 / 3) * 2.0 ** -8 + 2.0 ** -12 + worst_score(c, ref)


# ---------------------------------------------------------------------------
# attention
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,P,lens", [
    (1, 1, 1, 1, 64, 16, [0]),                 # one token, empty cache
    (1, 1, 4, 2, 128, 16, [1]),
    (2, 9, 4, 4, 64, 16, [127, 129]),          # a tile's edge
    (3, 2, 8, 1, 128, 32, [31, 256, 700]),     # eight query heads on one KV head
    (2, 64, 2, 2, 128, 64, [64, 517]),         # 64 rows exactly
    (2, 65, 2, 2, 128, 128, [1000, 3]),        # one more
    (1, 33, 6, 2, 64, 64, [391]),              # three heads a group: rows across nodes
    (2, 129, 2, 1, 128, 32, [0, 300]),         # several row blocks, two tree tiles
    (1, 341, 1, 1, 64, 128, [640]),
    (5, 1, 7, 7, 128, 64, [5, 1500, 64, 0, 128]),
])
def test_attention(medusa, B, N, Hq, Hkv, D, P, lens, dtype):
    c = attention_case(B * 1000 + N, B, N, Hq, Hkv, D, P, lens, dtype)
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_many_sequences_and_a_long_one(medusa, dtype):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 200).tolist() + [9000]
    c = attention_case(6, len(lens), 1, 2, 1, 64, 16, lens, dtype)
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["chain", "dense", "random"])
def test_attention_peaked_scores_and_trees(medusa, kind, dtype):
    # scores tens of units apart: the running maximum moves often
    c = attention_case(11, 2, 40, 2, 2, 64, 32, [300, 1111], dtype, kind, q_std=6.0)
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_growing_scores_and_uneven_scales(medusa, dtype):
    """The maximum grows with every page, and V's scales span 2^12: the sums are
    rescaled again and again."""
    c = attention_case(12, 1, 3, 1, 1, 128, 16, [900], dtype)
    for j, p in enumerate(c["table"][0]):
        if p >= 0:
            c["k_scale"][p] *= 2.0 ** (j // 8)
            c["v_scale"][p] *= 2.0 ** ((j * 5) % 13 - 6)
    ref = reference(c)
    got = attend(medusa, c)
    assert (np.abs(got - ref[0]) <= tolerance(c, ref)).all()


@pytest.mark.parametrize("N,Hq,Hkv,D,P", [(1, 120, 40, 128, 64), (9, 120, 120, 64, 16), (40, 80, 80, 128, 32), (70, 60, 60, 128, 128),
                                          (64, 40, 40, 64, 64)])
def test_attention_long_shares(medusa, N, Hq, Hkv, D, P):
    """Each CTA works through many tiles and several units: references move in the
    middle of a share (scores and V scales that grow from page to page, in some
    pages of some heads only), pages are missing, units end and begin."""
    c = attention_case(40 + N, 2, N, Hq, Hkv, D, P, [2000, 3171], "bf16", q_std=1.5)
    rng = np.random.default_rng(N)
    for b in range(2):
        for j, p in enumerate(c["table"][b]):
            if p >= 0:
                c["k_scale"][p] *= 2.0 ** rng.integers(0, 3, Hkv) * (1 + (j > 20))
                c["v_scale"][p] *= 2.0 ** rng.integers(-3, 4, Hkv)
    c["table"][0, 5] = c["table"][1, 9] = -1
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_scales_that_are_no_powers_of_two(medusa, dtype):
    c = attention_case(13, 2, 9, 4, 2, 64, 32, [100, 333], dtype)
    rng = np.random.default_rng(7)
    for n in ("k_scale", "v_scale"):
        c[n] = (c[n] * np.exp(rng.normal(0, 0.3, c[n].shape))).astype(np.float32)
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_skips_what_is_not_there(medusa, dtype):
    """Pages out of range, unreadable scales, NaN codes behind the end, lengths out
    of range: absent keys, and no trace of them in the output."""
    c = attention_case(14, 4, 5, 2, 2, 128, 32, [500, 200, 70, 95], dtype)
    c["table"][0, 3], c["table"][0, 7] = -1, 10 ** 6
    c["k_scale"][c["table"][1, 2]] = np.nan
    c["v_scale"][c["table"][1, 4]] = 0.0
    c["v_scale"][c["table"][1, 5], 1] = np.inf
    for b in (2, 3):  # the last page's slots behind the end: NaN in K and V
        L = c["kv_len"][b]
        p = c["table"][b, L // 32]
        c["k_pages"][p, :, L % 32:] = 0x7f
        c["v_pages"][p, :, L % 32:] = 0xff
    got = attend(medusa, c)
    check(c, got, reference(c))
    c["kv_len"][2], c["kv_len"][3] = -5, 10 ** 9  # clamped
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_masks_that_leave_rows_empty(medusa, dtype):
    c = attention_case(15, 2, 70, 2, 1, 64, 16, [0, 40], dtype)
    c["mask"][::3] = 0
    got, ref = attend(medusa, c), reference(c)
    check(c, got, ref)
    assert (got[0, ::3] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_infinities_where_the_mask_hides_them(medusa, dtype):
    """Node 3's K and node 4's V are not finite: rows that do not see them are as
    without, the others NaN."""
    c = attention_case(16, 1, 20, 2, 2, 128, 16, [200], dtype)
    ref = reference(c)
    c["k_tree"][0, 3], c["v_tree"][0, 4, 0, 5] = np.nan, np.inf
    seen = R.sees(c["mask"], 20)
    got = attend(medusa, c)
    for h in (0, 1):
        hurt = seen[:, 3] | (seen[:, 4] if h == 0 else False)
        tol = tolerance(c, ref)[0, ~hurt, h]
        assert (np.abs(got[0, ~hurt, h] - ref[0][0, ~hurt, h]) <= tol).all()
        assert np.isnan(got[0, hurt, h]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,P,lens", [(1, 1, 2, 1, 64, 16, [1]), (3, 1, 8, 2, 128, 32, [40, 0, 64]),
                                                 (70, 9, 4, 4, 64, 16, [37] * 70), (2, 64, 40, 40, 128, 64, [64, 17]),
                                                 (5, 33, 80, 80, 64, 64, [3, 64, 20, 0, 1]), (2, 90, 3, 3, 128, 16, [50, 64])])
def test_attention_narrow_and_wide_tables(medusa, B, N, Hq, Hkv, D, P, lens, dtype):
    """Short texts in tables that hold no more (units are not cut then) and in wide ones."""
    c = attention_case(45, B, N, Hq, Hkv, D, P, lens, dtype)
    c["table"] = c["table"][:, :-(-64 // P)]
    ref = reference(c)
    check(c, attend(medusa, c), ref)
    wide = dict(c, table=np.concatenate([c["table"], np.full((B, 3000 // P), -1, np.int32)], 1))
    check(wide, attend(medusa, wide), ref)


@pytest.mark.parametrize("N", [6, 70])
def test_attention_large_tree_values(medusa, N):
    """V of the tree up to 2^91 is summed without overflow, over pages of small scales
    too; from there on it counts as infinite."""
    c = attention_case(42, 1, N, 2, 2, 64, 16, [300], "bf16")
    c["v_scale"] = c["v_scale"] * np.float32(2.0 ** -20)
    c["v_tree"] = as_dtype(c["v_tree"] * 2.0 ** 88, "bf16")
    c["v_tree"][0, 0] = 2.0 ** 90.9
    c["v_tree"] = as_dtype(c["v_tree"], "bf16")
    assert np.abs(c["v_tree"]).max() < 2.0 ** 91
    check(c, attend(medusa, c), reference(c))
    c["v_tree"][0, 2, 1, 5] = -2.0 ** 91
    got, seen = attend(medusa, c), R.sees(c["mask"], N)
    assert np.isnan(got[0, seen[:, 2], 1]).all() and np.isfinite(got[0, ~seen[:, 2]]).all() and np.isfinite(got[0, :, 0]).all()


def test_attention_two_streams_at_once(medusa):
    """Calls on two streams, each with its workspace, do not disturb one another."""
    cases = [attention_case(43, 2, 64, 4, 4, 128, 64, [900, 400], "bf16"), attention_case(44, 3, 1, 8, 2, 128, 32, [3000, 1, 700], "bf16")]
    alone = [attend(medusa, c) for c in cases]
    t = [[dev(c[n], "bf16") for n in ("q", "k_tree", "v_tree")] + [to_dev(c[n]) for n in NAMES + ("table", "kv_len", "mask")] for c in cases]
    outs = [[torch.empty_like(x[0]) for _ in range(20)] for x in t]
    ws = [torch.empty(medusa.tree_attention_q8_workspace(*x[0].shape[:3], x[3].shape[1], x[0].shape[3]), dtype=torch.uint8, device="cuda")
          for x in t]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for i in range(20):
        for x, o, w, c, s in zip(t, outs, ws, cases, streams):
            medusa.tree_attention_q8(*x, c["scale"], out=o[i], ws=w, stream=s)
    torch.cuda.synchronize()
    medusa.device_status()
    for a, o in zip(alone, outs):
        for x in o:
            assert np.array_equal(x.double().cpu().numpy(), a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_same_call_same_bits_and_other_stream(medusa, dtype):
    c = attention_case(17, 3, 64, 4, 4, 128, 64, [700, 1300, 20], dtype)
    a = attend(medusa, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = attend(medusa, c, stream=s)
    s.synchronize()
    assert np.array_equal(a, b)


def test_attention_outputs_are_all_that_is_written(medusa):
    c = attention_case(18, 2, 9, 2, 2, 64, 16, [100, 50], "bf16")
    big = torch.full((2 + 2, 9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    attend(medusa, c, out=big[1:3])
    assert (big[0] == 7).all() and (big[3] == 7).all() and not (big[1:3] == 7).any()


# ---------------------------------------------------------------------------
# append
def run_append(M, pools, k, v, dtype, table, kv_len, **kw):
    t = [to_dev(x) for x in pools]
    kw = {n: to_dev(x) if isinstance(x, np.ndarray) and n != "hidden_rows" else x for n, x in kw.items()}
    r = M.kv_append_q8(dev(k, dtype), dev(v, dtype), *t, to_dev(table), to_dev(kv_len), **kw)
    torch.cuda.synchronize()
    return [to_np(x) for x in t], to_np(r["kv_len"]), to_np(r["appended"]), r


def same_pools(got, want):
    for n, g, w in zip(NAMES, got, want):
        if g.dtype == np.uint8:  # NaN codes: either sign
            g, w = np.where(g == 255, 127, g), np.where(w == 255, 127, w)
        assert np.array_equal(g, w, equal_nan=g.dtype != np.uint8), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,R_,Hkv,D,P,lens", [
    (1, 1, 0, 1, 64, 16, [0]),
    (2, 1, 0, 3, 128, 16, [15, 16]),
    (3, 64, 6, 2, 128, 64, [60, 64, 0]),       # accepted branches over a page's end
    (2, 9, 3, 4, 64, 32, [31, 95]),
    (2, 300, 0, 2, 128, 128, [0, 77]),         # prompts
    (4, 200, 0, 1, 64, 16, [3, 0, 15, 100]),
])
def test_append(medusa, B, T, R_, Hkv, D, P, lens, dtype):
    rng = np.random.default_rng(T * 7 + D)
    n_new = R_ or T
    M = -(-(max(lens) + n_new) // P)
    pools = pool(rng, B * M + 2, Hkv, P, D)
    table = tables(rng, np.array(lens) + n_new, M, P, B * M + 2)
    size = np.exp(rng.normal(0, 2, (B, T, 1, 1)))  # some rows need a larger scale
    k, v = as_dtype(rng.normal(0, 1, (B, T, Hkv, D)) * size, dtype), as_dtype(rng.normal(0, 1, (B, T, Hkv, D)), dtype)
    rows = np.sort(rng.integers(0, T, (B, R_)), 1).astype(np.int32) if R_ else None
    last = rng.integers(-1, n_new, B).astype(np.int32)
    last[0] = n_new - 1
    kv_len = np.array(lens, np.int32)
    got, new_len, count, _ = run_append(medusa, pools, k, v, dtype, table, kv_len, rows=rows, last=last)
    *want, want_len, want_count = R.append(k, v, *pools, table, kv_len, rows, last)
    same_pools(got, want)
    assert np.array_equal(new_len, want_len) and np.array_equal(count, want_count)


def test_append_extreme_values_and_row_by_row(medusa):
    """Zeros, infinities, NaN, the ends of float32 and growing rows, one token at a
    time: each step as the definition has it."""
    rng = np.random.default_rng(9)
    B, Hkv, D, P, M = 1, 2, 64, 16, 3
    pools = pool(rng, 5, Hkv, P, D)
    table, kv_len = tables(rng, [48], M, P, 5), np.array([0], np.int32)
    rows = [np.zeros((Hkv, D)), np.full((Hkv, D), 1e-38), rng.normal(0, 1e-3, (Hkv, D)), rng.normal(0, 1, (Hkv, D)),
            np.full((Hkv, D), np.inf), np.full((Hkv, D), np.nan), rng.normal(0, 1e6, (Hkv, D)), np.full((Hkv, D), 3e38),
            rng.normal(0, 1, (Hkv, D))]
    for i in range(40):
        x = as_dtype(rows[i % len(rows)].reshape(1, 1, Hkv, D), "f32")
        got, new_len, count, _ = run_append(medusa, pools, x, -x, "f32", table, kv_len)
        *want, want_len, _ = R.append(x, -x, *pools, table, kv_len)
        same_pools(got, want)
        assert new_len[0] == kv_len[0] + 1 and count[0] == 1
        pools, kv_len = want, want_len


def test_append_leaves_malformed_sequences_unchanged(medusa):
    rng = np.random.default_rng(10)
    B, T, Hkv, D, P, M = 9, 8, 2, 64, 16, 3
    pools = list(pool(rng, 40, Hkv, P, D))
    kv_len = np.array([10, 10, 10, 47, -1, 10, 10, 40, 10], np.int32)
    table = tables(rng, [48] * B, M, P, 40)
    last = np.array([3, 4, -2, 3, 3, 3, 3, -1, 3], np.int32)  # 1: beyond R; 2: below -1; 3: past the table; 7: nothing
    rows = np.tile(np.arange(4, dtype=np.int32), (B, 1))
    rows[5, 2] = 8
    table[6, 0] = 40
    best = np.zeros(B, np.int32)
    best[8] = 8
    k, v = (as_dtype(rng.normal(0, 1, (B, T, Hkv, D)), "bf16") for _ in "kv")
    hidden = torch.randn(B, T, 72, device="cuda").bfloat16()
    got, new_len, count, r = run_append(medusa, pools, k, v, "bf16", table, kv_len, rows=rows, last=last, best_node=best,
                                        hidden_rows=hidden)
    *want, want_len, want_count = R.append(k, v, *pools, table, kv_len, rows, last, best)
    same_pools(got, want)
    assert np.array_equal(new_len, want_len) and np.array_equal(count, want_count)
    assert count.tolist() == [4, -2, -2, -2, -2, -2, -2, 0, -2]
    assert torch.equal(r["h_next"][0], hidden[0, 0]) and torch.equal(r["h_next"][7], hidden[7, 0])


def test_append_to_an_unreadable_page_leaves_it(medusa):
    rng = np.random.default_rng(11)
    pools = list(pool(rng, 3, 2, 16, 64))
    table, kv_len = np.array([[1, 2]], np.int32), np.array([14], np.int32)
    pools[2][1, 0], pools[3][1, 1] = np.nan, -1.0
    x = as_dtype(rng.normal(0, 1, (1, 4, 2, 64)), "f32")
    got, _, count, _ = run_append(medusa, pools, x, x, "f32", table, kv_len)
    *want, _, _ = R.append(x, x, *pools, table, kv_len)
    same_pools(got, want)
    assert count[0] == 4


# ---------------------------------------------------------------------------
# fork and compact
def same_fork(M, rng, lens, Mx, P, n, src, need, held=None, spare=0, Hkv=2, D=64, table=None):
    pools = pool(rng, n, Hkv, P, D)
    table = tables(rng, lens, Mx, P, n, spare) if table is None else table
    kv_len = np.array(lens, np.int32)
    i32 = lambda x: None if x is None else np.asarray(x, np.int32)  # noqa: E731
    t = [to_dev(x) for x in pools]
    r = M.kv_pages_fork(*t, to_dev(table), to_dev(kv_len), *(None if x is None else to_dev(i32(x)) for x in (src, need, held)))
    torch.cuda.synchronize()
    want_t, want_len, want_refs, want_taken, copies = R.fork(table, kv_len, n, P, src, need, held)
    for name, w in (("page_table", want_t), ("kv_len", want_len), ("refs", want_refs), ("taken", want_taken)):
        assert np.array_equal(to_np(r[name]), w), (name, to_np(r[name]), w)
    for a, d, rows in copies:
        for x in pools[:2]:
            x[d, :, :rows] = x[a, :, :rows]
        for x in pools[2:]:
            x[d] = x[a]
    same_pools([to_np(x) for x in t], pools)
    return r


@pytest.mark.parametrize("B,Mx,P,n", [(1, 1, 16, 1), (4, 5, 16, 30), (64, 40, 16, 1500), (200, 9, 32, 3000), (1024, 6, 64, 9000),
                                      (3, 700, 128, 2500)])
def test_fork_random(medusa, B, Mx, P, n):
    rng = np.random.default_rng(B + n)
    for trial in range(3):
        lens = rng.integers(0, Mx * P + 1, B)
        while (-(-lens // P)).sum() > n:
            lens = lens // 2
        src = None if trial == 0 else rng.integers(-1, B, B)
        same_fork(medusa, rng, lens, Mx, P, n, src, rng.integers(-3, 3 * P, B), Hkv=1, D=64)


def test_fork_identity_free_all_and_one_to_all(medusa):
    rng = np.random.default_rng(20)
    lens = [33, 0, 16, 70, 5]
    same_fork(medusa, rng, lens, 6, 16, 40, None, None)
    same_fork(medusa, rng, lens, 6, 16, 40, [-1] * 5, [7] * 5)
    same_fork(medusa, rng, lens, 6, 16, 40, [3] * 5, [7, 0, 30, 1, 2])


def test_fork_reserved_and_held_pages(medusa):
    rng = np.random.default_rng(21)
    held = (rng.random(60) < 0.3).astype(np.int32) * 2 - (rng.random(60) < 0.1)
    same_fork(medusa, rng, [33, 20, 16, 70, 5], 8, 16, 60, [0, 0, 3, 3, 4], [40, 3, 16, 0, 100], held=held, spare=2)


def test_fork_when_pages_run_out(medusa):
    rng = np.random.default_rng(22)
    for n in range(13, 22):
        same_fork(medusa, rng, [33, 20, 16, 70, 5], 8, 16, n, [0, 0, 0, 3, 3], [40, 3, 16, 0, 60])
    same_fork(medusa, rng, [33, 20], 4, 16, 60, None, [200, 1])  # more than the table's row holds


def test_fork_malformed_rows_become_empty(medusa):
    rng = np.random.default_rng(23)
    lens = [33, 20, 200, -4, 40, 17]
    table = tables(rng, [33, 20, 60, 0, 40, 17], 8, 16, 60)
    table[4, 1] = 77  # a page that the length needs
    same_fork(medusa, rng, lens, 8, 16, 60, [0, 9, 2, 3, 4, -7], [0] * 6, table=table)


def test_fork_pages_of_dropped_rows_are_free_at_once(medusa):
    rng = np.random.default_rng(24)
    r = same_fork(medusa, rng, [60, 60, 60], 5, 16, 12, [0, 0, 0], [0, 0, 0])
    assert to_np(r["taken"]).tolist() == [0, 1, 1]


@pytest.mark.parametrize("B,Mx,P,n,Hkv,D", [(1, 1, 16, 1, 1, 64), (3, 5, 16, 40, 2, 64), (9, 60, 32, 900, 1, 128),
                                            (64, 30, 16, 9000, 1, 64), (2, 4, 128, 33, 5, 128)])
def test_compact(medusa, B, Mx, P, n, Hkv, D):
    rng = np.random.default_rng(n)
    for frac in (0.0, 0.3, 1.0):
        pools = pool(rng, n, Hkv, P, D) if n < 1000 else [rng.integers(0, 127, (n, Hkv, P, D)).astype(np.uint8) for _ in "kv"] + [
            rng.random((n, Hkv)).astype(np.float32) for _ in "kv"]
        table = np.where(rng.random((B, Mx)) < frac, rng.integers(0, n, (B, Mx)), -1).astype(np.int32)
        if B > 1:
            table[1, 0] = n + 3  # no page: dropped
        held = (rng.random(n) < 0.05).astype(np.int32) if frac else None
        t = [to_dev(x) for x in pools]
        r = medusa.kv_pages_compact(*t, to_dev(table), held=None if held is None else to_dev(held))
        torch.cuda.synchronize()
        want_t, want_new, live, moves = R.compact(table, n, held)
        assert np.array_equal(to_np(r["page_table"]), want_t) and np.array_equal(to_np(r["new_page"]), want_new)
        assert to_np(r["live"]).tolist() == [live]
        for x in pools:
            for a, d in moves:
                x[d] = x[a]
        same_pools([to_np(x) for x in t], pools)


# ---------------------------------------------------------------------------
# together: a prompt, a fork into two branches, decode rounds with trees, a
# compaction in between; what attention reads is checked against the values that
# the definitions hold after the same steps
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rounds_with_the_paged_cache(medusa, dtype):
    rng = np.random.default_rng(30)
    B, Hkv, Hq, D, P, M, n = 3, 2, 4, 64, 16, 12, 40
    pools = list(pool(rng, n, Hkv, P, D))
    t = [to_dev(x) for x in pools]
    table, kv_len = np.full((B, M), -1, np.int32), np.zeros(B, np.int32)
    scale, node_mask = 0.125, tree("dense", 9, rng)

    def fork(src, need):
        nonlocal table, kv_len
        r = medusa.kv_pages_fork(*t, to_dev(table), to_dev(kv_len), None if src is None else to_dev(np.array(src, np.int32)),
                                 to_dev(np.array(need, np.int32)))
        w_t, w_len, _, _, copies = R.fork(table, kv_len, n, P, src, need)
        assert np.array_equal(to_np(r["page_table"]), w_t) and np.array_equal(to_np(r["kv_len"]), w_len)
        for a, d, m in copies:
            for x in pools[:2]:
                x[d, :, :m] = x[a, :, :m]
            for x in pools[2:]:
                x[d] = x[a]
        table, kv_len = w_t, w_len

    def append(k, v, rows=None, last=None):
        nonlocal pools, kv_len
        r = medusa.kv_append_q8(dev(k, dtype), dev(v, dtype), *t, to_dev(table), to_dev(kv_len),
                                rows=None if rows is None else to_dev(rows), last=to_dev(last))
        *pools, w_len, _ = R.append(k, v, *pools, table, kv_len, rows, last)
        assert np.array_equal(to_np(r["kv_len"]), w_len)
        kv_len = w_len

    draw = lambda T: as_dtype(rng.normal(0, 1, (B, T, Hkv, D)), dtype)  # noqa: E731
    fork(None, [50, 20, 0])
    append(draw(50), draw(50), last=np.array([49, 19, -1], np.int32))
    fork([0, 1, 0], [30, 30, 30])
    for step in range(4):
        k, v = draw(9), draw(9)
        q = as_dtype(rng.normal(0, 1, (B, 9, Hq, D)), dtype)
        c = dict(q=q, k_tree=k, v_tree=v, table=table, kv_len=kv_len, mask=node_mask, scale=scale, dtype=dtype,
                 **dict(zip(NAMES, pools)))
        out = medusa.tree_attention_q8(dev(q, dtype), dev(k, dtype), dev(v, dtype), *t, to_dev(table), to_dev(kv_len),
                                       to_dev(node_mask), scale)
        check(c, out.double().cpu().numpy(), reference(c))
        path = np.tile(np.array([0, 2, 8], np.int32), (B, 1))
        append(k, v, path, rng.integers(0, 3, B).astype(np.int32))
        if step == 1:
            r = medusa.kv_pages_compact(*t, to_dev(table))
            table, _, _, moves = R.compact(table, n)
            assert np.array_equal(to_np(r["page_table"]), table)
            for x in pools:
                for a, d in moves:
                    x[d] = x[a]
        fork([0, 1, 2] if step != 2 else [1, 1, -1], [10, 10, 10])
    same_pools([to_np(x) for x in t], pools)


def test_rounds_captured_and_replayed(medusa):
    """Reserve, attend and append as one graph on alternating buffers, replayed on
    new inputs: the same bits as eager calls."""
    rng = np.random.default_rng(31)
    B, Hkv, Hq, D, P, M, n, N = 2, 2, 4, 128, 32, 6, 14, 7
    base = [to_dev(x) for x in pool(rng, n, Hkv, P, D)]
    table0, len0 = to_dev(tables(rng, [70, 5], M, P, n)), to_dev(np.array([70, 5], np.int32))
    mask, need = to_dev(tree("random", N, rng)), to_dev(np.full(B, 3, np.int32))
    path, last = to_dev(np.tile(np.array([0, 1, 2], np.int32), (B, 1))), to_dev(np.array([2, 0], np.int32))
    q = torch.zeros(B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros(B, N, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, N, Hkv, D, dtype=torch.bfloat16, device="cuda")

    def make(pools):
        f = [dict(page_table=torch.empty_like(table0), kv_len=torch.empty_like(len0),
                  refs=torch.empty(n, dtype=torch.int32, device="cuda"), taken=torch.empty_like(len0)) for _ in range(2)]
        lens = [torch.empty_like(len0) for _ in range(2)]
        fws = torch.empty(medusa.kv_pages_fork_workspace(B, n), dtype=torch.uint8, device="cuda")
        aws = torch.empty(medusa.tree_attention_q8_workspace(B, N, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(q) for _ in range(2)]

        def rounds():
            t, L = f[1]["page_table"], lens[1]
            for i in range(2):
                medusa.kv_pages_fork(*pools, t, L, need=need, out=f[i], ws=fws)
                t, L = f[i]["page_table"], f[i]["kv_len"]
                medusa.tree_attention_q8(q, k, v, *pools, t, L, mask, 0.1, out=outs[i], ws=aws)
                medusa.kv_append_q8(k, v, *pools, t, L, rows=path, last=last, out=dict(kv_len=lens[i]))
                L = lens[i]
        f[1]["page_table"].copy_(table0)
        lens[1].copy_(len0)
        return rounds, outs, lens, f

    pools_a, pools_b = [x.clone() for x in base], [x.clone() for x in base]
    eager, out_a, len_a, f_a = make(pools_a)
    graphed, out_b, len_b, f_b = make(pools_b)
    warm = [x.clone() for x in base]
    w, *_ = make(warm)
    w()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graphed()
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        eager()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out_a + len_a + pools_a, out_b + len_b + pools_b):
            assert torch.equal(a, b)
        assert torch.equal(f_a[1]["page_table"], f_b[1]["page_table"])
    assert to_np(len_a[1]).tolist() == [70 + 18, 5 + 6]


def test_paged_attention_agrees_with_the_dense_cache(medusa):
    """The dense bf16 cache holding the same values gives the same attention: codes
    times a power of two are bf16 numbers."""
    c = attention_case(33, 2, 64, 4, 4, 128, 64, [500, 1000], "bf16")
    Lmax = 1100
    kc, vc = np.zeros((2, 4, Lmax, 128)), np.zeros((2, 4, Lmax, 128))
    for b in range(2):
        L = int(c["kv_len"][b])
        for h in range(4):
            kc[b, h, :L] = R.prefix(c["k_pages"], c["k_scale"], c["v_scale"], c["table"][b], L, h)
            vc[b, h, :L] = R.prefix(c["v_pages"], c["v_scale"], c["k_scale"], c["table"][b], L, h)
            kc[b, h, L:L + 64], vc[b, h, L:L + 64] = c["k_tree"][b, :, h], c["v_tree"][b, :, h]
    dense = medusa.tree_attention(dev(c["q"], "bf16"), dev(kc, "bf16"), dev(vc, "bf16"), to_dev(c["kv_len"]), to_dev(c["mask"]),
                                  c["scale"]).double().cpu().numpy()
    got = attend(medusa, c)
    ref = reference(c)
    # each side is within its own rounding of the definition; the dense kernel rounds its weights to bf16, half a step 2^-8
    assert (np.abs(got - dense) <= 2 * tolerance(c, ref) + 2.0 ** -8 * ref[1]).all()
