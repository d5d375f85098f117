"""GPU parity of the chunk attention over the 8-bit pages against its definition in float64,
at the lengths, tables and values where it can go wrong."""
import numpy as np
import pytest
import torch

import chunk_ref as K
from test_parity_q8 import NAMES, as_dtype, dev, pool, tables
from util import to_dev

pytestmark = pytest.mark.gpu


def case(seed, B, T, Hq, Hkv, D, P, prefix, last, dtype, q_std=1.0, extra=3):
    rng = np.random.default_rng(seed)
    n = [T if last is None else x + 1 for x in (last or [0] * B)]
    lens = [p + m for p, m in zip(prefix, n)]
    M = max(1, -(-max(lens) // P)) + 1
    n_pages = sum(-(-L // P) for L in lens) + extra
    c = dict(zip(NAMES, pool(rng, n_pages, Hkv, P, D)))
    c["table"], c["kv_len"] = tables(rng, lens, M, P, n_pages), np.array(lens, np.int32)
    c["last"] = None if last is None else np.array(last, np.int32)
    c["q"] = as_dtype(rng.normal(0, q_std, (B, T, Hq, D)), dtype)
    c.update(scale=float(np.float32(1 / np.sqrt(D))), dtype=dtype)
    return c


def tensors(c):
    return [dev(c["q"], c["dtype"]), *(to_dev(c[n]) for n in NAMES), to_dev(c["table"]), to_dev(c["kv_len"]), c["scale"]], \
        None if c["last"] is None else to_dev(c["last"])


def attend(M, c, **kw):
    args, last = tensors(c)
    out = M.chunk_attention_q8(*args, last=last, **kw)
    torch.cuda.synchronize()
    M.device_status()
    return out.double().cpu().numpy()


def check(c, got):
    ref = K.attention(c["q"], *(c[n] for n in NAMES), c["table"], c["kv_len"], c["last"], c["scale"])
    tol = K.attention_tolerance(c["q"], c["k_pages"], c["table"], c["kv_len"], c["v_scale"], ref, c["dtype"] == "bf16")
    nan = np.isnan(ref[0])
    assert np.array_equal(np.isnan(got), nan)
    err = np.abs(got - ref[0])
    assert (nan | (err <= tol)).all(), float(np.nanmax(np.where(nan, 0, err - tol)))
    zero = (ref[1] == 0) & ~nan
    assert not got[zero].any()


SHAPES = [
    # B, T, Hq, Hkv, D, P, prefix, last
    (1, 1, 1, 1, 64, 16, [0], None),                        # the first token of all
    (1, 1, 4, 4, 128, 64, [127], None),
    (3, 1, 8, 2, 128, 32, [0, 128, 1000], None),            # plain decoding, shared heads
    (2, 1, 64, 1, 64, 128, [700, 3], None),                 # 64 query heads a KV head
    (2, 9, 4, 4, 64, 16, [128, 0], None),
    (3, 16, 8, 1, 128, 16, [0, 1, 500], [15, 3, -1]),       # 128 rows: one block, two streams
    (2, 33, 7, 1, 64, 32, [200, 31], None),                 # 231 rows, a group size that divides nothing
    (1, 130, 2, 1, 128, 64, [0], None),                     # two blocks, the second of 4 rows
    (2, 129, 3, 3, 64, 16, [5, 640], [128, 0]),
    (1, 300, 4, 2, 128, 128, [77], None),
    (4, 70, 5, 1, 128, 16, [0, 10, 300, 129], [69, 0, 31, -1]),
    (1, 520, 2, 2, 64, 32, [1], None),
    (2, 260, 6, 2, 128, 64, [0, 250], [259, 100]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_see_the_slots_up_to_their_own(medusa, shape, dtype):
    c = case(sum(shape[:6]), *shape, dtype)
    check(c, attend(medusa, c))


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,prefix,last", [
    (2, 1, 8, 8, 128, 64, [9000, 4000], None),      # units cut over many CTAs
    (1, 40, 8, 2, 64, 16, [5000], None),
    (7, 3, 4, 1, 128, 32, [3000, 0, 1, 900, 128, 127, 2000], [2, -1, 0, 1, 2, 2, 0]),
    (1, 100, 5, 1, 128, 64, [6000], [90]),
])
def test_units_that_several_blocks_share(medusa, B, T, Hq, Hkv, D, P, prefix, last):
    c = case(50 + B, B, T, Hq, Hkv, D, P, prefix, last, "bf16", q_std=2.0)
    check(c, attend(medusa, c))


def test_many_sequences(medusa):
    rng = np.random.default_rng(3)
    B = 300
    c = case(4, B, 2, 2, 1, 64, 16, rng.integers(0, 90, B).tolist(), rng.integers(-1, 2, B).tolist(), "bf16")
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absent_pages_unreadable_scales_and_clamped_lengths(medusa, dtype):
    c = case(21, 4, 20, 4, 2, 64, 16, [100, 300, 50, 0], [19, 19, 5, 19], dtype)
    c["table"][0, 2], c["table"][0, 7] = -1, 10 ** 6
    c["k_scale"][c["table"][1, 3], 0], c["v_scale"][c["table"][1, 5], 1] = np.nan, 0.0
    c["v_scale"][c["table"][1, 6], 0], c["k_scale"][c["table"][1, 0], 1] = np.float32(2.0 ** 65), -1.0
    c["table"][3, :] = -1  # a sequence without a page: its rows see nothing
    check(c, attend(medusa, c))
    c["kv_len"][1], c["kv_len"][2], c["last"][0] = 10 ** 6, -5, 10 ** 6  # (absent pages behind the table's used part)
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_rows_than_slots(medusa, dtype):
    """kv_len below the chunk's rows: the first rows see nothing and are zero."""
    c = case(22, 2, 40, 4, 2, 128, 16, [0, 0], None, dtype)
    c["kv_len"][:] = [15, 0]
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes_count_where_they_are_seen_and_only_there(medusa, dtype, D):
    c = case(23, 2, 30, 4, 2, D, 16, [90, 200], [29, 20], dtype)
    t, n = c["table"], c["kv_len"]
    for b in range(2):  # slots behind the length, in the last page
        o = int(n[b]) % 16
        if o:
            c["k_pages"][t[b, n[b] // 16], :, o:] = 0x7f
            c["v_pages"][t[b, n[b] // 16], :, o:] = 0xff
    L = int(n[0])
    for slot, pages, h, code in ((L - 10, "v_pages", 0, 0x7f), (L - 4, "k_pages", 1, 0xff), (L - 3, "v_pages", 1, 0xff)):
        c[pages][t[0, slot // 16], h, slot % 16, 7] = code
    check(c, attend(medusa, c))
    c["v_pages"][t[1, 1], 0, 3, D - 1] = 0x7f  # in the prefix: every row of that head
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_that_are_not_finite(medusa, dtype):
    c = case(24, 2, 140, 4, 2, 64, 16, [90, 0], [139, 100], dtype)
    c["q"][0, 5, 1, 3], c["q"][0, 139, 2, 63], c["q"][1, 0, 0, 0] = np.inf, np.nan, -np.inf
    c["q"][1, 120] = np.nan  # behind the last row
    with np.errstate(invalid="ignore"):
        ref = K.attention(np.nan_to_num(c["q"], nan=0, posinf=0, neginf=0), *(c[n] for n in NAMES), c["table"], c["kv_len"], c["last"], c["scale"])
    got = attend(medusa, c)
    bad = np.zeros(got.shape, bool)
    bad[0, 5, 1] = bad[0, 139, 2] = bad[1, 0, 0] = True
    assert np.array_equal(np.isnan(got), bad)
    tol = K.attention_tolerance(np.nan_to_num(c["q"], nan=0, posinf=0, neginf=0), c["k_pages"], c["table"], c["kv_len"], c["v_scale"], ref, dtype == "bf16")
    assert (bad | (np.abs(np.nan_to_num(got) - ref[0]) <= tol)).all()


def test_scores_that_rise_along_the_sequence(medusa):
    """References move again and again; sums so far are scaled down each time."""
    for D, P in ((64, 16), (128, 64)):
        c = case(25, 1, 200, 2, 1, D, P, [900], None, "bf16", q_std=0.5)
        for j in range(c["table"].shape[1]):
            p = c["table"][0, j]
            if p >= 0:
                c["k_scale"][p] = 2.0 ** (-9 + 5 * j // c["table"].shape[1])
        check(c, attend(medusa, c))


def test_v_scales_far_apart(medusa):
    """A page's V scale counts as far as its weights do."""
    c = case(26, 2, 20, 4, 2, 128, 16, [300, 400], None, "bf16")
    rng = np.random.default_rng(8)
    c["v_scale"] = (2.0 ** rng.integers(-30, 1, c["v_scale"].shape)).astype(np.float32)
    check(c, attend(medusa, c))
    c["v_scale"] = (c["v_scale"] * np.float32(1.37)).astype(np.float32)  # log2 of the scale is rounded: 2^-24 of at most 32
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_and_large_queries_and_scales(medusa, dtype):
    for q_std, scale in ((1e-30, 1.0), (1e4, 1e-5), (20.0, 0.005)):
        c = case(27, 1, 20, 4, 2, 64, 32, [200], None, dtype, q_std=q_std)
        c["scale"] = scale
        check(c, attend(medusa, c))


def test_repeats_and_workspaces_give_the_same_bits(medusa):
    M = medusa
    c = case(28, 3, 140, 4, 2, 128, 16, [2000, 0, 333], [139, 100, 7], "bf16")
    args, last = tensors(c)
    a = M.chunk_attention_q8(*args, last=last)
    ws = torch.full((M.chunk_attention_q8_workspace(3, 140, 4, 2, 128),), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.full_like(a, float("nan"))
    assert M.chunk_attention_q8(*args, last=last, out=out, ws=ws) is out
    assert torch.equal(a, out)
    for _ in range(5):
        assert torch.equal(a, M.chunk_attention_q8(*args, last=last))


def test_other_streams_and_captured_calls(medusa):
    M = medusa
    c = case(29, 2, 60, 4, 2, 128, 16, [700, 40], [59, 20], "bf16")
    args, last = tensors(c)
    want = M.chunk_attention_q8(*args, last=last)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = M.chunk_attention_q8(*args, last=last, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.chunk_attention_q8(*args, last=last)
        again = M.chunk_attention_q8(*args, last=last)
    for shift in (0, 1):  # lengths change between replays
        args[6].copy_(to_dev(c["kv_len"] - shift))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(out, M.chunk_attention_q8(*args, last=last))
    M.device_status()


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,prefix", [
    (2, 1, 8, 2, 128, 64, [900, 30]),      # the streams take alternate tiles
    (2, 150, 4, 4, 64, 32, [1500, 77]),    # the streams share tiles
    (1, 300, 4, 4, 128, 32, [900]),
    (2, 20, 4, 2, 128, 64, [100, 30]),     # units that are not cut
])
def test_waits_that_run_out_are_reported_and_the_next_calls_are_correct(medusa, B, T, Hq, Hkv, D, P, prefix):
    M = medusa
    c = case(41, B, T, Hq, Hkv, D, P, prefix, None, "bf16")
    args, _ = tensors(c)

    def run():
        out = M.chunk_attention_q8(*args)
        torch.cuda.synchronize()
        return out.float().cpu().numpy()

    M.device_status()  # clear whatever an earlier test left
    before = run()
    M.device_status()
    assert np.isfinite(before).all()
    try:
        M.set_wait_limit(4)
        hurt = run()
    finally:
        M.set_wait_limit(0)
    with pytest.raises(M.MedusaError) as e:
        M.device_status()
    assert e.value.code == -5
    assert np.isnan(hurt).any() and (np.isnan(hurt) | (hurt == before)).all()
    assert np.array_equal(run(), before)
    M.device_status()


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,hi,wide", [
    (10, 4, 40, 40, 64, 64, 270, 0),     # two or three tiles a unit, units not cut
    (40, 1, 20, 20, 128, 32, 100, 0),    # one tile a unit, five units a block
    (40, 1, 20, 20, 128, 32, 300, 40),   # a wide table: units may be cut
    (30, 20, 32, 16, 64, 16, 90, 60),
    (8, 200, 16, 16, 128, 64, 60, 0),    # two streams' rows, one or two tiles
])
def test_many_short_units_with_nothing_in_the_caches(medusa, B, T, Hq, Hkv, D, P, hi, wide):
    """A block takes up one unit after the other: their queries are made ready ahead of the softmax,
    by one segment and, where segments have a tile, by two; cold memory changes who comes first."""
    M, flush = medusa, torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for seed in range(4):
        rng = np.random.default_rng(seed)
        c = case(seed, B, T, Hq, Hkv, D, P, rng.integers(0, hi, B).tolist(), rng.integers(0, T, B).tolist(), "bf16")
        c["table"] = np.concatenate([c["table"], np.full((B, wide), -1, np.int32)], 1)
        args, last = tensors(c)
        outs = []
        for _ in range(3):
            flush.zero_()
            torch.cuda.synchronize()
            outs.append(M.chunk_attention_q8(*args, last=last))
            torch.cuda.synchronize()
        M.device_status()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        if seed == 0:
            some = slice(0, 6)
            part = {**c, **{n: c[n][some] for n in ("q", "table", "kv_len", "last")}}
            check(part, outs[0][some].double().cpu().numpy())
