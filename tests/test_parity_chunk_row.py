"""GPU parity of the chunk attention of one row a sequence against its definition in float64: bf16
with at most 16 query heads a KV head is computed as a tree of no rows."""
import numpy as np
import pytest
import torch

import chunk_ref as K
from test_parity_chunk import NAMES, attend, case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,P", [(1, 1, 64, 16), (16, 1, 128, 64), (17, 1, 128, 64), (12, 4, 64, 32), (40, 40, 128, 128)])
def test_lengths_around_tiles_and_pages(medusa, Hq, Hkv, D, P):
    lens = [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 700]
    check(c := case(31, len(lens), 1, Hq, Hkv, D, P, [L - 1 for L in lens], None, "bf16"), attend(medusa, c))


@pytest.mark.parametrize("pages", [1, 40])
def test_sequences_without_a_row_or_a_key_are_zero(medusa, pages):
    """(short tables: units are not cut; of forty pages: they are)"""
    B = 6
    c = case(32, B, 1, 8, 2, 128, 16, [(16 * pages - 20 - b) % 16 + 16 * (pages - 2) * (pages > 1) for b in range(B)],
             [0, -1, 5, -7, 0, 0], "bf16")
    c["kv_len"][4] = -3
    c["table"][5, :] = -1
    got = attend(medusa, c)
    check(c, got)
    for b in (1, 3, 4, 5):
        assert not got[b].any()
    assert got[0].any() and got[2].any()


def test_absent_pages_and_unreadable_scales(medusa):
    c = case(33, 3, 1, 8, 2, 64, 16, [300, 299, 100], None, "bf16")
    c["table"][0, 2], c["table"][0, 7] = -1, 10 ** 6
    c["k_scale"][c["table"][1, 3], 0], c["v_scale"][c["table"][1, 5], 1] = np.nan, 0.0
    c["v_scale"][c["table"][1, 6], 0], c["k_scale"][c["table"][1, 0], 1] = np.float32(2.0 ** 65), -1.0
    check(c, attend(medusa, c))
    c["kv_len"][1] = 10 ** 6
    check(c, attend(medusa, c))


@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes(medusa, D):
    """Behind the length they do not matter; of K they make the rows that see them NaN, of V
    their column."""
    c = case(34, 2, 1, 8, 2, D, 16, [89, 200], None, "bf16")
    t, n = c["table"], c["kv_len"]
    for b in range(2):
        o = int(n[b]) % 16
        c["k_pages"][t[b, n[b] // 16], :, o:] = 0x7f
        c["v_pages"][t[b, n[b] // 16], :, o:] = 0xff
    check(c, attend(medusa, c))
    ref = K.attention(c["q"], *(c[x] for x in NAMES), t, n, None, c["scale"])
    tol = K.attention_tolerance(c["q"], c["k_pages"], t, n, c["v_scale"], ref, True)
    c["k_pages"][t[0, 2], 1, 3, 7], c["v_pages"][t[1, 4], 0, 15, D - 2] = 0xff, 0x7f
    got = attend(medusa, c)
    bad = np.zeros(got.shape, bool)
    bad[0, 0, 4:] = True
    bad[1, 0, :4, D - 2] = True
    assert np.array_equal(np.isnan(got), bad)
    assert (bad | (np.abs(np.nan_to_num(got) - ref[0]) <= tol)).all()


def test_queries_that_are_not_finite(medusa):
    c = case(35, 3, 1, 8, 2, 64, 16, [90, 0, 1000], None, "bf16")
    good = c["q"].copy()
    c["q"][0, 0, 1, 3], c["q"][1, 0, 7, 63], c["q"][2, 0, 0, 0] = np.inf, np.nan, -np.inf
    bad = np.zeros(c["q"].shape, bool)
    for b, h in ((0, 1), (1, 7), (2, 0)):
        bad[b, 0, h] = True
    ref = K.attention(good, *(c[x] for x in NAMES), c["table"], c["kv_len"], None, c["scale"])
    tol = K.attention_tolerance(good, c["k_pages"], c["table"], c["kv_len"], c["v_scale"], ref, True)
    got = attend(medusa, c)
    assert np.array_equal(np.isnan(got), bad)
    assert (bad | (np.abs(np.nan_to_num(got) - ref[0]) <= tol)).all()


def test_where_nothing_is_seen_a_query_that_is_not_finite_gives_zero(medusa):
    c = case(36, 2, 1, 4, 2, 128, 16, [50, 0], None, "bf16")
    c["table"][0, :], c["kv_len"][1] = -1, 0
    c["q"][:] = np.nan
    assert not attend(medusa, c).any()


def test_scores_that_rise_along_a_long_sequence(medusa):
    c = case(37, 1, 1, 4, 2, 64, 16, [9000], None, "bf16", q_std=0.5)
    n = c["table"].shape[1]
    for j, p in enumerate(c["table"][0]):
        if p >= 0:
            c["k_scale"][p] = 2.0 ** (-9 + 5 * j // n)
    check(c, attend(medusa, c))


def test_a_graph_replays_with_new_lengths(medusa):
    c = case(38, 3, 1, 8, 2, 128, 16, [500, 300, 7], [0, 0, 0], "bf16")
    from test_parity_chunk import tensors
    args, last = tensors(c)
    out = torch.empty_like(args[0])
    run = lambda: medusa.chunk_attention_q8(*args, last=last, out=out)
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lens, n in (([500, 300, 7], [0, 0, 0]), ([3, 301, 0], [0, -1, 0]), ([501, 17, 8], [-1, 0, 0])):
        c["kv_len"], c["last"] = np.array(lens, np.int32), np.array(n, np.int32)
        args[6].copy_(torch.from_numpy(c["kv_len"]))
        last.copy_(torch.from_numpy(c["last"]))
        g.replay()
        torch.cuda.synchronize()
        medusa.device_status()
        check(c, out.double().cpu().numpy())
