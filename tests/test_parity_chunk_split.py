"""GPU parity of the chunk attention of short chunks, whose two streams take alternate tiles: two to four
new tokens a sequence, or one with more than 16 query heads a KV head (fewer go to another kernel)."""
import numpy as np
import pytest
import torch

from test_parity_chunk import attend, case, check, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hkv,D,P", [(2, 1, 1, 64, 16), (2, 16, 1, 128, 64), (1, 17, 1, 128, 64), (3, 12, 4, 64, 32), (4, 40, 40, 128, 128), (1, 64, 1, 64, 16)])
def test_lengths_around_tiles_and_pages(medusa, T, Hq, Hkv, D, P):
    lens = [0, 1, 15, 16, 17, 126, 127, 128, 129, 254, 255, 256, 257, 300, 700]
    check(c := case(131, len(lens), T, Hq, Hkv, D, P, lens, None, "bf16"), attend(medusa, c))


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,prefix,last", [
    (2, 2, 8, 8, 128, 64, [9000, 4000], None),           # units cut over many CTAs
    (1, 1, 34, 2, 64, 16, [20000], None),
    (7, 2, 4, 1, 128, 32, [3000, 0, 1, 900, 128, 127, 2000], [1, -1, 0, 1, 1, 0, 0]),
    (16, 2, 32, 8, 128, 32, [777 + 1000 * i for i in range(16)], [i % 2 for i in range(16)]),
])
def test_units_that_several_blocks_share(medusa, B, T, Hq, Hkv, D, P, prefix, last):
    c = case(150 + B, B, T, Hq, Hkv, D, P, prefix, last, "bf16", q_std=2.0)
    check(c, attend(medusa, c))


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,hi,wide", [
    (40, 2, 20, 20, 128, 32, 100, 0),    # one tile a unit, five units a block
    (40, 2, 20, 20, 128, 32, 300, 40),   # a wide table: units may be cut
    (60, 1, 34, 2, 64, 16, 100, 0),      # one row of 17 heads, one tile a unit
    (200, 3, 8, 8, 64, 64, 60, 0),       # ten units a block
    (30, 2, 34, 2, 128, 16, 600, 60),
])
def test_many_short_units_with_nothing_in_the_caches(medusa, B, T, Hq, Hkv, D, P, hi, wide):
    """Queries of the next segments are ready before the softmax has handed out the last one's results."""
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
            some = slice(0, 8)
            check({**c, **{n: c[n][some] for n in ("q", "table", "kv_len", "last")}}, outs[0][some].double().cpu().numpy())


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,prefix", [
    (2, 2, 8, 2, 128, 64, [900, 30]),     # units cut, the streams take alternate tiles
    (1, 1, 17, 1, 64, 32, [6000]),        # one unit, cut over many CTAs
    (40, 2, 4, 4, 64, 16, [20] * 40),     # one tile a unit
])
def test_waits_that_run_out_are_reported_and_the_next_calls_are_correct(medusa, B, T, Hq, Hkv, D, P, prefix):
    M = medusa
    c = case(141, B, T, Hq, Hkv, D, P, prefix, None, "bf16")
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


@pytest.mark.parametrize("T,Hq", [(2, 8), (1, 34)])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes(medusa, D, T, Hq):
    """Of K or V: the rows that see them, on whichever stream's tile they lie; behind the length they do not matter."""
    c = case(134, 2, T, Hq, 2, D, 16, [89, 200], None, "bf16")
    t, n = c["table"], c["kv_len"]
    for b in range(2):
        o = int(n[b]) % 16
        c["k_pages"][t[b, n[b] // 16], :, o:] = 0x7f
        c["v_pages"][t[b, n[b] // 16], :, o:] = 0xff
    check(c, attend(medusa, c))
    c["k_pages"][t[0, 2], 1, 3, 7], c["v_pages"][t[1, 10], 0, 15, D - 2] = 0xff, 0x7f
    check(c, attend(medusa, c))
    c["v_pages"][t[0, (n[0] - 1) // 16], 0, (n[0] - 1) % 16, 0] = 0x7f  # the last row's own
    check(c, attend(medusa, c))
