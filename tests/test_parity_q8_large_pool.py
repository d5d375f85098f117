"""GPU test of a pool whose codes pass 32 bits: the same calls as on a small pool, on pages
at the far end, give the same bits."""
import numpy as np
import pytest
import torch

from test_parity_q8 import attention_case, dev
from util import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,D,P,dtype", [(2, 128, 128, "bf16"), (8, 64, 16, "f32")])
def test_pages_behind_the_first_4_gib(medusa, Hkv, D, P, dtype):
    N, lens = 20, [700, 333, 40]
    c = attention_case(170, 3, N, 2 * Hkv, Hkv, D, P, lens, dtype, extra=20)
    n = c["k_pages"].shape[0]
    big = (5 << 30) // (Hkv * P * D)
    shift = big - n
    small = [to_dev(c[k]) for k in ("k_pages", "v_pages", "k_scale", "v_scale")]
    large = [torch.zeros((big, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    for x, y in zip(large, small):
        x[shift:] = y
    table, lens = to_dev(c["table"]), to_dev(c["kv_len"])
    far = torch.where(table >= 0, table + shift, table)
    rows = [dev(c[k], dtype) for k in ("k_tree", "v_tree")]
    mask, q = to_dev(c["mask"]), dev(c["q"], dtype)
    src, need = to_dev(np.array([0, 0, 1], np.int32)), to_dev(np.array([25, 25, 25], np.int32))
    held = torch.zeros(big, dtype=torch.int32, device="cuda")
    held[:shift] = 1  # so that the fork takes pages at the far end, too

    def steps(pool, t, held):
        out = [medusa.tree_attention_q8(q, *rows, *pool, t, lens, mask, c["scale"])]
        f = medusa.kv_pages_fork(*pool, t, lens, src, need, held=held)
        a = medusa.kv_append_q8(*rows, *pool, f["page_table"], f["kv_len"])
        out += [medusa.tree_attention_q8(q, *rows, *pool, f["page_table"], a["kv_len"], mask, c["scale"]), f["taken"], a["appended"]]
        return out, f["page_table"], a["kv_len"]

    got, far2, len2 = steps(large, far, held)
    want, near2, len3 = steps(small, table, None)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert torch.equal(len2, len3) and torch.equal(far2, torch.where(near2 >= 0, near2 + shift, near2))
    for x, y in zip(large, small):
        assert torch.equal(x[shift:], y) and not x[:shift].any()
    # without `held` the same pages move to the front
    m = medusa.kv_pages_compact(*large, far2)
    medusa.device_status()
    assert m["live"].item() == (near2[near2 >= 0]).unique().numel()
    again = medusa.tree_attention_q8(q, *rows, *large, m["page_table"], len2, mask, c["scale"])
    assert torch.equal(again, want[1])
