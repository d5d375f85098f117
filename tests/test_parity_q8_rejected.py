"""GPU tests of the paged append: the hidden state of a sequence that it rejects."""
import numpy as np
import pytest
import torch

from util import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [8, 4096])
def test_h_next_of_a_rejected_sequence_is_zero(medusa, H, dtype):
    B, T, P, D = 4, 5, 16, 64
    codes = [torch.zeros(8, 2, P, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.ones(8, 2, device="cuda") for _ in "kv"]
    table = to_dev(np.array([[0, 1], [2, -1], [3, 4], [5, 6]], np.int32))
    kv_len, last = to_dev(np.array([3, 14, 3, 3], np.int32)), to_dev(np.array([1, 4, 1, -1], np.int32))  # 1: a page is missing
    best = to_dev(np.array([4, 0, 5, 2], np.int32))  # 2: behind the last row
    rows = [torch.randn(B, T, 2, D, device="cuda").to(dtype) for _ in "kv"]
    hidden = torch.randn(B, T, H, device="cuda").to(dtype)
    out = dict(kv_len=torch.empty_like(kv_len), appended=torch.empty_like(kv_len), h_next=torch.full((B, H), 7.0, dtype=dtype, device="cuda"))
    r = medusa.kv_append_q8(*rows, *codes, *scales, table, kv_len, last=last, best_node=best, hidden_rows=hidden, out=out)
    assert r["appended"].tolist() == [2, -2, -2, 0]
    assert torch.equal(r["h_next"][0], hidden[0, 4]) and torch.equal(r["h_next"][3], hidden[3, 2])
    assert not r["h_next"][1].any() and not r["h_next"][2].any()
