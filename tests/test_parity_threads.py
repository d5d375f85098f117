"""GPU tests: the first thing that a thread does with CUDA is a call of the library."""
import threading

import pytest
import torch

from test_parity_q8 import NAMES, attention_case, dev
from util import to_dev

pytestmark = pytest.mark.gpu


def in_a_new_thread(call):
    said = []

    def run():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            said.append(repr(e))

    torch.cuda.synchronize()
    th = threading.Thread(target=run)
    th.start()
    th.join()
    torch.cuda.synchronize()
    assert not said, said


def scratch(n):
    return torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_paged_attention(medusa, dtype):
    c = attention_case(160, 2, 9, 4, 2, 64, 16, [100, 37], dtype)
    t = [dev(c[n], dtype) for n in ("q", "k_tree", "v_tree")] + [to_dev(c[n]) for n in NAMES + ("table", "kv_len", "mask")]
    want, ws = medusa.tree_attention_q8(*t, c["scale"]), scratch(medusa.tree_attention_q8_workspace(2, 9, 4, 2, 64, t[0].dtype))
    got = torch.empty_like(want)
    in_a_new_thread(lambda: medusa.tree_attention_q8(*t, c["scale"], out=got, ws=ws))
    assert torch.equal(got, want)


def test_dense_attention(medusa):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((2, 64, 4, 128), (2, 4, 400, 128), (2, 4, 400, 128)))
    kv_len, mask = torch.tensor([300, 80], dtype=torch.int32, device="cuda"), torch.full((64, 1), -1, dtype=torch.int64, device="cuda")
    want, ws = medusa.tree_attention(q, k, v, kv_len, mask, 0.1), scratch(medusa.tree_attention_workspace(2, 64, 4, 4, 128, 400))
    got = torch.empty_like(want)
    in_a_new_thread(lambda: medusa.tree_attention(q, k, v, kv_len, mask, 0.1, out=got, ws=ws))
    assert torch.equal(got, want)


def test_heads(medusa):
    g = torch.Generator(device="cuda").manual_seed(2)
    h, w1, b1, w2 = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((4, 256), (3, 256, 256), (3, 256), (3, 1000, 256)))
    want, ws = medusa.heads_topk(h, w1, b1, w2, 4), scratch(medusa.heads_topk_workspace(4, 3, 256, 1000, 4))
    got = torch.empty_like(want[0]), torch.empty_like(want[1]), None
    in_a_new_thread(lambda: medusa.heads_topk(h, w1, b1, w2, 4, out=got, ws=ws))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_projection(medusa):
    g = torch.Generator(device="cuda").manual_seed(3)
    t = medusa.tree_layout([[0, 0], [0, 1], [1, 0]], 2)
    N = t["N"]
    hidden, lm = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((2, N, 256), (1000, 256)))
    cand = torch.randint(0, 1000, (2, N), generator=g, device="cuda").to(torch.int32)
    a = (hidden, lm, cand, to_dev(t["parent"]), to_dev(t["depth"]), 2)
    want, ws = medusa.verify_project_tree(*a), scratch(medusa.verify_project_workspace(2, N, 256, 1000))
    got = {k: torch.empty_like(x) for k, x in want.items()}
    in_a_new_thread(lambda: medusa.verify_project_tree(*a, out=got, ws=ws))
    for k in want:
        assert torch.equal(got[k], want[k])
