"""GPU tests of the paged tree attention called from several threads and with as many
sequences as a call takes."""
import threading

import numpy as np
import pytest
import torch

from test_parity_q8 import NAMES, attend, attention_case, check, dev, reference
from util import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", [(1, 2, 1, 64, 16), (20, 1, 1, 128, 16), (70, 1, 1, 128, 32)])
def test_attention_of_1024_sequences(medusa, N, Hq, Hkv, D, P, dtype):
    lens = np.random.default_rng(N).integers(0, 60, 1024).tolist()
    c = attention_case(50 + N, 1024, N, Hq, Hkv, D, P, lens, dtype)
    check(c, attend(medusa, c), reference(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_of_different_batches_from_two_threads(medusa, dtype):
    """A call of 1024 sequences and calls of one, launched at the same time: what one call
    needs of the kernel's settings is not taken away by the other."""
    cases = [attention_case(110, 1024, 1, 2, 2, 128, 16, [5] * 1024, dtype), attention_case(111, 1, 1, 2, 2, 128, 16, [5], dtype)]
    t = [[dev(c[n], dtype) for n in ("q", "k_tree", "v_tree")] + [to_dev(c[n]) for n in NAMES + ("table", "kv_len", "mask")] for c in cases]
    want = [medusa.tree_attention_q8(*x, c["scale"]) for x, c in zip(t, cases)]
    torch.cuda.synchronize()
    wrong = []

    def calls(x, c, w, n):
        s = torch.cuda.Stream()
        out = torch.empty_like(w)
        ws = torch.empty(medusa.tree_attention_q8_workspace(*x[0].shape[:3], x[3].shape[1], x[0].shape[3], x[0].dtype),
                         dtype=torch.uint8, device="cuda")
        try:
            for i in range(n):
                medusa.tree_attention_q8(*x, c["scale"], out=out, ws=ws, stream=s)
                if i % 100 == 99:
                    s.synchronize()
            s.synchronize()
            if not torch.equal(out, w):
                wrong.append("outputs differ")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=(*a, n)) for a in zip(t, cases, want) for n in (3000, 3000)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong[:3]
