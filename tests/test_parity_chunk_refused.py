"""A sequence that the rotating append refuses, and the attention behind it: with last = appended - 1 its rows
are zero, and the other sequences' are what they are without it."""
import numpy as np
import pytest
import torch

from test_parity_append_rope import case as append_case
from test_parity_chunk import check
from test_parity_q8 import NAMES, dev
from util import to_dev, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lens,last", [(1, [40, 33, 0], None), (30, [40, 33, 0], [29, 10, 5]), (200, [0, 300, 15], [199, 130, 0])])
@pytest.mark.parametrize("what", ["page", "kv_len"])
def test_refused_rows_are_answered_with_zeros(medusa, T, lens, last, dtype, what):
    M = medusa
    c = append_case(T, 3, T, 4, 2, 64, 16, 32, lens, last, dtype)
    if what == "page":
        c["table"][1, lens[1] // 16] = -1
    else:
        c["kv_len"][1] = -5
    pools = [to_dev(c[n].copy()) for n in NAMES]
    table = to_dev(c["table"])
    r = M.kv_append_rope_q8(dev(c["k"], dtype), dev(c["v"], dtype), *pools, table, to_dev(c["kv_len"]), to_dev(c["f"]),
                            last=None if last is None else to_dev(c["last"]), q=dev(c["q"], dtype))
    assert to_np(r["appended"])[1] == -2 and (to_np(r["appended"])[[0, 2]] > 0).all()
    wrote = r["appended"] - 1
    out = M.chunk_attention_q8(r["q"], *pools, table, r["kv_len"], 0.125, last=wrote)
    M.device_status()
    got = out.double().cpu().numpy()
    assert not got[1].any() and got[0].any() and got[2].any()
    check(dict(zip(NAMES, (to_np(x) for x in pools)), q=r["q"].double().cpu().numpy(), table=c["table"], kv_len=to_np(r["kv_len"]),
               last=to_np(wrote), scale=0.125, dtype=dtype), got)
    # captured together, replayed on lengths that refuse the other sequence
    kv_len = to_dev(c["kv_len"])
    graph = torch.cuda.CUDAGraph()
    k, v, q = dev(c["k"], dtype), dev(c["v"], dtype), dev(c["q"], dtype)
    f, last_t = to_dev(c["f"]), None if last is None else to_dev(c["last"])
    with torch.cuda.graph(graph):
        s = M.kv_append_rope_q8(k, v, *pools, table, kv_len, f, last=last_t, q=q)
        out = M.chunk_attention_q8(s["q"], *pools, table, s["kv_len"], 0.125, last=s["appended"] - 1)
    kv_len.copy_(to_dev(np.array([10 ** 6, -1, lens[2]], np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    M.device_status()
    assert not out[:2].any() and out[2].any() and to_np(s["appended"]).tolist()[:2] == [-2, -2]
