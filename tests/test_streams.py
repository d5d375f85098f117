"""Calls on a stream that is not the current one: what a call allocates belongs to the
stream that it works on, so that nothing else gets that memory before its kernels ran."""
import contextlib

import numpy as np
import pytest
import torch

from test_parity_q8 import NAMES, attention_case, dev
from util import to_dev


# ---------------------------------------------------------------------------
# which stream is current while a call allocates, with streams that are names
class Stream(str):
    device = "cuda:0"


@pytest.fixture
def streams(monkeypatch):
    from medusa_speculative_decoding_gb300 import api
    now = [Stream("main")]

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(api.torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(api.torch.cuda, "stream", stream)
    return now


def test_the_given_stream_is_current_while_a_call_allocates(streams):
    from medusa_speculative_decoding_gb300 import api

    at = []

    @api._in_stream
    def call(x, out=None, stream=None):
        at.append(streams[-1])

    call(1)
    call(1, out=2, stream=Stream("side"))
    call(1, 2, Stream("side"))
    call(1, 2, Stream("main"))
    assert at == ["main", "side", "side", "main"]
    assert streams == ["main"]


@pytest.mark.parametrize("name", ["heads_topk", "heads_topk_static", "build_tree", "tree_attention", "verify_accept_tree",
                                  "verify_accept_tree_sample", "verify_project_tree", "verify_accept_chain", "kv_compact",
                                  "tree_attention_q8", "kv_append_q8", "kv_pages_fork", "kv_pages_compact"])
def test_every_call_that_allocates_does_so(streams, monkeypatch, name):
    """The first thing that a call does with its stream's memory or arguments happens
    with that stream current."""
    from medusa_speculative_decoding_gb300 import api
    import inspect
    at = []

    class Looked(Exception):
        pass

    def look(*a, **k):
        at.append(streams[-1])
        raise Looked

    for f in ("_need", "_need_pool"):
        monkeypatch.setattr(api, f, look)
    f = getattr(api, name)
    n = [p for p in inspect.signature(f).parameters.values() if p.default is p.empty]
    with pytest.raises(Looked):
        f(*[torch.zeros(1) for _ in n], stream=Stream("side"))
    assert at == ["side"]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    from medusa_speculative_decoding_gb300 import api
    monkeypatch.setattr(api.torch.cuda, "current_device", lambda: 0)
    assert not api._elsewhere(0, "s") and not api._elsewhere(0, None) and api._elsewhere(1, None)
    with pytest.raises(ValueError, match="stream"):
        api._elsewhere(1, "s")


# ---------------------------------------------------------------------------
def on_a_busy_stream(call, sizes):
    """The call's result on a side stream that is still busy when the call returns, while
    the current stream takes and fills whatever memory of these sizes is free."""
    fill = lambda: [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(6)]  # noqa: E731
    s = torch.cuda.Stream()
    fill()  # (the allocator has such blocks from now on)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)  # about 50 ms
    result = call(s)
    taken = fill()
    assert not s.query()
    torch.cuda.synchronize()
    assert all((t == 0x7f).all() for t in taken)
    return result


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,lens", [(64, [900, 400]), (200, [1500, 70])])
def test_paged_attention(medusa, N, lens, dtype):
    c = attention_case(150 + N, 2, N, 4, 4, 128, 64, lens, dtype)
    t = [dev(c[n], dtype) for n in ("q", "k_tree", "v_tree")] + [to_dev(c[n]) for n in NAMES + ("table", "kv_len", "mask")]
    want = medusa.tree_attention_q8(*t, c["scale"])
    ws = medusa.tree_attention_q8_workspace(2, N, 4, 4, 128, t[0].dtype)
    got = on_a_busy_stream(lambda s: medusa.tree_attention_q8(*t, c["scale"], stream=s), [ws, want.numel() * want.element_size()])
    assert torch.equal(got, want)
    medusa.device_status()


@pytest.mark.gpu
def test_dense_attention(medusa):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((1, 64, 4, 128), (1, 4, 4200, 128), (1, 4, 4200, 128)))
    kv_len, mask = torch.tensor([4000], dtype=torch.int32, device="cuda"), torch.full((64, 1), -1, dtype=torch.int64, device="cuda")
    want = medusa.tree_attention(q, k, v, kv_len, mask, 0.1)
    ws = max(16, medusa.tree_attention_workspace(1, 64, 4, 4, 128, 4200))
    got = on_a_busy_stream(lambda s: medusa.tree_attention(q, k, v, kv_len, mask, 0.1, stream=s), [ws, want.numel() * 4])
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_heads_and_acceptance(medusa):
    g = torch.Generator(device="cuda").manual_seed(2)
    h, w1, b1, w2 = (torch.randn(s, generator=g, device="cuda") for s in ((2, 256), (3, 256, 256), (3, 256), (3, 1000, 256)))
    want = medusa.heads_topk(h, w1, b1, w2, 4)
    got = on_a_busy_stream(lambda s: medusa.heads_topk(h, w1, b1, w2, 4, stream=s), [medusa.heads_topk_workspace(2, 3, 256, 1000, 4), 512])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    p, q = (torch.softmax(torch.randn(s, 5000, generator=g, device="cuda"), -1) for s in (4 * 5, 4 * 4))
    p, q = p.view(4, 5, 5000), q.view(4, 4, 5000)
    draft = torch.randint(0, 5000, (4, 4), generator=g, device="cuda").to(torch.int32)
    want = medusa.verify_accept_chain(p, q, draft, 7, 1)
    got = on_a_busy_stream(lambda s: medusa.verify_accept_chain(p, q, draft, 7, 1, stream=s), [medusa.verify_chain_workspace(4, 4, 5000), 512])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_pages(medusa):
    """Fork with copies, append and compaction."""
    rng = np.random.default_rng(3)
    n, B, M, P = 600, 8, 40, 16
    pools = [rng.integers(0, 127, (n, 2, P, 64)).astype(np.uint8) for _ in "kv"] + [np.ones((n, 2), np.float32) for _ in "kv"]
    lens = rng.integers(100, 500, B).astype(np.int32)
    perm, table = rng.permutation(n).tolist(), np.full((B, M), -1, np.int32)
    for b in range(B):
        for j in range(-(-int(lens[b]) // P)):
            table[b, j] = perm.pop()
    src, need = to_dev(np.array([0, 0, 2, 2, 4, 4, -1, 7], np.int32)), to_dev(np.full(B, 30, np.int32))
    rows = [torch.randn(B, 9, 2, 64, device="cuda") for _ in "kv"]
    table, lens = to_dev(table), to_dev(lens)

    def steps(s):
        t = [to_dev(x) for x in pools]
        torch.cuda.current_stream().synchronize()
        a = medusa.kv_pages_fork(*t, table, lens, src, need, stream=s)
        b = medusa.kv_append_q8(*rows, *t, a["page_table"], a["kv_len"], stream=s)
        c = medusa.kv_pages_compact(*t, a["page_table"], stream=s)
        return t + [x for r in (a, b, c) for x in r.values() if x is not None]

    want = steps(None)
    got = on_a_busy_stream(steps, [medusa.kv_pages_fork_workspace(B, n), medusa.kv_pages_compact_workspace(n), 4 * B * M, 4 * n, 4 * B])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_side_stream_inside_a_capture(medusa):
    """A graph whose calls work on two streams, workspaces and outputs from its own memory."""
    cases = [attention_case(180, 2, 64, 4, 4, 128, 64, [900, 400], "bf16"), attention_case(181, 3, 9, 4, 2, 64, 16, [300, 1, 70], "f32")]
    t = [[dev(c[n], c["dtype"]) for n in ("q", "k_tree", "v_tree")] + [to_dev(c[n]) for n in NAMES + ("table", "kv_len", "mask")] for c in cases]
    want = [medusa.tree_attention_q8(*x, c["scale"]) for x, c in zip(t, cases)]
    forked = medusa.kv_pages_fork(*t[0][3:9])
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = [medusa.tree_attention_q8(*t[0], cases[0]["scale"]), medusa.tree_attention_q8(*t[1], cases[1]["scale"], stream=side)]
        again = medusa.kv_pages_fork(*t[0][3:9], stream=side)
        got.append(medusa.tree_attention_q8(*t[0], cases[0]["scale"], stream=side))
        main.wait_stream(side)
    for _ in range(5):
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, w in zip(got, (*want, want[0])):
            assert torch.equal(x, w)
        for k in forked:
            assert torch.equal(again[k], forked[k])
    medusa.device_status()
