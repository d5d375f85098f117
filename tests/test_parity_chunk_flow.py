"""The rotating append, the chunk attention, the rotation of tree rows and the acceptance by
drawn tokens used together, and the chunk attention at sizes where its work is cut in many ways."""
import threading

import numpy as np
import pytest
import torch

import chunk_ref as K
import q8_ref as R
from test_parity_chunk import case, check, tensors
from test_parity_q8 import NAMES, as_dtype, dev, pool, tree
from test_parity_rope import freqs
from util import to_dev, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_in_pieces_then_sampled_rounds(medusa, dtype):
    """Ragged prompts written and answered in two pieces, then rounds of tree attention, acceptance
    and append; what is answered is checked against the pages that the calls before left."""
    M, rng = medusa, np.random.default_rng(60)
    B, Hkv, Hq, D, P, Mx, n, V, scale = 3, 2, 6, 64, 16, 14, 48, 400, 0.125
    pools = [to_dev(x) for x in pool(rng, n, Hkv, P, D)]
    f = to_dev(freqs(16))
    table, kv_len = torch.full((B, Mx), -1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = lambda T, H: as_dtype(rng.normal(0, 1, (B, T, H, D)), dtype)  # noqa: E731

    def reserve(need):
        nonlocal table
        table = M.kv_pages_fork(*pools, table, kv_len, need=to_dev(np.array(need, np.int32)))["page_table"]

    for T, last in ((90, [89, 20, -1]), (33, [10, 32, 32])):
        reserve([x + 1 for x in last])
        q, k, v = rows(T, Hq), rows(T, Hkv), rows(T, Hkv)
        before = [to_np(x) for x in pools]
        last_t = to_dev(np.array(last, np.int32))
        r = M.kv_append_rope_q8(dev(k, dtype), dev(v, dtype), *pools, table, kv_len, f, last=last_t, q=dev(q, dtype))
        _, _, ks, vs, L, count, _, _ = K.append(k, v, *before, to_np(table), to_np(kv_len), freqs(16), False, None, last)
        assert np.array_equal(to_np(r["kv_len"]), L) and np.array_equal(to_np(pools[2]), ks) and np.array_equal(to_np(pools[3]), vs)
        kv_len = r["kv_len"]
        out = M.chunk_attention_q8(r["q"], *pools, table, kv_len, scale, last=last_t)
        c = dict(zip(NAMES, (to_np(x) for x in pools)), q=r["q"].double().cpu().numpy(), table=to_np(table), kv_len=L, last=np.array(last),
                 scale=scale, dtype=dtype)
        check(c, out.double().cpu().numpy())
    N = 9
    mask, parent = tree("dense", N, rng), np.array([-1] + [(i - 1) // 4 for i in range(1, N)], np.int32)
    depth = np.array([0, 1, 1, 1, 1, 2, 2, 2, 2], np.int32)
    accepted = 0
    for _ in range(4):
        q, k, v = rows(N, Hq), rows(N, Hkv), rows(N, Hkv)
        qt, kt = M.rope_rows(dev(q, dtype), dev(k, dtype), kv_len, f, depth=to_dev(depth))
        out = M.tree_attention_q8(qt, kt, dev(v, dtype), *pools, table, kv_len, to_dev(mask), scale)
        ref = R.attention(qt.double().cpu().numpy(), kt.double().cpu().numpy(), v, *(to_np(x) for x in pools), to_np(table), to_np(kv_len), mask, scale)
        assert np.abs(out.double().cpu().numpy() - ref[0]).max() < (0.05 if dtype == "bf16" else 1e-4)  # (its own tests say how near)
        p = rng.dirichlet(np.full(V, 0.02), (B, N)).astype(np.float32)
        cand = np.argsort(-p[:, np.maximum(parent, 0)], -1)[np.arange(B)[:, None], np.arange(N), (np.arange(N) - 1) % 4].astype(np.int32)
        u = rng.random((B, 3)).astype(np.float32)
        d = M.verify_accept_tree_draw(*(to_dev(x) for x in (p, cand, parent, depth, u)), 2)
        want = K.verify(p, cand, parent, u, 2)
        for name, x in want.items():
            assert np.array_equal(to_np(d[name]), x), name
        accepted += int(want["accept_len"].sum())
        reserve([4] * B)
        L = to_np(kv_len)
        a = M.kv_append_q8(kt, dev(v, dtype), *pools, table, kv_len, rows=d["path_nodes"].clamp(min=0).contiguous(), last=d["accept_len"])
        kv_len = a["kv_len"]
        assert np.array_equal(to_np(kv_len), L + want["accept_len"] + 1)
    assert accepted > 0
    # one decoded token, written and answered
    reserve([1] * B)
    q, k, v = rows(1, Hq), rows(1, Hkv), rows(1, Hkv)
    r = M.kv_append_rope_q8(dev(k, dtype), dev(v, dtype), *pools, table, kv_len, f, q=dev(q, dtype))
    out = M.chunk_attention_q8(r["q"], *pools, table, r["kv_len"], scale)
    check(dict(zip(NAMES, (to_np(x) for x in pools)), q=r["q"].double().cpu().numpy(), table=to_np(table), kv_len=to_np(r["kv_len"]), last=None,
               scale=scale, dtype=dtype), out.double().cpu().numpy())
    M.device_status()


def test_accepted_rows_may_be_turned_before_or_on_the_way(medusa):
    """A tree's accepted branch, rotated by rope_rows and appended, or appended unrotated: the same
    values but for the rounding between, and the same scales where 316 and 448 choose alike."""
    M, rng = medusa, np.random.default_rng(61)
    B, T, Hkv, D, P = 2, 9, 2, 128, 16
    pools = pool(rng, 8, Hkv, P, D)
    table, L = to_dev(np.array([[0, 1, 2], [3, 4, 5]], np.int32)), to_dev(np.array([20, 30], np.int32))
    k, v = dev(rng.normal(0, 1, (B, T, Hkv, D)), "f32"), dev(rng.normal(0, 1, (B, T, Hkv, D)), "f32")
    path, depth = to_dev(np.array([[0, 2, 7], [0, 4, 5]], np.int32)), to_dev(np.array([0, 1, 1, 1, 1, 2, 2, 2, 2], np.int32))
    f = to_dev(freqs(64))
    a, b = [to_dev(x) for x in pools], [to_dev(x) for x in pools]
    _, kt = M.rope_rows(k, k, L, f, depth=depth)
    M.kv_append_q8(kt, v, *a, table, L, rows=path)
    M.kv_append_rope_q8(k, v, *b, table, L, f, rows=path)
    assert torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])
    x, y = (R.decode(to_np(p[0])) * to_np(p[2])[:, :, None, None] for p in (a, b))
    held = np.zeros((8, 1, P, 1), bool)  # (slots behind the lengths hold anything)
    held[[0, 3, 4]], held[1, :, :23 - 16], held[5, :, :33 - 32] = True, True, True
    tol = 2 * 2.0 ** -4 * np.maximum(np.abs(x), np.abs(y)) + 2.0 ** -9 * np.maximum(to_np(a[2]), to_np(b[2]))[:, :, None, None]
    assert (~held | (np.abs(x - y) <= tol)).all()


def test_a_step_captured_and_replayed(medusa):
    """Append, attention, acceptance as one graph, twice in it, replayed on new inputs: the same bits as
    eager calls."""
    M, rng = medusa, np.random.default_rng(62)
    B, T, Hkv, Hq, D, P, n, V = 2, 40, 2, 4, 128, 16, 40, 500
    base = [to_dev(x) for x in pool(rng, n, Hkv, P, D)]
    pools = [x.clone() for x in base]
    table, L = to_dev(np.arange(n, dtype=np.int32).reshape(2, 20)), to_dev(np.array([100, 7], np.int32))
    f, last = to_dev(freqs(64)), to_dev(np.array([39, 11], np.int32))
    parent, depth = to_dev(np.array([-1, 0, 0], np.int32)), to_dev(np.array([0, 1, 1], np.int32))
    x = dict(q=torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda"), k=torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device="cuda"),
             v=torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device="cuda"), p=torch.zeros(B, 3, V, device="cuda"),
             cand=torch.zeros(B, 3, dtype=torch.int32, device="cuda"), u=torch.zeros(B, 2, device="cuda"))

    def step():
        r = M.kv_append_rope_q8(x["k"], x["v"], *pools, table, L, f, last=last, q=x["q"])
        o = M.chunk_attention_q8(r["q"], *pools, table, r["kv_len"], 0.1, last=last)
        d = M.verify_accept_tree_draw(x["p"], x["cand"], parent, depth, x["u"], 1)
        return [o, r["q"], r["kv_len"], d["next_tok"], d["accept_len"]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first, second = step(), step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for name in "qkv":
            x[name].normal_(generator=g)
        x["p"].copy_(torch.softmax(4 * torch.randn(B, 3, V, device="cuda", generator=g), -1))
        x["cand"].copy_(x["p"].topk(3, -1).indices[:, 0])
        x["u"].uniform_(generator=g)
        for p, b in zip(pools, base):
            p.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        after = [p.clone() for p in pools]
        for p, b in zip(pools, base):
            p.copy_(b)
        step()
        want = step()
        torch.cuda.synchronize()
        for a, b, w in zip(first, second, want):
            assert torch.equal(b, w) and a.shape == w.shape
        assert all(torch.equal(p, a) for p, a in zip(pools, after))
    M.device_status()


def exact_on_gpu(c):
    """The definition in float64 on the GPU, for sizes that loops over rows would take minutes for."""
    B, T, Hq, D = c["q"].shape
    Hkv, P = c["k_pages"].shape[1], c["k_pages"].shape[2]
    G = Hq // Hkv
    out = torch.zeros(c["q"].shape, dtype=torch.float64, device="cuda")
    values = {n: torch.from_numpy(R.decode(c[n + "_pages"])).cuda() * torch.from_numpy(c[n + "_scale"]).cuda().double()[:, :, None, None] for n in "kv"}
    q = torch.from_numpy(c["q"]).cuda()
    for b in range(B):
        L, n = int(c["kv_len"][b]), T if c["last"] is None else int(c["last"][b]) + 1
        pages = torch.from_numpy(c["table"][b, :-(-L // P)].astype(np.int64)).cuda()
        hidden = torch.ones(n, L, dtype=torch.bool, device="cuda").triu(L - n + 1)
        for h in range(Hkv):
            k, v = (values[x][pages, h].reshape(-1, D)[:L] for x in "kv")
            for g in range(h * G, h * G + G):
                z = (q[b, :n, g] @ k.T * c["scale"]).masked_fill(hidden, -float("inf"))
                out[b, :n, g] = torch.softmax(z, -1) @ v
    return out.cpu().numpy()


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,prefix,last", [
    (2, 1500, 8, 2, 128, 64, [2000, 0], [1499, 700]),
    (1, 2100, 6, 6, 64, 16, [0], None),
    (3, 700, 10, 2, 128, 16, [5000, 100, 1], [699, 255, -1]),
    (1, 5, 64, 1, 128, 32, [20000], None),
    (20, 3, 16, 4, 64, 128, [100 * i for i in range(20)], [i % 3 for i in range(20)]),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_chunks_and_caches(medusa, B, T, Hq, Hkv, D, P, prefix, last, dtype):
    c = case(70 + B, B, T, Hq, Hkv, D, P, prefix, last, dtype)
    args, last_t = tensors(c)
    got = medusa.chunk_attention_q8(*args, last=last_t)
    medusa.device_status()
    got, want = got.double().cpu().numpy(), exact_on_gpu(c)
    # scores of these inputs stay below 12 in magnitude sum, V below 30: the terms of
    # chunk_ref.attention_tolerance with spread <= max |v| = 30 and the sums' rounding over 25000 keys
    err = np.abs(got - want)
    tol = np.abs(want) * 2.0 ** -8 + 30 * (2.0 ** -11 + 2.1 * 2.0 ** -16) if dtype == "bf16" else np.abs(want) * 2.0 ** -24 + 30 * 50064 * 2.0 ** -24
    assert (err <= tol).all() and np.sqrt((err ** 2).mean()) <= (2.0 ** -9 if dtype == "bf16" else 1e-5) * np.sqrt((want ** 2).mean())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,P", [(1, 2, 1, 64, 16), (20, 1, 1, 128, 16), (140, 2, 1, 128, 32)])
def test_1024_sequences(medusa, T, Hq, Hkv, D, P, dtype):
    rng = np.random.default_rng(T)
    c = case(80 + T, 1024, T, Hq, Hkv, D, P, rng.integers(0, 40, 1024).tolist(), np.minimum(rng.integers(-1, 6, 1024), T - 1).tolist(), dtype)
    args, last = tensors(c)
    check(c, medusa.chunk_attention_q8(*args, last=last).double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_of_different_batches_from_two_threads(medusa, dtype):
    cases = [case(90, 1024, 1, 2, 2, 128, 16, [5] * 1024, None, dtype), case(91, 1, 200, 2, 2, 128, 16, [5], None, dtype)]
    t = [tensors(c)[0] for c in cases]
    want = [medusa.chunk_attention_q8(*x) for x in t]
    torch.cuda.synchronize()
    wrong = []

    def calls(x, w):
        s = torch.cuda.Stream()
        out = torch.empty_like(w)
        ws = torch.empty(medusa.chunk_attention_q8_workspace(*x[0].shape[:3], x[1].shape[1], x[0].shape[3], x[0].dtype), dtype=torch.uint8, device="cuda")
        try:
            for i in range(1000):
                medusa.chunk_attention_q8(*x, out=out, ws=ws, stream=s)
                if i % 100 == 99:
                    s.synchronize()
            s.synchronize()
            if not torch.equal(out, w):
                wrong.append("outputs differ")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=calls, args=a) for a in zip(t, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong[:3]


@pytest.mark.parametrize("Hkv,D,P,dtype", [(2, 128, 128, "bf16"), (8, 64, 16, "f32")])
def test_pages_behind_the_first_4_gib(medusa, Hkv, D, P, dtype):
    M = medusa
    c = case(95, 3, 60, 2 * Hkv, Hkv, D, P, [700, 333, 40], [59, 20, 5], dtype, extra=20)
    n = c["k_pages"].shape[0]
    big = (5 << 30) // (Hkv * P * D)
    shift = big - n
    small = [to_dev(c[k]) for k in NAMES]
    large = [torch.zeros((big, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    for x, y in zip(large, small):
        x[shift:] = y
    args, last = tensors(c)
    q, table, kv_len = args[0], args[5], args[6]
    far = torch.where(table >= 0, table + shift, table)
    rng = np.random.default_rng(96)
    k, v = (dev(rng.normal(0, 3, (3, 60, Hkv, D)), dtype) for _ in "kv")
    start, f = kv_len - last - 1, to_dev(freqs(D // 2))
    got = []
    for pools, t in ((small, table), (large, far)):
        r = M.kv_append_rope_q8(k, v, *pools, t, start, f, last=last, q=q)
        got.append([r["appended"], r["q"], M.chunk_attention_q8(r["q"], *pools, t, r["kv_len"], c["scale"], last=last)])
    M.device_status()
    assert (got[0][0] > 0).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for x, y in zip(large, small):
        assert torch.equal(x[shift:], y) and not x[:shift].any()


def test_outputs_are_all_that_is_written(medusa):
    M = medusa
    for T, last in ((9, [8, 3]), (300, [299, 20])):
        c = case(97, 2, T, 4, 2, 64, 16, [100, 50], last, "bf16")
        args, last_t = tensors(c)
        big = torch.full((4, T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        M.chunk_attention_q8(*args, last=last_t, out=big[1:3])
        assert (big[0] == 7).all() and (big[3] == 7).all() and not (big[1:3] == 7).any()
        q = torch.full((4, T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        k = torch.full((4, T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        x = dev(c["q"], "bf16")
        M.rope_rows(x, x[:, :, :2].contiguous(), args[6], to_dev(freqs(16)), out=(q[1:3], k[1:3]))
        for y in (q, k):
            assert (y[0] == 7).all() and (y[3] == 7).all()


CALLS = {
    "rope_rows": lambda z, p: dict(q=z(2, 1, 4, 64, d=torch.float32), k=z(2, 1, 2, 64, d=torch.float32), kv_len=p["kv_len"],
                                   inv_freq=z(32, d=torch.float32), depth=z(1)),
    "kv_append_rope_q8": lambda z, p: dict(k_rows=z(2, 1, 2, 64, d=torch.float32), v_rows=z(2, 1, 2, 64, d=torch.float32), **p,
                                           inv_freq=z(32, d=torch.float32), last=z(2), q=z(2, 1, 4, 64, d=torch.float32)),
    "chunk_attention_q8": lambda z, p: dict(q=z(2, 1, 4, 64, d=torch.float32), **p, scale=0.1, last=z(2)),
    "verify_accept_tree_draw": lambda z, p: dict(probs=z(2, 3, 5, d=torch.float32), cand=z(2, 3), parent=z(3), depth=z(3),
                                                 u=z(2, 2, d=torch.float32), max_depth=1),
}


@pytest.mark.parametrize("name", CALLS)
def test_missing_and_wrong_arguments(medusa, name):
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    p = dict(k_pages=z(4, 2, 16, 64, d=torch.uint8), v_pages=z(4, 2, 16, 64, d=torch.uint8), k_scale=torch.ones(4, 2, device="cuda"),
             v_scale=torch.ones(4, 2, device="cuda"), page_table=z(2, 3), kv_len=z(2))
    args = CALLS[name](z, p)
    f = getattr(medusa, name)
    optional = ("depth", "last", "q" if name == "kv_append_rope_q8" else "", "k")
    for k in args:
        if k in ("scale", "max_depth"):
            continue
        for wrong in [args[k].cpu(), args[k].to(torch.float64), torch.cat([args[k]] * 2)] + ([] if k in optional else [None]):
            if k == "inv_freq" and wrong is not None and wrong.is_cuda and wrong.dtype == torch.float32:
                with pytest.raises(medusa.MedusaError):  # more frequencies than half a head
                    f(**{**args, k: wrong})
                continue
            with pytest.raises(ValueError):
                f(**{**args, k: wrong})
    torch.cuda.synchronize()
    f(**args)
    torch.cuda.synchronize()
