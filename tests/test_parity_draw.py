"""GPU parity of tree acceptance by drawn tokens against its definition in whole numbers."""
import numpy as np
import pytest
import torch

import chunk_ref as K
from util import to_dev

pytestmark = pytest.mark.gpu


def parents(kind, N, rng):
    if kind == "chain":
        return np.arange(N, dtype=np.int32) - 1
    if kind == "dense":
        return np.array([-1] + [(i - 1) // 4 for i in range(1, N)], np.int32)
    return np.array([-1] + [int(rng.integers(0, i)) for i in range(1, N)], np.int32)


def case(seed, B, N, V, kind, peak=5.0):
    rng = np.random.default_rng(seed)
    par = parents(kind, N, rng)
    depth = np.zeros(N, np.int32)
    for i in range(1, N):
        depth[i] = depth[par[i]] + 1
    z = rng.normal(0, peak, (B, N, V))
    p = np.exp(z - z.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True)).astype(np.float32)
    cand = np.zeros((B, N), np.int32)
    best = np.argsort(-p, -1, kind="stable")[:, :, :16]
    seen = {}
    for i in range(N):
        r = seen.get(par[i], 0)
        seen[par[i]] = r + 1
        cand[:, i] = best[:, max(par[i], 0), min(r, best.shape[2] - 1)]
    u = rng.random((B, depth.max() + 1)).astype(np.float32)
    return dict(probs=p, cand=cand, parent=par, depth=depth, u=u, max_depth=int(depth.max()))


def run(M, c, **kw):
    r = M.verify_accept_tree_draw(*(to_dev(c[n]) for n in ("probs", "cand", "parent", "depth", "u")), c["max_depth"], **kw)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in r.items()}


def check(c, got):
    want = K.verify(c["probs"], c["cand"], c["parent"], c["u"], c["max_depth"])
    for n, x in want.items():
        assert np.array_equal(got[n], x), n


@pytest.mark.parametrize("B,N,V,kind", [
    (1, 1, 1, "chain"), (2, 1, 5, "chain"), (3, 9, 100, "random"), (2, 64, 1000, "random"), (1, 64, 8192, "random"), (2, 33, 8193, "dense"),
    (1, 20, 32000, "random"), (3, 5, 4097, "chain"), (2, 341, 130, "dense"), (1, 512, 33, "chain"), (40, 16, 1001, "dense"),
])
def test_tokens_and_paths(medusa, B, N, V, kind):
    c = case(B * 7 + N, B, N, V, kind)
    check(c, run(medusa, c))


@pytest.mark.parametrize("B,N,V", [(3, 200, 32001), (2, 60, 128256), (1, 400, 40000)])
def test_walks_over_rows_too_many_to_draw_from_all(medusa, B, N, V):
    assert B * N * V * 4 > 48 << 20
    c = case(N, B, N, V, "dense", peak=6.0)
    check(c, run(medusa, c))


def test_numbers_next_to_a_boundary(medusa):
    """u on, below and above a boundary of the row: 2^-20 each, sums are exact."""
    V = 1 << 14
    p = np.full((1, 1, V), 2.0 ** -14, np.float32)
    for v in (0, 1, 4095, 4096, 8191, 8192, V - 1):
        for u, want in ((v / V, v), (np.nextafter(np.float32(v / V), np.float32(1)), v), (np.nextafter(np.float32((v + 1) / V), np.float32(0)), v)):
            c = dict(probs=p, cand=np.zeros((1, 1), np.int32), parent=np.array([-1], np.int32), depth=np.zeros(1, np.int32),
                     u=np.full((1, 1), u, np.float32), max_depth=0)
            assert run(medusa, c)["next_tok"][0] == want


def test_many_numbers_on_a_flat_row(medusa):
    """A flat row of 128256 tokens has a boundary next to every number: 64-bit sums find the token."""
    V, B = 128256, 64
    rng = np.random.default_rng(11)
    row = (rng.random(V) / V).astype(np.float32)
    c = dict(probs=np.broadcast_to(row, (B, 1, V)).copy(), cand=np.zeros((B, 1), np.int32), parent=np.array([-1], np.int32),
             depth=np.zeros(1, np.int32), u=rng.random((B, 1)).astype(np.float32), max_depth=0)
    check(c, run(medusa, c))


def test_rows_without_weight_and_values_that_are_none(medusa):
    c = case(5, 6, 9, 300, "dense")
    c["probs"][0, 0] = 0
    c["probs"][1, 0] = np.nan
    c["probs"][2, 0, ::2] = -1
    c["probs"][3, 0, 5:] = np.inf
    c["probs"][4, :, :] *= 0.001
    c["u"][5, 0] = 0.0
    check(c, run(medusa, c))
    for u in (1.0, 7.0, -1.0, np.nan, np.inf):
        c["u"][:] = u
        check(c, run(medusa, c))


def test_trees_that_are_none(medusa):
    c = case(6, 3, 12, 50, "dense")
    c["parent"][:] = [-1, 5, 0, 0, 4, 7, 1, -3, 99, 2, 3, 11]
    c["cand"][0, 2:4] = -1
    c["cand"][1] = c["cand"][1, 1]  # two children with one token: the lower one
    check(c, run(medusa, c))


def test_unaligned_rows_and_given_outputs(medusa):
    c = case(7, 2, 9, 1003, "random")
    M = medusa
    flat = torch.empty(2 * 9 * 1003 + 1, device="cuda")
    probs = flat[1:].view(2, 9, 1003)
    probs.copy_(to_dev(c["probs"]))
    t = [probs, *(to_dev(c[n]) for n in ("cand", "parent", "depth", "u"))]
    out = {k: torch.full(s, -9, dtype=torch.int32, device="cuda") for k, s in
           (("accept_len", (2,)), ("best_node", (2,)), ("next_tok", (2,)), ("path_nodes", (2, c["max_depth"] + 1)))}
    ws = torch.empty(M.verify_draw_workspace(2, 9, 1003), dtype=torch.uint8, device="cuda")
    assert M.verify_accept_tree_draw(*t, c["max_depth"], out=out, ws=ws) is out
    check(c, {k: v.cpu().numpy() for k, v in out.items()})


@pytest.mark.parametrize("B,N,V", [(2, 30, 5000), (2, 60, 128256)])
def test_captured_and_on_another_stream(medusa, B, N, V):
    M = medusa
    c = case(8, B, N, V, "dense", peak=6.0)
    t = [to_dev(c[n]) for n in ("probs", "cand", "parent", "depth", "u")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = M.verify_accept_tree_draw(*t, c["max_depth"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(c, {k: v.cpu().numpy() for k, v in r.items()})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = M.verify_accept_tree_draw(*t, c["max_depth"])
    for seed in (1, 2):
        c["u"] = np.random.default_rng(seed).random(c["u"].shape).astype(np.float32)
        t[4].copy_(to_dev(c["u"]))
        graph.replay()
        torch.cuda.synchronize()
        check(c, {k: v.cpu().numpy() for k, v in r.items()})
