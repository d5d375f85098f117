"""Arguments that the rotating append, the chunk attention, the rotation of rows and the
acceptance by drawn tokens refuse: checked on the host, with nothing enqueued.  No test here
launches a kernel."""
import ctypes as C

import pytest
import torch

from test_q8_refusals import BF16, M, ODD, X, Y  # noqa: F401  (M: fixture)

Z = C.c_void_p(12288)


def attend(M, q=X, dtype=BF16, kp=X, vp=X, ks=X, vs=X, table=X, kv_len=X, last=None, B=1, T=64, Hq=32, Hkv=8, D=128, P=64,  # noqa: F811
           n_pages=100, W=40, scale=0.1, out=Y, ws=X, ws_bytes=1 << 40):
    return M.lib().medusa_chunk_attention_q8(q, dtype, kp, vp, ks, vs, table, kv_len, last, B, T, Hq, Hkv, D, P, n_pages, W,
                                             C.c_float(scale), out, ws, ws_bytes, None)


def append(M, kr=X, vr=X, dtype=BF16, kp=X, vp=X, ks=X, vs=X, table=X, kv_len=X, rows=None, last=None, freq=X, n_freq=64, q=None,  # noqa: F811
           q_out=None, B=1, T=64, R=64, Hq=0, Hkv=8, D=128, P=64, n_pages=100, W=40, best=None, hidden=None, h_next=None, H=0, out=Y,
           appended=None):
    return M.lib().medusa_kv_append_rope_q8(kr, vr, dtype, kp, vp, ks, vs, table, kv_len, rows, last, freq, n_freq, 0, q, q_out, B, T,
                                            R, Hq, Hkv, D, P, n_pages, W, best, hidden, h_next, H, out, appended, None)


def rope(M, q=X, k=Y, dtype=BF16, kv_len=X, depth=None, freq=X, B=1, T=64, Hq=32, Hkv=8, D=128, n_freq=64, q_out=X, k_out=Y):  # noqa: F811
    return M.lib().medusa_rope_rows(q, k, dtype, kv_len, depth, freq, B, T, Hq, Hkv, D, n_freq, 0, q_out, k_out, None)


def draw(M, p=X, cand=X, parent=X, depth=X, u=X, B=1, N=64, V=1000, Dmax=5, a=Y, b=Y, c=Y, d=Y, ws=X, ws_bytes=1 << 20):  # noqa: F811
    return M.lib().medusa_verify_accept_tree_draw(p, cand, parent, depth, u, B, N, V, Dmax, a, b, c, d, ws, ws_bytes, None)


POOL = [(dict(D=96), -2), (dict(P=48), -2), (dict(P=256), -2), (dict(B=0), -1), (dict(B=1025), -2), (dict(Hkv=0), -1),
        (dict(n_pages=0), -1), (dict(W=0), -1), (dict(n_pages=1 << 24, Hkv=32, Hq=32), -2), (dict(W=1 << 25), -2),
        (dict(kp=None), -1), (dict(vp=ODD), -1), (dict(table=None), -1), (dict(kv_len=None), -1), (dict(ks=None), -1), (dict(T=0), -1),
        (dict(dtype=2), -2)]


@pytest.mark.parametrize("call", [attend, append], ids=lambda f: f.__name__)
@pytest.mark.parametrize("args,code", POOL, ids=str)
def test_pool_arguments(M, call, args, code):  # noqa: F811
    if call is append:
        args = {k: v for k, v in args.items() if k != "Hq"}
    assert call(M, **args) == code
    assert M.lib().medusa_last_error()


@pytest.mark.parametrize("args,code", [
    (dict(Hq=12), -2), (dict(Hq=1024), -2), (dict(q=None), -1), (dict(out=ODD), -1), (dict(q=ODD), -1), (dict(out=X), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(scale=2.5e38), -1), (dict(ws=None), -3), (dict(ws_bytes=1024), -3), (dict(ws=ODD), -1), (dict(T=(1 << 20) + 1), -2),
    (dict(B=1024, T=1 << 20, Hkv=32, Hq=32, W=1 << 14), -2)], ids=str)
def test_chunk_attention_arguments(M, args, code):  # noqa: F811
    assert attend(M, **args) == code


def test_workspace_queries(M):  # noqa: F811
    assert M.chunk_attention_q8_workspace(1, 64, 32, 8, 128) > 0 and M.verify_draw_workspace(2, 64, 1000) == 512
    assert M.lib().medusa_chunk_attention_q8_workspace(1, 64, 32, 8, 96, BF16) == 0
    assert M.lib().medusa_chunk_attention_q8_workspace(1, 64, 30, 8, 128, BF16) == 0
    assert M.verify_draw_workspace(0, 64, 1000) == 0


@pytest.mark.parametrize("args,code", [
    (dict(R=0), -1), (dict(R=65), -1), (dict(kr=None), -1), (dict(vr=ODD), -1), (dict(out=None), -1), (dict(out=X), -1),
    (dict(best=X), -1), (dict(hidden=X, h_next=X), -1), (dict(best=X, hidden=X, h_next=X, H=4), -2), (dict(best=X, hidden=ODD, h_next=X, H=64), -1),
    (dict(T=1 << 24, R=1 << 24, P=16), -2), (dict(freq=None), -1), (dict(n_freq=0), -2), (dict(n_freq=12), -2), (dict(n_freq=72), -2),
    (dict(q=X), -1), (dict(Hq=8), -1), (dict(q=X, Hq=8), -1), (dict(q=X, q_out=Z, Hq=8, rows=X), -1), (dict(q=X, q_out=ODD, Hq=8), -1),
    (dict(q=X, q_out=Z, Hq=1025), -2), (dict(q=X, q_out=Z, Hq=8, R=63), -1), (dict(kr=Y, vr=Z, q=X, q_out=Z, Hq=8), -1),
    (dict(last=Y), -1), (dict(appended=X), -1), (dict(appended=Y), -1), (dict(rows=Y), -1)], ids=str)
def test_append_arguments(M, args, code):  # noqa: F811
    assert append(M, **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(B=0), -1), (dict(T=0), -1), (dict(Hq=0), -1), (dict(Hkv=-1), -1), (dict(dtype=3), -2), (dict(D=120), -2), (dict(D=1024), -2),
    (dict(n_freq=4), -2), (dict(n_freq=72), -2), (dict(freq=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(Hkv=0), -1),
    (dict(k_out=None), -1), (dict(kv_len=None), -1), (dict(q=ODD), -1), (dict(k_out=ODD), -1), (dict(k_out=X), -1), (dict(q_out=Y, k_out=Z), -1),
    (dict(Hq=1025), -2), (dict(B=65536), -2)], ids=str)
def test_rope_arguments(M, args, code):  # noqa: F811
    assert rope(M, **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(B=0), -1), (dict(N=0), -1), (dict(V=0), -1), (dict(Dmax=-1), -1), (dict(N=513), -2), (dict(Dmax=512), -2), (dict(V=(1 << 24) + 1), -2),
    (dict(B=65536), -2), (dict(p=None), -1), (dict(u=None), -1), (dict(d=None), -1), (dict(ws=None), -3), (dict(ws_bytes=255), -3),
    (dict(ws=C.c_void_p(4098)), -1)], ids=str)
def test_draw_arguments(M, args, code):  # noqa: F811
    assert draw(M, **args) == code


def test_binding_refuses_host_tensors(M):  # noqa: F811
    pages, scale = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.ones(4, 2)
    table, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x, f = torch.zeros(1, 1, 2, 64), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        M.rope_rows(x, x, n, f)
    with pytest.raises(ValueError, match="CUDA"):
        M.kv_append_rope_q8(x, x, pages, pages, scale, scale, table, n, f)
    with pytest.raises(ValueError, match="CUDA"):
        M.chunk_attention_q8(x, pages, pages, scale, scale, table, n, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        M.verify_accept_tree_draw(torch.zeros(1, 1, 5), n.view(1, 1), n, n, torch.zeros(1, 1), 0)
