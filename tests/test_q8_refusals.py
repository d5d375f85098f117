"""Arguments that the 8-bit paged cache's entry points refuse: checked on the
host, with nothing enqueued.  No test here launches a kernel."""
import ctypes as C

import pytest
import torch

BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def M():
    from medusa_speculative_decoding_gb300 import build
    build.build()
    import medusa_speculative_decoding_gb300 as M
    return M


X = C.c_void_p(4096)   # an aligned address that no refused call looks at
Y = C.c_void_p(8192)
ODD = C.c_void_p(4100)


def attend(M, q=X, kt=X, vt=X, dtype=BF16, kp=X, vp=X, ks=X, vs=X, table=X, kv_len=X, mask=X, B=1, N=64, Hq=32, Hkv=8,
           D=128, P=64, n_pages=100, W=40, scale=0.1, out=X, ws=None, ws_bytes=0):
    return M.lib().medusa_tree_attention_q8(q, kt, vt, dtype, kp, vp, ks, vs, table, kv_len, mask, B, N, Hq, Hkv, D, P,
                                            n_pages, W, C.c_float(scale), out, ws, ws_bytes, None)


def append(M, kr=X, vr=X, dtype=BF16, kp=X, vp=X, ks=X, vs=X, table=X, kv_len=X, rows=X, last=X, B=1, T=64, R=6, Hkv=8, D=128,
           P=64, n_pages=100, W=40, best=None, hidden=None, h_next=None, H=0, out=Y, appended=None):
    return M.lib().medusa_kv_append_q8(kr, vr, dtype, kp, vp, ks, vs, table, kv_len, rows, last, B, T, R, Hkv, D, P, n_pages, W,
                                       best, hidden, h_next, H, out, appended, None)


def fork(M, kp=X, vp=X, ks=X, vs=X, table=X, kv_len=X, src=None, need=None, held=None, B=4, Hkv=8, D=128, P=64, n_pages=100,
         W=40, table_out=Y, len_out=Y, refs=Y, taken=Y, ws=X, ws_bytes=1 << 20):
    return M.lib().medusa_kv_pages_fork(kp, vp, ks, vs, table, kv_len, src, need, held, B, Hkv, D, P, n_pages, W, table_out,
                                        len_out, refs, taken, ws, ws_bytes, None)


def compact(M, kp=X, vp=X, ks=X, vs=X, table=X, held=None, B=4, Hkv=8, D=128, P=64, n_pages=100, W=40, table_out=Y, new=Y,
            live=Y, ws=X, ws_bytes=1 << 20):
    return M.lib().medusa_kv_pages_compact(kp, vp, ks, vs, table, held, B, Hkv, D, P, n_pages, W, table_out, new, live, ws,
                                           ws_bytes, None)


POOL = [(dict(D=96), -2), (dict(P=48), -2), (dict(P=256), -2), (dict(B=0), -1), (dict(B=1025), -2), (dict(Hkv=0), -1),
        (dict(n_pages=0), -1), (dict(W=0), -1), (dict(n_pages=1 << 24, Hkv=32, Hq=32), -2), (dict(W=1 << 25), -2),
        (dict(kp=None), -1), (dict(vp=ODD), -1), (dict(table=None), -1)]


@pytest.mark.parametrize("call", [attend, append, fork, compact], ids=lambda f: f.__name__)
@pytest.mark.parametrize("args,code", POOL, ids=str)
def test_pool_arguments(M, call, args, code):
    if call is not attend:
        args = {k: v for k, v in args.items() if k != "Hq"}
    assert call(M, **args) == code
    assert M.lib().medusa_last_error()


@pytest.mark.parametrize("args,code", [
    (dict(N=0), -1), (dict(N=513), -2), (dict(Hq=12), -2), (dict(Hq=1024), -2), (dict(dtype=2), -2), (dict(q=None), -1),
    (dict(out=ODD), -1), (dict(kt=ODD), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(ws=None), -3), (dict(ws=X, ws_bytes=1024), -3), (dict(mask=None), -1)], ids=str)
def test_attention_arguments(M, args, code):
    assert attend(M, **args) == code


def test_attention_workspace_must_be_aligned(M):
    assert M.tree_attention_q8_workspace(1, 64, 32, 8, 128) > 0
    assert attend(M, ws=ODD, ws_bytes=1 << 40) == -1
    assert M.lib().medusa_tree_attention_q8_workspace(1, 64, 32, 8, 96, BF16) == 0


@pytest.mark.parametrize("args,code", [
    (dict(T=0), -1), (dict(R=0), -1), (dict(rows=None, R=65), -1), (dict(dtype=7), -2), (dict(kr=None), -1), (dict(vr=ODD), -1),
    (dict(out=None), -1), (dict(out=X), -1), (dict(best=X), -1), (dict(hidden=X, h_next=X), -1),
    (dict(best=X, hidden=X, h_next=X, H=4), -2), (dict(best=X, hidden=ODD, h_next=X, H=64), -1),
    (dict(rows=None, T=1 << 24, R=1 << 24, P=16), -2)], ids=str)
def test_append_arguments(M, args, code):
    assert append(M, **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(table_out=X), -1), (dict(len_out=X), -1), (dict(refs=None), -1), (dict(taken=None), -1), (dict(ws=None), -3),
    (dict(ws_bytes=16), -3), (dict(ws=ODD), -1)], ids=str)
def test_fork_arguments(M, args, code):
    assert fork(M, **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(new=None), -1), (dict(live=None), -1), (dict(ws=None), -3), (dict(ws_bytes=16), -3), (dict(ws=ODD), -1)], ids=str)
def test_compact_arguments(M, args, code):
    assert compact(M, **args) == code


def test_workspace_queries_of_bad_sizes(M):
    assert M.kv_pages_fork_workspace(0, 5) == 0 and M.kv_pages_compact_workspace(0) == 0
    assert M.kv_pages_fork_workspace(4, 100) > 0 and M.kv_pages_compact_workspace(100) > 0


def test_binding_refuses_host_tensors(M):
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    scale = torch.ones(4, 2)
    table, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        M.kv_pages_fork(pages, pages, scale, scale, table, n)
    with pytest.raises(ValueError, match="CUDA"):
        M.kv_pages_compact(pages, pages, scale, scale, table)
    with pytest.raises(ValueError, match="CUDA"):
        M.kv_append_q8(torch.zeros(1, 1, 2, 64), torch.zeros(1, 1, 2, 64), pages, pages, scale, scale, table, n)
    with pytest.raises(ValueError, match="CUDA"):
        M.tree_attention_q8(torch.zeros(1, 1, 2, 64), None, None, pages, pages, scale, scale, table, n, None, 0.1)
