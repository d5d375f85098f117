"""Python binding of the C ABI (include/medusa.h) for torch tensors.

Argument marshalling only: checks device, dtype and contiguity, allocates the
outputs and workspaces with torch, and passes raw pointers plus the current CUDA
stream to libmedusa_gb300.so.  Every step of the computation runs in the
library's kernels.  With `stream` given a call works on that stream, and what it
allocates belongs to it; inputs have to be ready there.
"""
from __future__ import annotations

import ctypes as C
import functools
import inspect

import numpy as np
import torch

from ._native import GREEDY, MEDUSA_BF16, MEDUSA_F32, TYPICAL, check, lib

_DT = {torch.float32: MEDUSA_F32, torch.bfloat16: MEDUSA_BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _need(t, name, dtype=None, cuda=True):
    if t is None:
        raise ValueError(f"{name} is required")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _dtype_of(t):
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _tensors(x):
    if torch.is_tensor(x):
        yield x
    elif x is not None:
        for y in x.values() if isinstance(x, dict) else x:
            yield from _tensors(y)


def _in_stream(f):
    """Makes `stream`, where one is given, the current one while f allocates and
    launches.  Memory belongs to the stream that it was allocated on: a workspace of
    another stream would go to that stream's next tensors when f returns, with the
    call's kernels still to come.  Results may be used on either stream; the caller
    orders the two, as for the inputs."""
    at = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        s = args[at] if len(args) > at else kw.get("stream")
        if s is None or s == torch.cuda.current_stream():
            return f(*args, **kw)
        outer = torch.cuda.current_stream(s.device)
        with torch.cuda.stream(s):
            result = f(*args, **kw)
        for t in _tensors(result):
            t.record_stream(outer)
        return result

    return call


# ----------------------------------------------------------------------------
def device_status(stream=None):
    """Synchronises the stream and raises MedusaError (code MEDUSA_ERR_TIMEOUT,
    -5) if a bounded wait of a tensor-core kernel on this device gave up since
    the previous check; returns None otherwise."""
    check(lib().medusa_device_status(_stream(stream)))


def set_wait_limit(cycles):
    """Test hook: limit (SM clock cycles) of the tensor-core kernels' first
    waits on the current device; cycles <= 0 restores the default."""
    check(lib().medusa_set_wait_limit(int(cycles)))


# ----------------------------------------------------------------------------
def heads_topk_workspace(B, K, H, V, topk):
    return int(lib().medusa_heads_topk_workspace(B, K, H, V, topk))


@_in_stream
def heads_topk(h, w1, b1, w2, topk, want_logits=False, out=None, ws=None, stream=None):
    """Medusa heads + per-head top-k.  Returns (topk_idx [B,K,topk] int32,
    topk_val [B,K,topk] float32, logits [B,K,V] float32 or None)."""
    for n, t in (("h", h), ("w1", w1), ("b1", b1), ("w2", w2)):
        _need(t, n, h.dtype)
    B, H = h.shape
    K, V = w2.shape[0], w2.shape[1]
    dev = h.device
    if out is None:
        idx = torch.empty((B, K, topk), dtype=torch.int32, device=dev)
        val = torch.empty((B, K, topk), dtype=torch.float32, device=dev)
        lg = torch.empty((B, K, V), dtype=torch.float32, device=dev) if want_logits else None
    else:
        idx, val, lg = out
    need = heads_topk_workspace(B, K, H, V, topk)
    if ws is None:
        ws = _ws(need, dev)
    check(lib().medusa_heads_topk(_ptr(h), _ptr(w1), _ptr(b1), _ptr(w2), _dtype_of(h), B, K, H, V,
                                  topk, _ptr(idx), _ptr(val), _ptr(lg), _ptr(ws), ws.numel(),
                                  _stream(stream)))
    return idx, val, lg


HEADS_STATIC_SCRATCH_BYTES = 4 << 20


@_in_stream
def heads_topk_static(h, w1, b1, w2, topk, want_logits=False, out=None, stream=None):
    """heads_topk without a workspace, for callers that cannot allocate device
    memory: the library's own 4 MiB device scratch array is used instead.  Calls
    share that array, so calls whose GPU work overlaps race; keep them on one
    stream."""
    for n, t in (("h", h), ("w1", w1), ("b1", b1), ("w2", w2)):
        _need(t, n, h.dtype)
    B, H = h.shape
    K, V = w2.shape[0], w2.shape[1]
    dev = h.device
    if out is None:
        idx = torch.empty((B, K, topk), dtype=torch.int32, device=dev)
        val = torch.empty((B, K, topk), dtype=torch.float32, device=dev)
        lg = torch.empty((B, K, V), dtype=torch.float32, device=dev) if want_logits else None
    else:
        idx, val, lg = out
    check(lib().medusa_heads_topk_static(_ptr(h), _ptr(w1), _ptr(b1), _ptr(w2), _dtype_of(h), B, K, H,
                                         V, topk, _ptr(idx), _ptr(val), _ptr(lg), _stream(stream)))
    return idx, val, lg


# ----------------------------------------------------------------------------
def sparse_tree_paths(n_nodes, max_depth, max_rank, head_p, rank_p):
    out = np.zeros((n_nodes - 1, max_depth), np.int32)
    check(lib().medusa_sparse_tree_paths(n_nodes, max_depth, max_rank, float(head_p), float(rank_p),
                                         out.ctypes.data_as(C.c_void_p)))
    return out


def tree_layout(paths, max_depth, cap_nodes=4096):
    """Host node table of the tree spanned by rank tuples (numpy in and out)."""
    paths = np.ascontiguousarray(paths, dtype=np.int32).reshape(-1, max_depth)
    P = paths.shape[0]
    W_cap = (cap_nodes + 63) // 64
    parent = np.zeros(cap_nodes, np.int32)
    depth = np.zeros(cap_nodes, np.int32)
    rank = np.zeros(cap_nodes, np.int32)
    mask = np.zeros(cap_nodes * W_cap, np.uint64)
    retrieve = np.zeros((cap_nodes, max_depth + 1), np.int32)
    N, W, NP = C.c_int(), C.c_int(), C.c_int()
    p = lambda a: a.ctypes.data_as(C.c_void_p)
    check(lib().medusa_tree_layout(p(paths), P, max_depth, cap_nodes, cap_nodes, p(parent),
                                   p(depth), p(rank), p(mask), p(retrieve), C.byref(N), C.byref(W),
                                   C.byref(NP)))
    n, w, npth = N.value, W.value, NP.value
    return dict(N=n, W=w, n_paths=npth, parent=parent[:n].copy(), depth=depth[:n].copy(),
                rank=rank[:n].copy(), mask=mask[: n * w].reshape(n, w).copy(),
                retrieve=retrieve[:npth].copy(), max_depth=max_depth)


@_in_stream
def build_tree(topk_idx, root_tok, depth, rank, out=None, stream=None):
    _need(topk_idx, "topk_idx", torch.int32)
    _need(root_tok, "root_tok", torch.int32)
    _need(depth, "depth", torch.int32)
    _need(rank, "rank", torch.int32)
    B, K, k = topk_idx.shape
    N = depth.shape[0]
    cand = out if out is not None else torch.empty((B, N), dtype=torch.int32, device=topk_idx.device)
    check(lib().medusa_build_tree(_ptr(topk_idx), _ptr(root_tok), _ptr(depth), _ptr(rank), B, K, k,
                                  N, _ptr(cand), _stream(stream)))
    return cand


# ----------------------------------------------------------------------------
def tree_attention_workspace(B, N, Hq, Hkv, D, Lmax):
    return int(lib().medusa_tree_attention_workspace(B, N, Hq, Hkv, D, Lmax))


@_in_stream
def tree_attention(q, k_cache, v_cache, kv_len, mask, scale, out=None, ws=None, stream=None):
    """Tree attention; `scale` multiplies q.k inside the softmax (the model's
    choice, usually 1/sqrt(head dim)); it is passed to the library as given."""
    _need(q, "q")
    _need(k_cache, "k_cache", q.dtype)
    _need(v_cache, "v_cache", q.dtype)
    _need(kv_len, "kv_len", torch.int32)
    _need(mask, "mask", torch.int64)
    B, N, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    o = out if out is not None else torch.empty((B, N, Hq, D), dtype=torch.float32, device=q.device)
    need = tree_attention_workspace(B, N, Hq, Hkv, D, Lmax)
    if ws is None:
        ws = _ws(need, q.device)
    check(lib().medusa_tree_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len),
                                      _ptr(mask), _dtype_of(q), B, N, Hq, Hkv, D, Lmax,
                                      float(scale), _ptr(o), _ptr(ws), ws.numel(), _stream(stream)))
    return o


# ----------------------------------------------------------------------------
def verify_accept_workspace(B, N, V):
    return int(lib().medusa_verify_accept_workspace(B, N, V))


@_in_stream
def verify_accept_tree(logits, cand, parent, depth, max_depth, mode="greedy", temperature=1.0,
                       eps=0.09, delta=0.3, out=None, ws=None, stream=None):
    _need(logits, "logits", torch.float32)
    _need(cand, "cand", torch.int32)
    _need(parent, "parent", torch.int32)
    _need(depth, "depth", torch.int32)
    B, N, V = logits.shape
    dev = logits.device
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   best_node=torch.empty(B, dtype=torch.int32, device=dev),
                   path_nodes=torch.empty((B, max_depth + 1), dtype=torch.int32, device=dev),
                   next_tok=torch.empty(B, dtype=torch.int32, device=dev))
    if ws is None:
        ws = _ws(verify_accept_workspace(B, N, V), dev)
    m = {"greedy": GREEDY, "typical": TYPICAL}[mode]
    check(lib().medusa_verify_accept_tree(_ptr(logits), _ptr(cand), _ptr(parent), _ptr(depth), B,
                                          N, V, max_depth, m, float(temperature), float(eps),
                                          float(delta), _ptr(out["accept_len"]),
                                          _ptr(out["best_node"]), _ptr(out["path_nodes"]),
                                          _ptr(out["next_tok"]), _ptr(ws), ws.numel(),
                                          _stream(stream)))
    return out


def verify_sample_workspace(B, N, V):
    return int(lib().medusa_verify_sample_workspace(B, N, V))


@_in_stream
def verify_accept_tree_sample(logits, cand, parent, depth, max_depth, seed, round_, temperature=1.0,
                              eps=0.09, delta=0.3, out=None, ws=None, stream=None):
    """Typical acceptance; the next token drawn from the best node's softmax."""
    _need(logits, "logits", torch.float32)
    _need(cand, "cand", torch.int32)
    _need(parent, "parent", torch.int32)
    _need(depth, "depth", torch.int32)
    B, N, V = logits.shape
    dev = logits.device
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   best_node=torch.empty(B, dtype=torch.int32, device=dev),
                   path_nodes=torch.empty((B, max_depth + 1), dtype=torch.int32, device=dev),
                   next_tok=torch.empty(B, dtype=torch.int32, device=dev))
    if ws is None:
        ws = _ws(verify_sample_workspace(B, N, V), dev)
    check(lib().medusa_verify_accept_tree_sample(_ptr(logits), _ptr(cand), _ptr(parent), _ptr(depth), B, N,
                                                 V, max_depth, float(temperature), float(eps), float(delta),
                                                 C.c_uint64(seed), C.c_uint64(round_),
                                                 _ptr(out["accept_len"]), _ptr(out["best_node"]),
                                                 _ptr(out["path_nodes"]), _ptr(out["next_tok"]), _ptr(ws),
                                                 ws.numel(), _stream(stream)))
    return out


def verify_project_workspace(B, N, H, V):
    return int(lib().medusa_verify_project_workspace(B, N, H, V))


@_in_stream
def verify_project_tree(hidden_tree, lm_head, cand, parent, depth, max_depth, mode="greedy",
                        temperature=1.0, eps=0.09, delta=0.3, out=None, ws=None, stream=None):
    """verify_accept_tree with the verifier logits defined as lm_head . hidden_tree,
    computed and reduced on the GPU without materialising them."""
    _need(hidden_tree, "hidden_tree", torch.bfloat16)
    _need(lm_head, "lm_head", torch.bfloat16)
    _need(cand, "cand", torch.int32)
    _need(parent, "parent", torch.int32)
    _need(depth, "depth", torch.int32)
    B, N, H = hidden_tree.shape
    V = lm_head.shape[0]
    dev = hidden_tree.device
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   best_node=torch.empty(B, dtype=torch.int32, device=dev),
                   path_nodes=torch.empty((B, max_depth + 1), dtype=torch.int32, device=dev),
                   next_tok=torch.empty(B, dtype=torch.int32, device=dev))
    if ws is None:
        ws = _ws(verify_project_workspace(B, N, H, V), dev)
    m = {"greedy": GREEDY, "typical": TYPICAL}[mode]
    check(lib().medusa_verify_project_tree(_ptr(hidden_tree), _ptr(lm_head), _dtype_of(hidden_tree),
                                           _ptr(cand), _ptr(parent), _ptr(depth), B, N, H, V,
                                           max_depth, m, float(temperature), float(eps),
                                           float(delta), _ptr(out["accept_len"]),
                                           _ptr(out["best_node"]), _ptr(out["path_nodes"]),
                                           _ptr(out["next_tok"]), _ptr(ws), ws.numel(),
                                           _stream(stream)))
    return out


def verify_chain_workspace(B, gamma, V):
    return int(lib().medusa_verify_chain_workspace(B, gamma, V))


@_in_stream
def verify_accept_chain(p, q, draft, seed, round_, out=None, ws=None, stream=None):
    _need(p, "p", torch.float32)
    B, g1, V = p.shape
    gamma = g1 - 1
    if gamma > 0:
        _need(q, "q", torch.float32)
        _need(draft, "draft", torch.int32)
    dev = p.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev),
               torch.empty((B, gamma + 1), dtype=torch.int32, device=dev))
    if ws is None:
        ws = _ws(verify_chain_workspace(B, gamma, V), dev)
    n_acc, out_tok = out
    check(lib().medusa_verify_accept_chain(_ptr(p), _ptr(q) if gamma > 0 else None,
                                           _ptr(draft) if gamma > 0 else None, B, gamma, V,
                                           C.c_uint64(seed), C.c_uint64(round_), _ptr(n_acc),
                                           _ptr(out_tok), _ptr(ws), ws.numel(), _stream(stream)))
    return n_acc, out_tok


def verify_draw_workspace(B, N, V):
    return int(lib().medusa_verify_draw_workspace(B, N, V))


@_in_stream
def verify_accept_tree_draw(probs, cand, parent, depth, u, max_depth, out=None, ws=None, stream=None):
    """Acceptance by drawn tokens: at each node of the path the token that u[b, depth]
    in [0, 1) picks from row probs[b, node] (the smallest v with p_0 + .. + p_v above u
    times the row's sum); the child that holds it is accepted, else it is next_tok.
    probs [B,N,V] float32, u [B, max_depth + 1] float32.  A row need not sum to 1, but its
    entries count as at most 1 (below 0 and NaN: 0): weights above 1 are not told apart."""
    if probs is None or probs.dim() != 3:
        raise ValueError("probs must be [B, N, V]")
    _need(probs, "probs", torch.float32)
    B, N, V = probs.shape
    dev = probs.get_device()
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return verify_accept_tree_draw(probs, cand, parent, depth, u, max_depth, out, ws, stream)
    _need_shape(cand, "cand", (B, N), _I32, dev)
    _need_shape(parent, "parent", (N,), _I32, dev)
    _need_shape(depth, "depth", (N,), _I32, dev)
    _need_shape(u, "u", (B, max_depth + 1), _F32, dev)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=_I32, device=probs.device),
                   best_node=torch.empty(B, dtype=_I32, device=probs.device),
                   path_nodes=torch.empty((B, max_depth + 1), dtype=_I32, device=probs.device),
                   next_tok=torch.empty(B, dtype=_I32, device=probs.device))
    else:
        for n, shape in (("accept_len", (B,)), ("best_node", (B,)), ("path_nodes", (B, max_depth + 1)), ("next_tok", (B,))):
            _need_shape(out[n], f"out {n}", shape, _I32, dev)
    if ws is None:
        ws = torch.empty(_draw_bytes(B, N, V), dtype=torch.uint8, device=probs.device)
    else:
        _need_ws(ws, dev)
    check(lib().medusa_verify_accept_tree_draw(probs.data_ptr(), cand.data_ptr(), parent.data_ptr(), depth.data_ptr(),
                                               u.data_ptr(), B, N, V, max_depth, out["accept_len"].data_ptr(),
                                               out["best_node"].data_ptr(), out["path_nodes"].data_ptr(),
                                               out["next_tok"].data_ptr(), ws.data_ptr(), ws.numel(),
                                               _raw_stream(stream, dev)))
    return out


# ----------------------------------------------------------------------------
@_in_stream
def kv_compact(k_cache, v_cache, kv_len, path_nodes, accept_len, best_node, N, max_depth,
               hidden_tree=None, h_next=None, src_idx=None, stream=None):
    _need(k_cache, "k_cache")
    _need(v_cache, "v_cache", k_cache.dtype)
    _need(kv_len, "kv_len", torch.int32)
    for n, t in (("path_nodes", path_nodes), ("accept_len", accept_len), ("best_node", best_node)):
        _need(t, n, torch.int32)
    B, Hkv, Lmax, D = k_cache.shape
    H = 0
    if hidden_tree is not None:
        _need(hidden_tree, "hidden_tree", k_cache.dtype)
        H = hidden_tree.shape[-1]
        if h_next is None:
            h_next = torch.empty((B, H), dtype=k_cache.dtype, device=k_cache.device)
    if src_idx is None:
        src_idx = torch.empty((B, max_depth + 1), dtype=torch.int32, device=k_cache.device)
    check(lib().medusa_kv_compact(_ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(path_nodes),
                                  _ptr(accept_len), _ptr(best_node), _ptr(hidden_tree),
                                  _ptr(h_next), _dtype_of(k_cache), B, Hkv, D, Lmax, N, H,
                                  max_depth, _ptr(src_idx), _stream(stream)))
    return h_next, src_idx


# ----------------------------------------------------------------------------
# The 8-bit paged KV cache.  Pools: k_pages, v_pages [n_pages, Hkv, P, D]
# (torch.uint8 or torch.float8_e4m3fn) and k_scale, v_scale [n_pages, Hkv]
# float32; page_table [B, M] and kv_len [B] int32.  These calls take microseconds
# on the device, so their checks are kept to one pass over each tensor.
_I32, _F32 = torch.int32, torch.float32
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _need_shape(t, name, shape, dtype, dev):
    """t, a contiguous tensor of that shape and type on CUDA device number dev."""
    if t is not None and t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    _need(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


_NO_LENGTHS = object()  # the call takes none


def _need_pool(k_pages, v_pages, k_scale, v_scale, page_table, kv_len=_NO_LENGTHS):
    _need(k_pages, "k_pages")
    if k_pages.dtype not in _CODES or k_pages.dim() != 4:
        raise ValueError("k_pages must be [n_pages, Hkv, P, D] e4m3 codes (uint8 or float8_e4m3fn)")
    shape, dev = k_pages.shape, k_pages.get_device()
    _need_shape(v_pages, "v_pages", shape, k_pages.dtype, dev)
    _need_shape(k_scale, "k_scale", shape[:2], _F32, dev)
    _need_shape(v_scale, "v_scale", shape[:2], _F32, dev)
    if page_table is None or page_table.dim() != 2:
        raise ValueError("page_table must be [B, M]")
    _need_shape(page_table, "page_table", page_table.shape, _I32, dev)
    if kv_len is not _NO_LENGTHS:
        _need_shape(kv_len, "kv_len", page_table.shape[:1], _I32, dev)
    return (*page_table.shape, *shape, dev)


def _need_ws(ws, dev):
    if ws.get_device() != dev or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{dev}")


def _elsewhere(dev, stream):
    """Whether CUDA device number dev is not the current one (the library works on
    the current device)."""
    if dev == torch.cuda.current_device():
        return False
    if stream is not None:
        raise ValueError(f"stream must be on cuda:{dev}")
    return True


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


@functools.lru_cache(maxsize=256)
def _attention_q8_bytes(dev, B, N, Hq, Hkv, D, dtype):
    return max(16, lib().medusa_tree_attention_q8_workspace(B, N, Hq, Hkv, D, dtype))


@functools.lru_cache(maxsize=256)
def _chunk_q8_bytes(dev, B, T, Hq, Hkv, D, dtype):
    return max(16, lib().medusa_chunk_attention_q8_workspace(B, T, Hq, Hkv, D, dtype))


@functools.lru_cache(maxsize=256)
def _draw_bytes(B, N, V):
    return max(16, verify_draw_workspace(B, N, V))


@functools.lru_cache(maxsize=256)
def _fork_bytes(B, n_pages):
    return max(16, kv_pages_fork_workspace(B, n_pages))


@functools.lru_cache(maxsize=256)
def _compact_bytes(n_pages):
    return max(16, kv_pages_compact_workspace(n_pages))


def tree_attention_q8_workspace(B, N, Hq, Hkv, D, dtype=torch.bfloat16):
    return int(lib().medusa_tree_attention_q8_workspace(B, N, Hq, Hkv, D, _DT[dtype]))


@_in_stream
def tree_attention_q8(q, k_tree, v_tree, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, mask, scale,
                      out=None, ws=None, stream=None):
    """Tree attention over the 8-bit paged cache: q [B,N,Hq,D] against the pages'
    prefix and the tree rows k_tree, v_tree [B,N,Hkv,D] under mask [N, ceil(N/64)].
    Returns out [B,N,Hq,D] in q's type.  N = 1 with mask [[1]] is plain decoding."""
    B, M, n_pages, Hkv, P, D, dev = _need_pool(k_pages, v_pages, k_scale, v_scale, page_table, kv_len)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return tree_attention_q8(q, k_tree, v_tree, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, mask,
                                     scale, out, ws, stream)
    if q is None or q.dim() != 4:
        raise ValueError(f"q must be [{B}, N, Hq, {D}]")
    N, Hq, dtype = q.shape[1], q.shape[2], q.dtype
    code = _dtype_of(q)
    _need_shape(q, "q", (B, N, Hq, D), dtype, dev)
    _need_shape(k_tree, "k_tree", (B, N, Hkv, D), dtype, dev)
    _need_shape(v_tree, "v_tree", (B, N, Hkv, D), dtype, dev)
    _need_shape(mask, "mask", (N, (N + 63) // 64), torch.int64, dev)
    o = torch.empty_like(q) if out is None else _need_shape(out, "out", q.shape, dtype, dev)
    if ws is None:
        ws = torch.empty(_attention_q8_bytes(dev, B, N, Hq, Hkv, D, code), dtype=torch.uint8, device=q.device)
    else:
        _need_ws(ws, dev)
    check(lib().medusa_tree_attention_q8(q.data_ptr(), k_tree.data_ptr(), v_tree.data_ptr(), code, k_pages.data_ptr(),
                                         v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                         page_table.data_ptr(), kv_len.data_ptr(), mask.data_ptr(), B, N, Hq, Hkv, D, P,
                                         n_pages, M, scale, o.data_ptr(), ws.data_ptr(), ws.numel(),
                                         _raw_stream(stream, dev)))
    return o


@_in_stream
def kv_append_q8(k_rows, v_rows, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, rows=None, last=None,
                 best_node=None, hidden_rows=None, out=None, stream=None):
    """Quantises rows 0..last[b] of `rows` (tree nodes; None: rows in order) of
    k_rows, v_rows [B,T,Hkv,D] into the pages behind kv_len.  `last` None takes
    all.  Returns dict(kv_len, appended, h_next); the pools change in place."""
    B, M, n_pages, Hkv, P, D, dev = _need_pool(k_pages, v_pages, k_scale, v_scale, page_table, kv_len)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return kv_append_q8(k_rows, v_rows, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, rows, last,
                                best_node, hidden_rows, out, stream)
    if k_rows is None or k_rows.dim() != 4:
        raise ValueError(f"k_rows must be [{B}, T, {Hkv}, {D}]")
    T, dtype = k_rows.shape[1], k_rows.dtype
    code = _dtype_of(k_rows)
    _need_shape(k_rows, "k_rows", (B, T, Hkv, D), dtype, dev)
    _need_shape(v_rows, "v_rows", (B, T, Hkv, D), dtype, dev)
    R = T
    if rows is not None:
        if rows.dim() != 2:
            raise ValueError("rows must be [B, R]")
        R = rows.shape[1]
        _need_shape(rows, "rows", (B, R), _I32, dev)
    if last is not None:
        _need_shape(last, "last", (B,), _I32, dev)
    if (hidden_rows is None) != (best_node is None):
        raise ValueError("best_node and hidden_rows go together")
    H = 0
    if hidden_rows is not None:
        H = hidden_rows.shape[-1]
        _need_shape(hidden_rows, "hidden_rows", (B, T, H), dtype, dev)
        _need_shape(best_node, "best_node", (B,), _I32, dev)
    if out is None:
        out = dict(kv_len=torch.empty_like(kv_len), appended=torch.empty_like(kv_len),
                   h_next=torch.empty((B, H), dtype=dtype, device=kv_len.device) if H else None)
    else:
        _need_shape(out["kv_len"], "out kv_len", (B,), _I32, dev)
        if out.get("appended") is not None:
            _need_shape(out["appended"], "out appended", (B,), _I32, dev)
        if H:
            _need_shape(out["h_next"], "out h_next", (B, H), dtype, dev)
    check(lib().medusa_kv_append_q8(k_rows.data_ptr(), v_rows.data_ptr(), code, k_pages.data_ptr(), v_pages.data_ptr(),
                                    k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(),
                                    _ptr(rows), _ptr(last), B, T, R, Hkv, D, P, n_pages, M, _ptr(best_node),
                                    _ptr(hidden_rows), out["h_next"].data_ptr() if H else None, H,
                                    out["kv_len"].data_ptr(), _ptr(out.get("appended")), _raw_stream(stream, dev)))
    return out


def _need_freqs(inv_freq, D, dev):
    if inv_freq is None or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [n_freq]")
    _need_shape(inv_freq, "inv_freq", inv_freq.shape, _F32, dev)
    return inv_freq.shape[0]


@_in_stream
def rope_rows(q, k, kv_len, inv_freq, depth=None, interleaved=False, out=None, stream=None):
    """Rotary positions: row i of q [B,T,Hq,D] and k [B,T,Hkv,D] (k may be None) turns by
    the angles (kv_len[b] + depth[i]) * inv_freq (i where depth is None), in pairs
    (j, n_freq + j), or (2j, 2j + 1) where interleaved.  Returns (q, k) rotated; `out`
    may be (q, k) itself."""
    if q is None or q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    _need(q, "q")
    B, T, Hq, D = q.shape
    dev, code = q.get_device(), _dtype_of(q)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return rope_rows(q, k, kv_len, inv_freq, depth, interleaved, out, stream)
    Hkv = 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError(f"k must be [{B}, {T}, Hkv, {D}]")
        Hkv = k.shape[2]
        _need_shape(k, "k", (B, T, Hkv, D), q.dtype, dev)
    _need_shape(kv_len, "kv_len", (B,), _I32, dev)
    n_freq = _need_freqs(inv_freq, D, dev)
    if depth is not None:
        _need_shape(depth, "depth", (T,), _I32, dev)
    if out is None:
        out = torch.empty_like(q), torch.empty_like(k) if Hkv else None
    else:
        _need_shape(out[0], "out q", q.shape, q.dtype, dev)
        if Hkv:
            _need_shape(out[1], "out k", k.shape, q.dtype, dev)
    check(lib().medusa_rope_rows(q.data_ptr(), _ptr(k), code, kv_len.data_ptr(), _ptr(depth), inv_freq.data_ptr(), B, T, Hq,
                                 Hkv, D, n_freq, bool(interleaved), out[0].data_ptr(), out[1].data_ptr() if Hkv else None,
                                 _raw_stream(stream, dev)))
    return out


@_in_stream
def kv_append_rope_q8(k_rows, v_rows, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, inv_freq, rows=None, last=None,
                      q=None, interleaved=False, best_node=None, hidden_rows=None, out=None, stream=None):
    """kv_append_q8 of K rows that are not rotated yet: row i turns by the position of its
    slot, kv_len[b] + i, on its way into the pages, and so do the queries q [B,T,Hq,D] of
    the same rows, where given (rows then has to be None).  Returns dict(kv_len, appended,
    h_next, q); rows of q behind last[b] are zero; the pools change in place.  A sequence
    that is refused (appended -2) keeps its kv_len and its queries are rotated all the same:
    chunk_attention_q8(.., last=appended - 1) answers such rows with zeros."""
    B, M, n_pages, Hkv, P, D, dev = _need_pool(k_pages, v_pages, k_scale, v_scale, page_table, kv_len)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return kv_append_rope_q8(k_rows, v_rows, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, inv_freq, rows,
                                     last, q, interleaved, best_node, hidden_rows, out, stream)
    if k_rows is None or k_rows.dim() != 4:
        raise ValueError(f"k_rows must be [{B}, T, {Hkv}, {D}]")
    T, dtype = k_rows.shape[1], k_rows.dtype
    code = _dtype_of(k_rows)
    _need_shape(k_rows, "k_rows", (B, T, Hkv, D), dtype, dev)
    _need_shape(v_rows, "v_rows", (B, T, Hkv, D), dtype, dev)
    n_freq = _need_freqs(inv_freq, D, dev)
    R = T
    if rows is not None:
        if rows.dim() != 2:
            raise ValueError("rows must be [B, R]")
        R = rows.shape[1]
        _need_shape(rows, "rows", (B, R), _I32, dev)
    if last is not None:
        _need_shape(last, "last", (B,), _I32, dev)
    Hq = 0
    if q is not None:
        if q.dim() != 4:
            raise ValueError(f"q must be [{B}, {T}, Hq, {D}]")
        Hq = q.shape[2]
        _need_shape(q, "q", (B, T, Hq, D), dtype, dev)
    if (hidden_rows is None) != (best_node is None):
        raise ValueError("best_node and hidden_rows go together")
    H = 0
    if hidden_rows is not None:
        H = hidden_rows.shape[-1]
        _need_shape(hidden_rows, "hidden_rows", (B, T, H), dtype, dev)
        _need_shape(best_node, "best_node", (B,), _I32, dev)
    if out is None:
        out = dict(kv_len=torch.empty_like(kv_len), appended=torch.empty_like(kv_len),
                   h_next=torch.empty((B, H), dtype=dtype, device=kv_len.device) if H else None,
                   q=torch.empty_like(q) if Hq else None)
    else:
        _need_shape(out["kv_len"], "out kv_len", (B,), _I32, dev)
        if out.get("appended") is not None:
            _need_shape(out["appended"], "out appended", (B,), _I32, dev)
        if H:
            _need_shape(out["h_next"], "out h_next", (B, H), dtype, dev)
        if Hq:
            _need_shape(out["q"], "out q", q.shape, dtype, dev)
    check(lib().medusa_kv_append_rope_q8(k_rows.data_ptr(), v_rows.data_ptr(), code, k_pages.data_ptr(), v_pages.data_ptr(),
                                         k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(),
                                         _ptr(rows), _ptr(last), inv_freq.data_ptr(), n_freq, bool(interleaved), _ptr(q),
                                         out["q"].data_ptr() if Hq else None, B, T, R, Hq, Hkv, D, P, n_pages, M,
                                         _ptr(best_node), _ptr(hidden_rows), out["h_next"].data_ptr() if H else None, H,
                                         out["kv_len"].data_ptr(), _ptr(out.get("appended")), _raw_stream(stream, dev)))
    return out


def chunk_attention_q8_workspace(B, T, Hq, Hkv, D, dtype=torch.bfloat16):
    return int(lib().medusa_chunk_attention_q8_workspace(B, T, Hq, Hkv, D, _DT[dtype]))


@_in_stream
def chunk_attention_q8(q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, scale, last=None, out=None, ws=None,
                       stream=None):
    """Attention of new tokens over the 8-bit paged cache that holds their keys already: row
    i of the last[b] + 1 rows of q [B,T,Hq,D] (all T where last is None) is that of slot
    kv_len[b] - last[b] - 1 + i and sees the slots up to it.  Returns out [B,T,Hq,D] in q's
    type; rows behind last[b] are zero.  T = 1 is plain decoding.  Behind an append that may
    have refused a sequence, last is its appended - 1."""
    B, M, n_pages, Hkv, P, D, dev = _need_pool(k_pages, v_pages, k_scale, v_scale, page_table, kv_len)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return chunk_attention_q8(q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, scale, last, out, ws, stream)
    if q is None or q.dim() != 4:
        raise ValueError(f"q must be [{B}, T, Hq, {D}]")
    T, Hq, dtype = q.shape[1], q.shape[2], q.dtype
    code = _dtype_of(q)
    _need_shape(q, "q", (B, T, Hq, D), dtype, dev)
    if last is not None:
        _need_shape(last, "last", (B,), _I32, dev)
    o = torch.empty_like(q) if out is None else _need_shape(out, "out", q.shape, dtype, dev)
    if ws is None:
        ws = torch.empty(_chunk_q8_bytes(dev, B, T, Hq, Hkv, D, code), dtype=torch.uint8, device=q.device)
    else:
        _need_ws(ws, dev)
    check(lib().medusa_chunk_attention_q8(q.data_ptr(), code, k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                                          v_scale.data_ptr(), page_table.data_ptr(), kv_len.data_ptr(), _ptr(last), B, T, Hq,
                                          Hkv, D, P, n_pages, M, scale, o.data_ptr(), ws.data_ptr(), ws.numel(),
                                          _raw_stream(stream, dev)))
    return o


def kv_pages_fork_workspace(B, n_pages):
    return int(lib().medusa_kv_pages_fork_workspace(B, n_pages))


@_in_stream
def kv_pages_fork(k_pages, v_pages, k_scale, v_scale, page_table, kv_len, src=None, need=None, held=None,
                  out=None, ws=None, stream=None):
    """Forks, frees and reserves: row b goes on from row src[b] (-1: freed; None:
    every row from itself) with room for need[b] more tokens.  Returns
    dict(page_table, kv_len, refs, taken); open pages are copied in the pools."""
    B, M, n_pages, Hkv, P, D, dev = _need_pool(k_pages, v_pages, k_scale, v_scale, page_table, kv_len)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return kv_pages_fork(k_pages, v_pages, k_scale, v_scale, page_table, kv_len, src, need, held, out, ws, stream)
    if src is not None:
        _need_shape(src, "src", (B,), _I32, dev)
    if need is not None:
        _need_shape(need, "need", (B,), _I32, dev)
    if held is not None:
        _need_shape(held, "held", (n_pages,), _I32, dev)
    if out is None:
        out = dict(page_table=torch.empty_like(page_table), kv_len=torch.empty_like(kv_len),
                   refs=torch.empty(n_pages, dtype=_I32, device=kv_len.device), taken=torch.empty_like(kv_len))
    else:
        for n, shape in (("page_table", (B, M)), ("kv_len", (B,)), ("refs", (n_pages,)), ("taken", (B,))):
            _need_shape(out[n], f"out {n}", shape, _I32, dev)
    if ws is None:
        ws = torch.empty(_fork_bytes(B, n_pages), dtype=torch.uint8, device=kv_len.device)
    else:
        _need_ws(ws, dev)
    check(lib().medusa_kv_pages_fork(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                     page_table.data_ptr(), kv_len.data_ptr(), _ptr(src), _ptr(need), _ptr(held), B,
                                     Hkv, D, P, n_pages, M, out["page_table"].data_ptr(), out["kv_len"].data_ptr(),
                                     out["refs"].data_ptr(), out["taken"].data_ptr(), ws.data_ptr(), ws.numel(),
                                     _raw_stream(stream, dev)))
    return out


def kv_pages_compact_workspace(n_pages):
    return int(lib().medusa_kv_pages_compact_workspace(n_pages))


@_in_stream
def kv_pages_compact(k_pages, v_pages, k_scale, v_scale, page_table, held=None, out=None, ws=None, stream=None):
    """Moves the pages in use into [0, live).  Returns dict(page_table, new_page,
    live); the pools change in place."""
    B, M, n_pages, Hkv, P, D, dev = _need_pool(k_pages, v_pages, k_scale, v_scale, page_table)
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev):
            return kv_pages_compact(k_pages, v_pages, k_scale, v_scale, page_table, held, out, ws, stream)
    if held is not None:
        _need_shape(held, "held", (n_pages,), _I32, dev)
    if out is None:
        out = dict(page_table=torch.empty_like(page_table),
                   new_page=torch.empty(n_pages, dtype=_I32, device=page_table.device),
                   live=torch.empty(1, dtype=_I32, device=page_table.device))
    else:
        for n, shape in (("page_table", (B, M)), ("new_page", (n_pages,)), ("live", (1,))):
            _need_shape(out[n], f"out {n}", shape, _I32, dev)
    if ws is None:
        ws = torch.empty(_compact_bytes(n_pages), dtype=torch.uint8, device=page_table.device)
    else:
        _need_ws(ws, dev)
    check(lib().medusa_kv_pages_compact(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                        page_table.data_ptr(), _ptr(held), B, Hkv, D, P, n_pages, M,
                                        out["page_table"].data_ptr(), out["new_page"].data_ptr(),
                                        out["live"].data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)))
    return out
