"""Measured cases of the operators that fill the 8-bit paged KV cache from a model's unrotated rows and answer from it:
the rotary positions of a tree's queries and keys, the append that rotates new keys on the way into the pages, the
attention of a chunk of new tokens over the pages, and the acceptance of a tree by tokens drawn from the target's
probabilities.

The pool holds e4m3 codes [n_pages, Hkv, P, D] for K and V with one float32 scale per page and KV head; page_table
[B, M] (-1: no page) and kv_len [B] say what each sequence holds.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
K_MAX = 316.0  # of a row before its rotation, which makes a value at most sqrt(2) larger


# ---------------------------------------------------------------------------------------------------------------------
# cases


def _rotate(name, B, N, Hq, Hkv, D, n_freq, hi, dtype, tree, interleaved=False):
    return dict(name=name, op="rotate", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, n_freq=n_freq, hi=hi, dtype=dtype, tree=tree,
                interleaved=interleaved)


def _append(name, B, T, Hq, Hkv, D, P, n_freq, lo, hi, dtype, interleaved=False):
    return dict(name=name, op="append", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, P=P, n_freq=n_freq, lo=lo, hi=hi, dtype=dtype,
                interleaved=interleaved)


def _attend(name, B, T, least, Hq, Hkv, D, P, lo, hi, dtype):
    return dict(name=name, op="attend", B=B, T=T, least=least, Hq=Hq, Hkv=Hkv, D=D, P=P, lo=lo, hi=hi, dtype=dtype)


def _verify(name, B, N, V, tree):
    return dict(name=name, op="verify", B=B, N=N, V=V, tree=tree)


def listed():
    return [
        # the sparse 64-node tree of one sequence: what a call costs
        _rotate("rotate 64 nodes b1", 1, 64, 32, 32, 128, 64, 4096, "bf16", "random"),
        # the dense 341-node tree of 16 sequences far into long texts, float32, neighbouring pairs, half of a head rotated
        _rotate("rotate 341 nodes b16 f32", 16, 341, 40, 8, 128, 32, 1000000, "f32", "dense", True),
        # one decoded token of 16 sequences, shared KV heads, small pages
        _append("append 1 token b16 gqa", 16, 1, 32, 8, 128, 32, 64, 777, 16384, "bf16"),
        # four ragged prompts written at once
        _append("append prompts b4", 4, 4096, 32, 32, 128, 64, 64, 0, 200, "bf16"),
        # short float32 prompts of eight sequences, neighbouring pairs
        _append("append prompts b8 f32", 8, 300, 8, 8, 64, 16, 32, 0, 1500, "f32", True),
        # the tiny float32 model: nine rows on a short prefix
        _attend("attend 9 rows f32", 1, 9, 9, 4, 4, 64, 16, 128, 128, "f32"),
        # plain decoding, one token a sequence, shared KV heads, long ragged caches in small pages
        _attend("attend 1 token b16 gqa", 16, 1, 1, 32, 8, 128, 32, 777, 16384, "bf16"),
        # a later chunk of a long prompt: 512 rows on 8192 tokens
        _attend("attend 512 rows b1 kv8192", 1, 512, 512, 32, 8, 128, 64, 8192, 8192, "bf16"),
        # ragged chunks of a batch of eight of the 13B shape
        _attend("attend chunks b8 ragged", 8, 700, 1, 40, 40, 128, 16, 1024, 4096, "bf16"),
        # four whole prompts of up to 4096 tokens: the most arithmetic
        _attend("attend prompts b4", 4, 4096, 2048, 32, 32, 128, 64, 0, 200, "bf16"),
        # the sparse 64-node tree of one sequence, the smaller vocabulary
        _verify("verify 64 nodes b1", 1, 64, 32000, "random"),
        # a batch of 32 with the larger vocabulary
        _verify("verify 64 nodes b32", 32, 64, 128256, "narrow"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "attend", "verify"])
    D = rng.choice([64, 128, 128])
    P = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
    G = rng.choice([g for g in (1, 1, 2, 3, 4, 5, 7, 8) if g * Hkv <= 64])
    n_freq = rng.choice([D // 2, D // 2, D // 4])
    interleaved = rng.random() < 0.3
    if op == "rotate":
        N = rng.choice([1, 2, 9, 33, 64, 65, 129, 341])
        B = min(_log_int(rng, 1, 64), 16 * 341 * 48 * 128 // (N * (G + 1) * Hkv * D) + 1)
        return dict(op=op, B=B, N=N, Hq=G * Hkv, Hkv=Hkv, D=D, n_freq=n_freq, hi=_log_int(rng, 10, 1000000), dtype=dtype,
                    tree=rng.choice(["random", "narrow", "dense", "chain"]), interleaved=interleaved)
    if op == "append":
        B = _log_int(rng, 1, 32)
        T = min(_log_int(rng, 1, 4096), (1 << 26) // (B * (G + 1) * Hkv * D))
        return dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, n_freq=n_freq, lo=0, hi=_log_int(rng, 1, 1500), dtype=dtype,
                    interleaved=interleaved)
    if op == "attend":
        B = _log_int(rng, 1, 16)
        T = _log_int(rng, 1, 4096)
        hi = _log_int(rng, 40, 16384)
        # no more to do than the largest listed cases, 1 GB of cache and 2 GB of scores in the plain form
        most = (1 << 29) if dtype == "bf16" else (1 << 25)
        T = max(1, min(T, most // (40 * B * G * Hkv)))
        hi = max(40, min(hi, most // (B * T * G * Hkv) - T, (1 << 29) // (B * Hkv * D)))
        return dict(op=op, B=B, T=T, least=rng.choice([1, T, max(1, T // 2)]), Hq=G * Hkv, Hkv=Hkv, D=D, P=P,
                    lo=rng.choice([0, hi, hi // 2]), hi=hi, dtype=dtype)
    V = _log_int(rng, 100, 128256)
    N = rng.choice([1, 2, 9, 33, 64, 129, 341])
    B = max(1, min(_log_int(rng, 1, 64), (1 << 28) // (N * V)))
    return dict(op=op, B=B, N=N, V=V, tree=rng.choice(["random", "narrow", "dense", "chain"]))


# ---------------------------------------------------------------------------------------------------------------------
# inputs


def _quantised(x):
    """Codes and scales of x [n, Hkv, P, D]: the smallest power of two that brings a page's largest value to at most 448."""
    top = x.abs().amax((2, 3)).float()
    m, e = torch.frexp(top / E4M3_MAX)
    scale = torch.exp2(torch.where(m > 0.5, e, e - 1).float().clamp(-64, 64))
    return (x.float() / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _pool(g, n, Hkv, P, D, dev):
    """K and V pages as a model leaves them: some channels of K larger than others, V of a size that varies by page."""
    out = {}
    chan = torch.exp(0.5 * torch.randn(Hkv, 1, D, generator=g, device=dev))
    size = torch.exp(0.5 * torch.randn(n, Hkv, 1, 1, generator=g, device=dev))
    for name, by in (("k", chan), ("v", size)):
        codes = torch.empty(n, Hkv, P, D, dtype=torch.uint8, device=dev)
        scale = torch.empty(n, Hkv, dtype=torch.float32, device=dev)
        step = max(1, (1 << 27) // (Hkv * P * D))
        for i in range(0, n, step):
            m = min(step, n - i)
            x = torch.randn(m, Hkv, P, D, generator=g, device=dev) * (by if name == "k" else by[i:i + m])
            codes[i:i + m], scale[i:i + m] = _quantised(x)
        out[name + "_pages"], out[name + "_scale"] = codes, scale
    return out


def _lengths(g, B, lo, hi, dev):
    return torch.randint(lo, hi + 1, (B,), generator=g, device=dev).to(torch.int32)


def _table(g, lens, M, P, n_pages, dev):
    """Each sequence's pages, drawn without repetition from the pool."""
    perm = torch.randperm(n_pages, generator=g, device=dev)
    used = (lens.long() + P - 1) // P
    first = torch.cumsum(used, 0) - used
    j = torch.arange(M, device=dev)
    at = (first[:, None] + j[None, :]).clamp(max=n_pages - 1)
    return torch.where(j[None, :] < used[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32).contiguous()


def _parents(kind, N):
    """A tree is the program's choice, not the input's: the same for every seed."""
    if kind == "chain":
        return [-1] + list(range(N - 1))
    if kind == "dense":
        return [-1] + [(i - 1) // 4 for i in range(1, N)]
    if kind == "narrow":
        return [-1] + [max(0, (i - 1) // 3) for i in range(1, N)]
    u = torch.rand(N, generator=torch.Generator().manual_seed(N)).tolist()
    return [-1] + [int(u[i] * i) for i in range(1, N)]


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _inv_freq(n, dev):
    """The usual frequencies, 10000^(-i / n)."""
    return (10000.0 ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    dtype = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    B = c["B"]
    if c["op"] == "rotate":
        s["q"] = torch.randn(B, c["N"], c["Hq"], c["D"], generator=g, device=dev).to(dtype)
        s["k"] = torch.randn(B, c["N"], c["Hkv"], c["D"], generator=g, device=dev).to(dtype)
        s["kv_len"] = _lengths(g, B, 0, c["hi"], dev)
        s["inv_freq"] = _inv_freq(c["n_freq"], dev)
        s["depth"] = torch.tensor(_depths(_parents(c["tree"], c["N"])), dtype=torch.int32, device=dev)
    elif c["op"] == "append":
        T, P, D, Hkv = c["T"], c["P"], c["D"], c["Hkv"]
        M = -(-(c["hi"] + T) // P)
        n_pages = B * M + 3
        s.update(_pool(g, n_pages, Hkv, P, D, dev))
        s["kv_len"] = _lengths(g, B, c["lo"], c["hi"], dev)
        s["last"] = torch.randint(T // 2, T, (B,), generator=g, device=dev).to(torch.int32)
        s["page_table"] = _table(g, s["kv_len"] + s["last"] + 1, M, P, n_pages, dev)
        size = torch.exp(0.7 * torch.randn(B, T, 1, 1, generator=g, device=dev))
        s["q"] = torch.randn(B, T, c["Hq"], D, generator=g, device=dev).to(dtype)
        s["k_rows"] = torch.randn(B, T, Hkv, D, generator=g, device=dev).to(dtype)
        s["v_rows"] = (torch.randn(B, T, Hkv, D, generator=g, device=dev) * size).to(dtype)
        s["inv_freq"] = _inv_freq(c["n_freq"], dev)
    elif c["op"] == "attend":
        T, P, D, Hkv = c["T"], c["P"], c["D"], c["Hkv"]
        M = -(-(c["hi"] + T) // P) + 1
        n_pages = B * M + 3
        s.update(_pool(g, n_pages, Hkv, P, D, dev))
        s["last"] = torch.randint(c["least"] - 1, T, (B,), generator=g, device=dev).to(torch.int32)
        s["kv_len"] = _lengths(g, B, c["lo"], c["hi"], dev) + s["last"] + 1  # the chunk's own rows are in the pages
        s["page_table"] = _table(g, s["kv_len"], M, P, n_pages, dev)
        s["q"] = torch.randn(B, T, c["Hq"], D, generator=g, device=dev).to(dtype)
        s["scale"] = 1.0 / math.sqrt(D)
    else:
        N, V = c["N"], c["V"]
        parents = _parents(c["tree"], N)
        depth = _depths(parents)
        probs = torch.empty(B, N, V, dtype=torch.float32, device=dev)
        for b in range(B):  # peaked rows, as a language model's are
            probs[b] = torch.softmax(5.0 * torch.randn(N, V, generator=g, device=dev), -1)
        # a node's children hold the likeliest tokens of its row, as well-trained heads guess them
        rank, seen = [], {}
        for p in parents:
            rank.append(seen.get(p, 0))
            seen[p] = rank[-1] + 1
        k = min(V, 16)
        best = torch.topk(probs, k, -1).indices
        up = torch.tensor([max(p, 0) for p in parents], device=dev)
        r = torch.tensor(rank, device=dev)
        spare = torch.randint(0, V, (B, N), generator=g, device=dev)
        s["cand"] = torch.where(r < k, best[:, up, r.clamp(max=k - 1)], spare).to(torch.int32).contiguous()
        s["probs"] = probs
        s["parent"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        s["depth"] = torch.tensor(depth, dtype=torch.int32, device=dev)
        s["max_depth"] = max(depth)
        s["u"] = torch.rand(B, max(depth) + 1, generator=g, device=dev)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms


def _f32(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _turned(x, pos, inv_freq, interleaved):
    """x [B, T, H, D] at positions pos [B, T]: the first 2n values of a head are n pairs, (i, n + i) or neighbours."""
    n, f = inv_freq.shape[0], x.float()
    angle = pos.double()[:, :, None, None] * inv_freq.double()
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (f[..., 0:2 * n:2], f[..., 1:2 * n:2]) if interleaved else (f[..., :n], f[..., n:2 * n])
    pair = (a * c - b * s, b * c + a * s)
    turned = torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)
    return torch.cat([turned, f[..., 2 * n:]], -1)


def _plain_rotate(s):
    pos = s["kv_len"][:, None].long() + s["depth"][None].long()
    return {n: _turned(s[n], pos, s["inv_freq"], s["case"]["interleaved"]).to(s[n].dtype) for n in ("q", "k")}


def _new_scale(top, most):
    m, e = torch.frexp(top.double() / most)
    e = torch.where(m > 0.5, e, e - 1).float().clamp(-64, 64)
    return torch.where(top > 0, torch.exp2(e), torch.full_like(top, 2.0 ** -64))


def _plain_append(s):
    kv_len, last = s["kv_len"].long(), s["last"].long()
    B, T, Hkv, D = s["k_rows"].shape
    P, M = s["k_pages"].shape[2], s["page_table"].shape[1]
    dev = kv_len.device
    row = torch.arange(T, device=dev)
    pos = kv_len[:, None] + row
    inter = s["case"]["interleaved"]
    windows = (T + P - 2) // P + 1  # pages that T rows can touch
    page = (kv_len // P)[:, None] + torch.arange(windows, device=dev)
    i = page[:, :, None] * P + torch.arange(P, device=dev) - kv_len[:, None, None]  # which of the new rows a slot takes
    fresh = (i >= 0) & (i <= last[:, None, None])
    old = i < 0
    b, w = torch.nonzero(fresh.any(2), as_tuple=True)
    at = torch.gather(s["page_table"].long(), 1, page.clamp(max=M - 1))
    i = i.clamp(0, T - 1)
    out = {}
    for name, most in (("k", K_MAX), ("v", E4M3_MAX)):
        codes, scale = s[name + "_pages"], s[name + "_scale"]
        given = s[name + "_rows"].float()
        rows = _turned(given, pos, s["inv_freq"], inter) if name == "k" else given
        pick = torch.arange(B, device=dev)[:, None, None]
        sel = fresh[:, :, None, :, None]
        top = torch.where(sel, given[pick, i].permute(0, 1, 3, 2, 4).abs(), torch.zeros((), device=dev)).amax((3, 4))
        new = rows[pick, i].permute(0, 1, 3, 2, 4)  # [B, W, Hkv, P, D]
        had = codes[at.clamp(min=0)]
        s0 = scale[at.clamp(min=0)]
        keep = old.any(2)[:, :, None] & (top.double() <= most * s0.double())
        s1 = torch.where(keep, s0, _new_scale(top, most))
        val = torch.where(sel, new, _f32(had) * s0[..., None, None]) / s1[..., None, None]
        q = val.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        q = torch.where(sel | old[:, :, None, :, None], q, had)
        codes[at[b, w]] = q[b, w]
        scale[at[b, w]] = s1[b, w]
        out[name + "_pages"], out[name + "_scale"] = codes.view(torch.float8_e4m3fn), scale
    q = _turned(s["q"], pos, s["inv_freq"], inter)
    out["q"] = torch.where((row <= last[:, None])[:, :, None, None], q, torch.zeros_like(q)).to(s["q"].dtype)
    out["kv_len"] = (kv_len + last + 1).to(torch.int32)
    return out


def _plain_attend(s):
    q = s["q"].float()
    B, T, Hq, D = q.shape
    Hkv, P = s["k_pages"].shape[1], s["k_pages"].shape[2]
    G, M = Hq // Hkv, s["page_table"].shape[1]
    at = s["page_table"].clamp(min=0).long()
    k = _f32(s["k_pages"][at]) * s["k_scale"][at][..., None, None]
    v = _f32(s["v_pages"][at]) * s["v_scale"][at][..., None, None]
    k = k.transpose(1, 2).reshape(B, Hkv, 1, M * P, D)
    v = v.transpose(1, 2).reshape(B, Hkv, 1, M * P, D)
    slot, row = torch.arange(M * P, device=q.device), torch.arange(T, device=q.device)
    held = (slot[None] < s["kv_len"][:, None])[:, None, None, :, None]
    k, v = torch.where(held, k, torch.zeros((), device=q.device)), torch.where(held, v, torch.zeros((), device=q.device))
    real = row[None] <= s["last"][:, None]
    limit = torch.where(real, (s["kv_len"] - s["last"] - 1)[:, None] + row, torch.full_like(row, -1))  # last slot a row sees
    z = torch.matmul(q.reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4), k.transpose(3, 4)) * s["scale"]
    z = z.masked_fill(slot > limit[:, None, None, :, None], -math.inf)
    z = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38))
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(s["q"].dtype)


def _plain_verify(s):
    p = s["probs"]
    B, N, V = p.shape
    Dmax = s["max_depth"]
    dev = p.device
    at = torch.arange(B, device=dev)
    node = torch.zeros(B, dtype=torch.long, device=dev)
    going = torch.ones(B, dtype=torch.bool, device=dev)
    path = torch.full((B, Dmax + 1), -1, dtype=torch.long, device=dev)
    path[:, 0] = 0
    token = torch.full((B,), -1, dtype=torch.long, device=dev)
    index = torch.arange(N, device=dev)
    for d in range(Dmax + 1):
        c = torch.cumsum(p[at, node].double(), -1)  # in 64 bits: a token may end next to the number drawn
        t = torch.searchsorted(c, s["u"][:, d:d + 1].double() * c[:, -1:], right=True)[:, 0].clamp(max=V - 1)
        token = torch.where(going, t, token)
        child = torch.where((s["parent"][None] == node[:, None]) & (s["cand"] == t[:, None]), index, N).amin(1)
        going = going & (child < N)
        if d < Dmax:
            node = torch.where(going, child, node)
            path[:, d + 1] = torch.where(going, child, path[:, d + 1])
    i32 = torch.int32
    return {"accept_len": s["depth"][node].to(i32), "best_node": node.to(i32), "path_nodes": path.to(i32), "next_tok": token.to(i32)}


# ---------------------------------------------------------------------------------------------------------------------
# one pass


def _pools(s):
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}[op](s)
    import medusa_speculative_decoding_gb300 as M

    if op == "rotate":
        q, k = M.rope_rows(s["q"], s["k"], s["kv_len"], s["inv_freq"], depth=s["depth"], interleaved=s["case"]["interleaved"])
        return {"q": q, "k": k}
    if op == "append":
        r = M.kv_append_rope_q8(s["k_rows"], s["v_rows"], *_pools(s), s["page_table"], s["kv_len"], s["inv_freq"],
                                last=s["last"], q=s["q"], interleaved=s["case"]["interleaved"])
        return {"q": r["q"], "kv_len": r["kv_len"], "k_pages": s["k_pages"].view(torch.float8_e4m3fn),
                "v_pages": s["v_pages"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "attend":
        return M.chunk_attention_q8(s["q"], *_pools(s), s["page_table"], s["kv_len"], s["scale"], last=s["last"])
    return M.verify_accept_tree_draw(s["probs"], s["cand"], s["parent"], s["depth"], s["u"], s["max_depth"])


# ---------------------------------------------------------------------------------------------------------------------
# work and the definition in 64 bits


def work(case):
    c = case
    B = c["B"]
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "rotate":
        n = B * c["N"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 2.0 * n * c["D"] * size + 4 * (B + c["N"] + c["n_freq"]), "flops": 6.0 * n * c["n_freq"]}
    if c["op"] == "append":
        n = B * 0.75 * c["T"]
        row = n * c["Hkv"] * c["D"]
        return {"bytes": 2 * row * (size + 1) + 2.0 * size * n * c["Hq"] * c["D"], "flops": 6.0 * n * (c["Hq"] + c["Hkv"]) * c["n_freq"] + 4 * row}
    if c["op"] == "attend":
        n = (c["least"] + c["T"]) / 2  # new rows of a sequence
        L = (c["lo"] + c["hi"]) / 2 + n
        seen = n * (L - n + (n + 1) / 2)
        reads = L * 2 * c["Hkv"] * c["D"] + L / c["P"] * (8 * c["Hkv"] + 4)
        return {"bytes": B * (reads + 2 * n * c["Hq"] * c["D"] * size), "flops": 4.0 * B * seen * c["Hq"] * c["D"]}
    rows = min(2.0, 1 + 0.5 * (c["N"] - 1))  # rows that a walk visits
    return {"bytes": B * (rows * c["V"] * 4 + c["N"] * 4) + 8 * c["N"], "flops": B * rows * c["V"]}


def _e4m3_values(dev):
    """The 127 magnitudes of e4m3, from its definition."""
    v = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=dev)


def _to_grid(x):
    """x to the nearest e4m3 value, ties to the even code, largest values held at 448."""
    grid = _e4m3_values(x.device)
    a = x.abs().clamp(max=E4M3_MAX).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[code], x)


def _code_values(codes):
    v = torch.cat([_e4m3_values(codes.device), torch.full((1,), math.nan, dtype=torch.float64, device=codes.device)])
    return torch.where(codes >= 128, -v[(codes & 127).long()], v[(codes & 127).long()])


def _exact_turn(x, pos, inv_freq, interleaved):
    """x [T, H, D] in 64 bits as complex numbers times e^(i angle); pos [T]."""
    n = inv_freq.shape[0]
    x = x.double()
    head, tail = x[..., :2 * n], x[..., 2 * n:]
    z = head.reshape(*head.shape[:-1], n, 2) if interleaved else head.reshape(*head.shape[:-1], 2, n).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous())
    angle = pos.double()[:, None, None] * inv_freq.double()
    z = torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle))
    head = z.reshape(head.shape) if interleaved else z.transpose(-1, -2).reshape(head.shape)
    return torch.cat([head, tail], -1)


def _place(codes_at, scale_at, top, most, x, o):
    """A page's values [Hkv, P, D] and scale [Hkv] after rows x [Hkv, n, D] from slot o on."""
    e = torch.ceil(torch.log2(top / most))  # put right below where the logarithm was rounded
    e = torch.where(top > most * torch.exp2(e), e + 1, e)
    e = torch.where(top <= most * torch.exp2(e - 1), e - 1, e)
    new = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -64.0)).clamp(-64, 64))
    if o:
        new = torch.where(top <= most * scale_at, scale_at, new)
        codes_at[:, :o] = _to_grid(codes_at[:, :o] * (scale_at / new)[:, None, None])
    codes_at[:, o:o + x.shape[1]] = _to_grid(x / new[:, None, None])
    return new


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None  # tokens and nodes
    s = prepare(case, seed)
    lens = s["kv_len"].tolist()
    B = c["B"]
    if c["op"] == "rotate":
        return {n: torch.stack([_exact_turn(s[n][b], lens[b] + s["depth"], s["inv_freq"], c["interleaved"]) for b in range(B)])
                for n in ("q", "k")}
    last = s["last"].tolist()
    P, Hkv, D = c["P"], c["Hkv"], c["D"]
    if c["op"] == "attend":
        if 4.0 * B * c["T"] * (c["hi"] + c["T"]) * c["Hq"] * D > 4e12:
            return None
        G = c["Hq"] // Hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        for b in range(B):
            pages = s["page_table"][b, : -(-lens[b] // P)].long()
            n = last[b] + 1
            hidden = torch.ones(n, lens[b], dtype=torch.bool, device=out.device).triu(lens[b] - n + 1)
            for h in range(Hkv):
                kv = [(_code_values(s[m + "_pages"][pages, h]) * s[m + "_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[: lens[b]]
                      for m in ("k", "v")]
                for h2 in range(h * G, h * G + G):
                    z = (s["q"][b, :n, h2].double() @ kv[0].T * s["scale"]).masked_fill(hidden, -math.inf)
                    out[b, :n, h2] = torch.softmax(z, -1) @ kv[1]
        return out
    if s["k_pages"].numel() > 1 << 28:
        return None
    result = {"kv_len": None, "q": torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)}
    step = torch.arange(c["T"], device=s["q"].device)
    for m, most in (("k", K_MAX), ("v", E4M3_MAX)):
        values, scale = _code_values(s[m + "_pages"]).contiguous(), s[m + "_scale"].double()
        for b in range(B):
            n, at = last[b] + 1, lens[b]
            given = s[m + "_rows"][b, :n].double()
            rows = _exact_turn(given, at + step[:n], s["inv_freq"], c["interleaved"]) if m == "k" else given
            while rows.shape[0]:
                page, o = int(s["page_table"][b, at // P]), at % P
                x, rows = rows[: P - o].transpose(0, 1), rows[P - o:]
                top, given = given[: P - o].abs().amax((0, 2)), given[P - o:]
                at += x.shape[1]
                scale[page] = _place(values[page], scale[page], top, most, x, o)
        result[m + "_pages"], result[m + "_scale"] = values, scale
    for b in range(B):
        n = last[b] + 1
        result["q"][b, :n] = _exact_turn(s["q"][b, :n], lens[b] + step[:n], s["inv_freq"], c["interleaved"])
    return result
