"""Measured cases of the operators around the 8-bit paged KV cache: tree attention that reads it, the append that
quantises new rows into it, the fork that shares, copies, frees and reserves its pages, and the compaction of its pool.

The pool holds e4m3 codes [n_pages, Hkv, P, D] for K and V with one float32 scale per page and KV head; page_table
[B, M] (-1: no page) and kv_len [B] say what each sequence holds.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------------------------
# cases


def _attention(name, B, N, Hq, Hkv, D, P, lo, hi, dtype, tree):
    return dict(name=name, op="attention", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, P=P, lo=lo, hi=hi, dtype=dtype, tree=tree)


def _append(name, B, T, R, Hkv, D, P, lo, hi, dtype):
    return dict(name=name, op="append", B=B, T=T, R=R, Hkv=Hkv, D=D, P=P, lo=lo, hi=hi, dtype=dtype)


def _fork(name, B, beams, need, Hkv, D, P, lo, hi):
    return dict(name=name, op="fork", B=B, beams=beams, need=need, Hkv=Hkv, D=D, P=P, lo=lo, hi=hi)


def _compact(name, B, n_pages, fill, Hkv, D, P):
    return dict(name=name, op="compact", B=B, n_pages=n_pages, fill=fill, Hkv=Hkv, D=D, P=P)


def listed():
    return [
        # the tiny float32 step: nine tree nodes on a short prefix, where the call's own cost is all there is
        _attention("attend tiny f32", 1, 9, 4, 4, 64, 16, 128, 128, "f32", "narrow"),
        # one sequence's sparse 64-node tree on a 2048-token prefix, 32 heads
        _attention("attend 64 nodes b1 kv2048", 1, 64, 32, 32, 128, 64, 2048, 2048, "bf16", "random"),
        # a batch of eight ragged sequences of the 13B shape
        _attention("attend 64 nodes b8 ragged", 8, 64, 40, 40, 128, 64, 1024, 4096, "bf16", "random"),
        # the dense 341-node tree at KV 8192: the most arithmetic
        _attention("attend 341 nodes b4 kv8192", 4, 341, 32, 32, 128, 128, 8192, 8192, "bf16", "dense"),
        # plain decoding, one token a sequence, shared KV heads, long ragged caches in small pages
        _attention("attend 1 token b16 gqa", 16, 1, 32, 8, 128, 32, 777, 16384, "bf16", "dense"),
        # the accepted branch of each tree written after a round, batch 8
        _append("append accepted b8", 8, 64, 6, 40, 128, 64, 1024, 4096, "bf16"),
        # four ragged prompts written at once
        _append("append prompts b4", 4, 4096, 0, 32, 128, 64, 0, 200, "bf16"),
        # each round's bookkeeping: room for the next accepted branch in a batch of 64, nothing forked
        _fork("reserve b64", 64, 0, 8, 8, 128, 16, 100, 8192),
        # sampling several continuations: every fourth row goes on in four rows, the other rows are dropped
        _fork("fork beams b64", 64, 4, 8, 8, 128, 64, 100, 2048),
        # a small pool with few holes
        _compact("compact 512 pages", 4, 512, 0.9, 8, 64, 16),
        # a large pool half freed
        _compact("compact 8192 pages", 64, 8192, 0.5, 8, 128, 64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "fork", "compact"])
    D = rng.choice([64, 128, 128])
    P = rng.choice([16, 32, 64, 128])
    if op == "attention":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hkv = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
        G = rng.choice([g for g in (1, 1, 2, 3, 4, 7, 8) if g * Hkv <= 64])
        N = rng.choice([1, 1, 2, 9, 33, 64, 64, 65, 129, 341])
        B = _log_int(rng, 1, 16)
        hi = _log_int(rng, 40, 16384)
        # no more to do than the largest listed cases: 341 nodes x 32 heads x 4 sequences at 8192, 2 GB of cache
        most = 4 * 341 * 32 * 8192 if dtype == "bf16" else 64 * 32 * 2048
        hi = max(40, min(hi, most // (B * N * G * Hkv), (1 << 30) // (2 * B * Hkv * D)))
        B = max(1, min(B, most // (hi * N * G * Hkv)))
        N = max(1, min(N, most // (hi * B * G * Hkv)))
        return dict(op=op, B=B, N=N, Hq=G * Hkv, Hkv=Hkv, D=D, P=P, lo=rng.randint(0, hi), hi=hi, dtype=dtype,
                    tree=rng.choice(["random", "narrow", "dense"]))
    Hkv = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        B = _log_int(rng, 1, 32)
        if rng.random() < 0.5:
            T, R = rng.choice([1, 9, 64, 341]), rng.randint(1, 7)
        else:
            T, R = min(_log_int(rng, 1, 4096), (1 << 26) // (B * Hkv * D)), 0
        return dict(op=op, B=B, T=T, R=R, Hkv=Hkv, D=D, P=P, lo=0, hi=_log_int(rng, 1, 1500), dtype=dtype)
    if op == "fork":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 8, min(8192, (1 << 30) // (2 * B * Hkv * D)))
        return dict(op=op, B=B, beams=rng.choice([0, 1, 2, 3, 5]), need=rng.choice([0, 1, 6, 40, 300]), Hkv=Hkv, D=D, P=P,
                    lo=rng.randint(0, hi), hi=hi)
    n = min(_log_int(rng, 20, 8192), (1 << 30) // (2 * Hkv * D * P))
    return dict(op=op, B=_log_int(rng, 1, 64), n_pages=max(20, n), fill=round(rng.uniform(0.1, 0.95), 3), Hkv=Hkv, D=D, P=P)


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


def _parents(kind, N, g):
    if kind == "dense":
        return [-1] + [(i - 1) // 4 for i in range(1, N)]
    if kind == "narrow":
        return [-1] + [max(0, (i - 1) // 3) for i in range(1, N)]
    u = torch.rand(N, generator=g).tolist()
    return [-1] + [int(u[i] * i) for i in range(1, N)]


def _mask(parents, dev):
    N = len(parents)
    rows = []
    for i in range(N):
        bits, j = 0, i
        while j >= 0:
            bits |= 1 << j
            j = parents[j]
        words = [(bits >> (64 * w)) & ((1 << 64) - 1) for w in range((N + 63) // 64)]
        rows.append([w - (1 << 64) if w >> 63 else w for w in words])
    return torch.tensor(rows, dtype=torch.int64, device=dev)


def _table(g, lens, M, P, n_pages, dev, spare=0):
    """Each sequence's pages, drawn without repetition from the pool."""
    perm = torch.randperm(n_pages, generator=g, device=dev)
    used = (lens.long() + P - 1) // P + spare
    first = torch.cumsum(used, 0) - used
    j = torch.arange(M, device=dev)
    at = (first[:, None] + j[None, :]).clamp(max=n_pages - 1)
    return torch.where(j[None, :] < used[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    dtype = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    P, D, Hkv, B = c["P"], c["D"], c["Hkv"], c["B"]
    if c["op"] == "attention":
        M = -(-c["hi"] // P) + 1
        n_pages = B * M + 3
        s.update(_pool(g, n_pages, Hkv, P, D, dev))
        s["kv_len"] = _lengths(g, B, c["lo"], c["hi"], dev)
        s["page_table"] = _table(g, s["kv_len"], M, P, n_pages, dev)
        N = c["N"]
        s["q"] = torch.randn(B, N, c["Hq"], D, generator=g, device=dev).to(dtype)
        s["k_tree"] = torch.randn(B, N, Hkv, D, generator=g, device=dev).to(dtype)
        s["v_tree"] = torch.randn(B, N, Hkv, D, generator=g, device=dev).to(dtype)
        s["mask"] = _mask(_parents(c["tree"], N, gc), dev)
        s["scale"] = 1.0 / math.sqrt(D)
    elif c["op"] == "append":
        R = c["R"] or c["T"]
        M = -(-(c["hi"] + R) // P)
        n_pages = B * M + 3
        s.update(_pool(g, n_pages, Hkv, P, D, dev))
        s["kv_len"] = _lengths(g, B, c["lo"], c["hi"], dev)
        s["last"] = torch.randint(-1 if c["R"] else c["T"] // 2, R, (B,), generator=g, device=dev).to(torch.int32)
        s["page_table"] = _table(g, s["kv_len"] + s["last"] + 1, M, P, n_pages, dev)
        size = torch.exp(0.7 * torch.randn(B, c["T"], 1, 1, generator=g, device=dev))
        s["k_rows"] = torch.randn(B, c["T"], Hkv, D, generator=g, device=dev).to(dtype)
        s["v_rows"] = (torch.randn(B, c["T"], Hkv, D, generator=g, device=dev) * size).to(dtype)
        s["rows"] = None
        if c["R"]:  # a branch from the root (row 0) down: rising rows
            r = torch.randint(0, c["T"], (B, R), generator=g, device=dev)
            r[:, 0] = 0
            s["rows"] = torch.sort(r, 1).values.to(torch.int32).contiguous()
    elif c["op"] == "fork":
        M = -(-(c["hi"] + c["need"]) // P)
        n_pages = B * (M + 2)
        s.update(_pool(g, n_pages, Hkv, P, D, dev))
        s["kv_len"] = _lengths(g, B, c["lo"], c["hi"], dev)
        s["page_table"] = _table(g, s["kv_len"], M, P, n_pages, dev)
        s["need"] = torch.randint(0, c["need"] + 1, (B,), generator=g, device=dev).to(torch.int32)
        s["src"] = None
        if c["beams"]:  # each group goes on from one of its rows; some rows end
            b = torch.arange(B, device=dev) // c["beams"] * c["beams"]
            pick = torch.randint(0, c["beams"], (B,), generator=g, device=dev)[b]
            src = torch.minimum(b + pick, torch.full_like(b, B - 1))
            ended = torch.rand(B, generator=g, device=dev) < 0.05
            s["src"] = torch.where(ended, torch.full_like(src, -1), src).to(torch.int32)
    else:
        n_pages = c["n_pages"]
        s.update(_pool(g, n_pages, Hkv, P, D, dev))
        used = max(B, int(n_pages * c["fill"]))
        cut = torch.sort(torch.randint(0, max(1, used - B) + 1, (B - 1,), generator=g, device=dev)).values
        edge = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), max(0, used - B))])
        pages = (edge[1:] - edge[:-1]).clamp(max=4 * used // B + 1)
        M = 4 * used // B + 2
        s["page_table"] = _table(g, (pages * P).to(torch.int32), M, P, n_pages, dev)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms


def _f32(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_attention(s):
    q, kt, vt = s["q"].float(), s["k_tree"].float(), s["v_tree"].float()
    B, N, Hq, D = q.shape
    Hkv, P = s["k_pages"].shape[1], s["k_pages"].shape[2]
    G, M = Hq // Hkv, s["page_table"].shape[1]
    at = s["page_table"].clamp(min=0).long()
    k = _f32(s["k_pages"][at]) * s["k_scale"][at][..., None, None]
    v = _f32(s["v_pages"][at]) * s["v_scale"][at][..., None, None]
    k = k.transpose(1, 2).reshape(B, Hkv, M * P, D)
    v = v.transpose(1, 2).reshape(B, Hkv, M * P, D)
    qh = q.reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    held = torch.arange(M * P, device=q.device)[None] < s["kv_len"][:, None]
    sp = torch.matmul(qh, k.transpose(2, 3)) * s["scale"]
    sp = sp.masked_fill(~held[:, None, None, :], -math.inf)
    bit = torch.arange(N, device=q.device)
    seen = ((s["mask"][:, bit // 64] >> (bit % 64)) & 1).bool()
    st = torch.matmul(qh, kt.permute(0, 2, 3, 1)) * s["scale"]
    st = st.masked_fill(~seen.repeat_interleave(G, 0), -math.inf)
    top = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
    sp, st = torch.exp(sp - top), torch.exp(st - top)
    v = torch.where(held[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(sp, v) + torch.matmul(st, vt.transpose(1, 2))
    o = o / (sp.sum(-1, keepdim=True) + st.sum(-1, keepdim=True))
    o = o.reshape(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    return o.to(s["q"].dtype)


def _new_scale(top):
    m, e = torch.frexp(top / E4M3_MAX)
    e = torch.where(m > 0.5, e, e - 1).float().clamp(-64, 64)
    return torch.where(top > 0, torch.exp2(e), torch.full_like(top, 2.0 ** -64))


def _plain_append(s):
    kv_len, last = s["kv_len"].long(), s["last"].long()
    B, T, Hkv, D = s["k_rows"].shape
    P, M = s["k_pages"].shape[2], s["page_table"].shape[1]
    R = s["rows"].shape[1] if s["rows"] is not None else T
    dev = kv_len.device
    windows = (R + P - 2) // P + 1  # pages that R rows can touch
    first = kv_len // P
    page = first[:, None] + torch.arange(windows, device=dev)
    slot = page[:, :, None] * P + torch.arange(P, device=dev)
    i = slot - kv_len[:, None, None]  # which of the new rows the slot takes
    fresh = (i >= 0) & (i <= last[:, None, None])
    old = i < 0
    touched = fresh.any(2)
    i = i.clamp(0, R - 1)
    r = i if s["rows"] is None else torch.gather(s["rows"].long(), 1, i.reshape(B, -1)).reshape(i.shape)
    at = torch.gather(s["page_table"].long(), 1, page.clamp(max=M - 1))
    out = {}
    for name in ("k", "v"):
        codes, scale = s[name + "_pages"], s[name + "_scale"]
        new = s[name + "_rows"][torch.arange(B, device=dev)[:, None, None], r].float()  # [B, W, P, Hkv, D]
        new = new.permute(0, 1, 3, 2, 4)
        sel = fresh[:, :, None, :, None]
        top = torch.where(sel, new.abs(), torch.zeros_like(new)).amax((3, 4))
        had = codes[at.clamp(min=0)]
        s0 = scale[at.clamp(min=0)]
        keep = old.any(2)[:, :, None] & (top <= E4M3_MAX * s0)
        s1 = torch.where(keep, s0, _new_scale(top))
        val = torch.where(sel, new, _f32(had) * s0[..., None, None]) / s1[..., None, None]
        q = val.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        q = torch.where(sel | old[:, :, None, :, None], q, had)
        b, w = torch.nonzero(touched, as_tuple=True)
        codes[at[b, w]] = q[b, w]
        scale[at[b, w]] = s1[b, w]
        out[name + "_pages"], out[name + "_scale"] = codes.view(torch.float8_e4m3fn), scale
    out["kv_len"] = (kv_len + last + 1).to(torch.int32)
    return out


def _plain_fork(s):
    table, kv_len, need = s["page_table"].long(), s["kv_len"].long(), s["need"].long()
    B, M = table.shape
    n, P = s["k_pages"].shape[0], s["k_pages"].shape[2]
    dev = table.device
    b, j = torch.arange(B, device=dev), torch.arange(M, device=dev)
    src = s["src"].long() if s["src"] is not None else b
    alive = src >= 0
    at = src.clamp(min=0)
    length = torch.where(alive, kv_len[at], torch.zeros_like(src))
    # of the rows that go on from one source, the source itself or else the first keeps its open page
    same = (src[:, None] == src[None, :]) & alive[:, None]
    lead = torch.where(same, torch.where(b[None, :] == src[None, :], -1, b[None, :]), B).amin(1)
    lead = torch.where(lead < 0, src, lead)
    keeps = alive & (lead == b)
    whole, pages = length // P, (length + P - 1) // P
    valid = (table >= 0) & (table < n)
    run = torch.cumprod(valid.long(), 1).sum(1)[at]  # leading pages of the source
    have = torch.where(keeps, run, whole) * alive
    out = torch.where(j[None] < have[:, None], table[at], torch.full_like(table, -1))
    copies = alive & ~keeps & (pages > whole)
    want = (length + need + P - 1) // P
    fits = want <= M
    takes = (want - have).clamp(min=0) * alive
    takes = torch.where(copies, torch.maximum(takes, torch.ones_like(takes)), takes) * fits
    used = torch.zeros(n + 1, dtype=torch.long, device=dev).scatter_add_(
        0, torch.where(out >= 0, out, torch.full_like(out, n)).reshape(-1), torch.ones(B * M, dtype=torch.long, device=dev))[:n]
    free = torch.sort(torch.where(used == 0, torch.arange(n, device=dev), torch.full_like(used, n))).values
    first = torch.cumsum(takes, 0) - takes
    served = fits & (first + takes <= (used == 0).sum())
    k = j[None] - have[:, None]
    gets = served[:, None] & (k >= 0) & (k < takes[:, None])
    out = torch.where(gets, free[(first[:, None] + k).clamp(0, n - 1)], out)
    copied = torch.nonzero(copies & served, as_tuple=True)[0]
    if copied.numel():
        a, d = table[at[copied], whole[copied]], out[copied, whole[copied]]
        rows = torch.arange(P, device=dev)[None] < (length - whole * P)[copied][:, None]
        for name in ("k", "v"):
            codes, scale = s[name + "_pages"], s[name + "_scale"]
            codes[d] = torch.where(rows[:, None, :, None], codes[a], codes[d])
            scale[d] = scale[a]
    length = torch.where(copies & ~served, whole * P, length)
    used = used.scatter_add(0, torch.where(gets, out, torch.zeros_like(out)).reshape(-1), gets.long().reshape(-1))
    i32 = torch.int32
    return {"page_table": out.to(i32), "kv_len": length.to(i32), "refs": used.to(i32),
            "taken": torch.where(served, takes, torch.where(alive, -1, 0)).to(i32),
            "k_pages": s["k_pages"].view(torch.float8_e4m3fn), "v_pages": s["v_pages"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_compact(s):
    table = s["page_table"].long()
    n, dev = s["k_pages"].shape[0], table.device
    valid = (table >= 0) & (table < n)
    live = torch.zeros(n + 1, dtype=torch.bool, device=dev)
    live[torch.where(valid, table, torch.full_like(table, n)).reshape(-1)] = True
    live = live[:n]
    count = live.sum()
    idx = torch.arange(n, device=dev)
    src = torch.nonzero(live & (idx >= count), as_tuple=True)[0]
    dst = torch.nonzero(~live & (idx < count), as_tuple=True)[0]
    new = torch.where(live, idx, torch.full_like(idx, -1))
    new[src] = dst
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        s[name][dst] = s[name][src]
    out = torch.where(valid, new[table.clamp(0, n - 1)], torch.full_like(table, -1))
    return {"page_table": out.to(torch.int32), "new_page": new.to(torch.int32), "live": count.to(torch.int32).reshape(1),
            "k_pages": s["k_pages"].view(torch.float8_e4m3fn), "v_pages": s["v_pages"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ---------------------------------------------------------------------------------------------------------------------
# one pass


def _pools(s):
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _with_pools(s, out):
    return {**out, "k_pages": s["k_pages"].view(torch.float8_e4m3fn), "v_pages": s["v_pages"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"attention": _plain_attention, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}[op](s)
    import medusa_speculative_decoding_gb300 as M

    if op == "attention":
        return M.tree_attention_q8(s["q"], s["k_tree"], s["v_tree"], *_pools(s), s["page_table"], s["kv_len"], s["mask"], s["scale"])
    if op == "append":
        r = M.kv_append_q8(s["k_rows"], s["v_rows"], *_pools(s), s["page_table"], s["kv_len"], rows=s["rows"], last=s["last"])
        return _with_pools(s, {"kv_len": r["kv_len"]})
    if op == "fork":
        r = M.kv_pages_fork(*_pools(s), s["page_table"], s["kv_len"], src=s["src"], need=s["need"])
        return _with_pools(s, {k: r[k] for k in ("page_table", "kv_len", "refs", "taken")})
    r = M.kv_pages_compact(*_pools(s), s["page_table"])
    return _with_pools(s, {k: r[k] for k in ("page_table", "new_page", "live")})


# ---------------------------------------------------------------------------------------------------------------------
# work and the definition in 64 bits


def work(case):
    c = case
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    row = 2 * Hkv * D  # bytes of one token's codes, K and V
    if c["op"] == "attention":
        size = 4 if c["dtype"] == "f32" else 2
        L = B * (c["lo"] + c["hi"]) / 2
        reads = L * row + (L / P) * Hkv * 8 + L / P * 4 + B * c["N"] * 2 * Hkv * D * size
        q = B * c["N"] * c["Hq"] * D * size
        return {"bytes": reads + 2 * q, "flops": 4.0 * D * c["N"] * c["Hq"] * (L + B * c["N"])}
    if c["op"] == "append":
        size = 4 if c["dtype"] == "f32" else 2
        n = B * (c["R"] / 2 if c["R"] else 0.75 * c["T"])
        return {"bytes": n * row * (size + 1) + B * 12, "flops": 2.0 * n * row}
    if c["op"] == "fork":
        M = -(-(c["hi"] + c["need"]) // P)
        moved = B * 0.95 * (1 - 1 / c["beams"]) * P / 2 * row if c["beams"] else 0
        return {"bytes": 2 * moved + 8.0 * B * M + 4.0 * B * (M + 2), "flops": 0}
    moves = c["n_pages"] * c["fill"] * (1 - c["fill"])
    M = 4 * int(c["n_pages"] * c["fill"]) // B + 2
    return {"bytes": 2 * moves * P * row + 8.0 * B * M + 4.0 * c["n_pages"], "flops": 0}


_GRID = None


def _e4m3_values(dev):
    """The 127 magnitudes of e4m3, from its definition."""
    v = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=dev)


def _to_grid(x):
    """x to the nearest e4m3 value, ties to the even code, largest values held at 448."""
    grid = _e4m3_values(x.device)
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[code], x)


def _code_values(codes):
    v = torch.cat([_e4m3_values(codes.device), torch.full((1,), math.nan, dtype=torch.float64, device=codes.device)])
    return torch.where(codes >= 128, -v[(codes & 127).long()], v[(codes & 127).long()])


def exact(case, seed):
    c = case
    if c["op"] not in ("attention", "append"):
        return None  # pages, counts and moved bytes: nothing is computed
    s = prepare(case, seed)
    lens = s["kv_len"].tolist()
    B, P, Hkv, D = c["B"], c["P"], c["Hkv"], c["D"]
    if c["op"] == "attention":
        G, N = c["Hq"] // Hkv, c["N"]
        words = s["mask"].cpu().tolist()
        sees = torch.tensor([[(words[i][m // 64] >> (m % 64)) & 1 for m in range(N)] for i in range(N)], dtype=torch.bool, device=s["q"].device)
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        for b in range(B):
            pages = s["page_table"][b, : -(-lens[b] // P)].long()
            for h in range(Hkv):
                kv = []
                for n in ("k", "v"):
                    x = _code_values(s[n + "_pages"][pages, h]) * s[n + "_scale"][pages, h].double()[:, None, None]
                    kv.append(torch.cat([x.reshape(-1, D)[: lens[b]], s[n + "_tree"][b, :, h].double()]))
                for h2 in range(h * G, h * G + G):
                    z = s["q"][b, :, h2].double() @ kv[0].T * s["scale"]
                    z[:, lens[b]:][~sees] = -math.inf
                    out[b, :, h2] = torch.softmax(z, -1) @ kv[1]
        return out
    result = {}
    last = s["last"].tolist()
    for n in ("k", "v"):
        codes, scale = s[n + "_pages"], s[n + "_scale"].double()
        if codes.numel() > 1 << 28:
            return None
        values = _code_values(codes).contiguous()
        for b in range(B):
            rows = s[n + "_rows"][b].double()
            rows = rows[s["rows"][b].long()] if s["rows"] is not None else rows
            rows, at = rows[: last[b] + 1], lens[b]
            while rows.shape[0]:
                page, o = int(s["page_table"][b, at // P]), at % P
                x, rows = rows[: P - o], rows[P - o:]
                x = x.transpose(0, 1)  # [Hkv, n, D]
                at += x.shape[1]
                top = x.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / E4M3_MAX))  # put right below where the logarithm was rounded
                e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
                e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
                new = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -64.0)).clamp(-64, 64))
                if o:
                    new = torch.where(top <= E4M3_MAX * scale[page], scale[page], new)
                    values[page, :, :o] = _to_grid((values[page, :, :o] * (scale[page] / new)[:, None, None]).contiguous())
                values[page, :, o:o + x.shape[1]] = _to_grid((x / new[:, None, None]).contiguous())
                scale[page] = new
        result[n + "_pages"], result[n + "_scale"] = values, scale
    result["kv_len"] = None
    return result
