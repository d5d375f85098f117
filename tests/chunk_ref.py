"""Plain definitions of the operators that fill the 8-bit paged cache from unrotated rows
and answer from it, in float64 and in sequential Python, written from the header's text
(include/medusa.h, parts 4d and 6e to 6g).  They share nothing with the library."""
import numpy as np

import q8_ref as R


def turned(x, pos, inv_freq, interleaved):
    """x [T, H, D], pos [T]: pair i of the row at p turns by p * inv_freq[i] (exact in float64
    for positions below 2^29)."""
    x = np.asarray(x, np.float64)
    n = len(inv_freq)
    out = x.copy()
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    t = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    out[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    out[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
    return out


def turn_error(x, n, interleaved):
    """What float32 may make of a turned value: cosine and sine are off by at most 2^-23 each
    (the angle by 2^-30, the functions and their argument's rounding by less than 1.5 units of
    2^-24), a product and the sum round once each: (|a| + |b|) * (2^-23 + 2 * 2^-24) = 2^-22."""
    x = np.abs(np.asarray(x, np.float64))
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    e = np.zeros_like(x)
    e[..., a] = e[..., b] = (x[..., a] + x[..., b]) * 2.0 ** -22
    return e


def fitting_scale(values, most):
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    top = v.max() if v.size else 0.0
    e = -64
    while e < 64 and top > most * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(k_rows, v_rows, k_pages, v_pages, k_scale, v_scale, table, kv_len, inv_freq, interleaved, rows=None, last=None, best=None):
    """(k values, v values, k_scale, v_scale, kv_len, appended, slack): values are the decoded
    codes [n, Hkv, P, D]; slack [n, Hkv, P, D] what a K value may be off by beside the nearest
    code's own distance, 0 where the code is fixed; exact: the exact quotients there."""
    n_pages, Hkv, P, D = k_pages.shape
    kc, vc, ks, vs = k_pages.copy(), v_pages.copy(), k_scale.copy(), v_scale.copy()
    slack, exact = np.zeros(k_pages.shape), R.decode(k_pages)
    B, T = k_rows.shape[:2]
    M = table.shape[1]
    width = rows.shape[1] if rows is not None else T
    new_len, count = kv_len.copy(), np.zeros(B, np.int32)
    for b in range(B):
        L, n = int(kv_len[b]), (int(last[b]) if last is not None else width - 1) + 1
        ok = 0 <= n <= width and 0 <= L and L + n <= M * P
        ok = ok and all(0 <= table[b, j] < n_pages for j in range(L // P, (L + n - 1) // P + 1 if n else L // P))
        ok = ok and (rows is None or all(0 <= r < T for r in rows[b, :n]))
        ok = ok and (best is None or 0 <= best[b] < T)
        if not ok:
            count[b] = -2
            continue
        take = rows[b, :n] if rows is not None else np.arange(n)
        for codes, scale, src, most in ((kc, ks, k_rows, 316.0), (vc, vs, v_rows, 448.0)):
            given = np.asarray(src[b, take], np.float64)
            turn = codes is kc
            with np.errstate(invalid="ignore"):
                value = turned(given, L + np.arange(n), inv_freq, interleaved) if turn else given
            off = turn_error(given, len(inv_freq), interleaved) if turn else np.zeros_like(given)
            for h in range(Hkv):
                done = 0
                while done < n:
                    at = L + done
                    p, o = int(table[b, at // P]), at % P
                    m = min(P - o, n - done)
                    s0 = float(scale[p, h])
                    g, y, e = given[done:done + m, h], value[done:done + m, h], off[done:done + m, h]
                    done += m
                    fin = np.abs(g[np.isfinite(g)])
                    if o and not R.readable(s0):
                        continue
                    if o and (fin.max() if fin.size else 0.0) <= most * s0:
                        s1 = s0
                    else:
                        s1 = fitting_scale(g, most)
                        if o:
                            codes[p, h, :o] = R.encode(R.decode(codes[p, h, :o]) * s0 / s1)
                    scale[p, h] = s1
                    codes[p, h, o:o + m] = R.encode(y / s1)
                    if turn:
                        slack[p, h, o:o + m] = np.where(np.isfinite(e), 2 * e / s1, 0)
                        exact[p, h, o:o + m] = y / s1
                        exact[p, h, :o] = R.decode(codes[p, h, :o])
        new_len[b], count[b] = L + n, n
    return kc, vc, ks, vs, new_len, count, slack, exact


def attention(q, k_pages, v_pages, k_scale, v_scale, table, kv_len, last, scale):
    """(out, spread, bounds) as q8_ref.attention, of a chunk: row i sees [0, L - n + i]."""
    B, T, Hq, D = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    G, cap = Hq // Hkv, table.shape[1] * P
    out, spread, bounds = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, 2))
    for b in range(B):
        L = min(max(int(kv_len[b]), 0), cap)
        n = T if last is None else min(max(int(last[b]), -1), T - 1) + 1
        for h in range(Hkv):
            k, v, there = np.zeros((L, D)), np.zeros((L, D)), np.zeros(L, bool)
            for s in range(0, L, P):
                p, m = int(table[b, s // P]), min(P, L - s)
                if 0 <= p < len(k_pages) and R.readable(k_scale[p, h]) and R.readable(v_scale[p, h]):
                    k[s:s + m] = R.decode(k_pages[p, h, :m]) * float(k_scale[p, h])
                    v[s:s + m] = R.decode(v_pages[p, h, :m]) * float(v_scale[p, h])
                    there[s:s + m] = True
            for i in range(n):
                see = np.flatnonzero(there[:max(0, L - n + i + 1)])
                if not len(see):
                    continue
                kk, vv = k[see], v[see]
                for g in range(h * G, h * G + G):
                    z = kk @ q[b, i, g] * scale
                    if np.isnan(z).any() or np.isnan(vv).any():
                        out[b, i, g] = np.nan
                        continue
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[b, i, g], spread[b, i, g] = p @ vv, p @ np.abs(vv)
                    bounds[b, i, g] = (np.abs(kk) @ np.abs(q[b, i, g])).max() * scale, np.abs(kk).sum(1).max() * scale
    return out, spread, bounds


U = 2.0 ** -24  # half a unit in the last place of float32, relative


def attention_tolerance(q, k_pages, table, kv_len, v_scale, ref, bf16):
    """What rounding may make of each output, from the call's documentation.

    Scores: products summed in float32, D terms, relative to sum |q||k|; a score off by e makes
    its weight off by e^e - 1 <= 1.01 e for e < 0.01, and the sum it is divided by likewise: 2.1 e.
    exp2's argument stays below 2^7 and rounds a few times (8 U * 128 of it in units of the
    score).  Sums over the keys in float32: each addition rounds once, relative to the sum of
    magnitudes.  bf16: q enters to 2^-21 of its row's largest; weights are rounded to f16, 2^-11,
    and below its normal range to half of its least step, 2^-25, in units of which the row's
    largest weight * V scale is at least 2^8: 2^-33, times a code of at most 448 and the V scale, for
    each key; the output rounds to bf16: 2^-8 (float32: 2^-24).
    bf16, T = 1 and at most 16 query heads a KV head, which is computed as a tree of no rows: q enters to
    2^-17 of the largest of its block (all of q here), weights have 9 bits, 2^-9, and below that half of
    e5m2's least step, 2^-17, in planes that hold at least 2^9 for the largest weight * V scale: 2^-26."""
    out, spread, bounds = ref
    row = bf16 and q.shape[1] == 1 and q.shape[2] <= 16 * k_pages.shape[1]
    keys = min(int(kv_len.max()), table.shape[1] * k_pages.shape[2])
    D = q.shape[3]
    e = (D + 8) * U * bounds[..., 0] + 8 * U * 128
    per = (2 * keys + 64) * U
    if bf16:
        e = e + (2.0 ** -17 * np.abs(q).max() if row else 2.0 ** -21 * np.abs(q).max(-1)) * bounds[..., 1]
        per = per + (2.0 ** -9 if row else 2.0 ** -11)
    tol = spread * (2.1 * e[..., None] + per)
    if bf16:
        vs = np.where(np.isfinite(v_scale), v_scale, 0)
        tol = tol + keys * (2.0 ** -26 if row else 2.0 ** -33) * 448 * vs[vs <= 2.0 ** 64].max(initial=0)
    return tol + np.abs(out) * (2.0 ** -8 if bf16 else 2.0 ** -24) + 1e-30


def draw(p, u):
    """The smallest v with p_0 + .. + p_v > u * sum, in whole numbers (float32 is a multiple
    of 2^-149); -1 where the row has no weight."""
    p = np.asarray(p, np.float32)
    p = np.where(p > 0, np.minimum(p, np.float32(1)), np.float32(0))
    w = [int(x) for x in p.astype(np.float64) * 2.0 ** 149]
    num, den = min(max(u, 0.0), 2.0).as_integer_ratio() if u == u else (0, 1)
    total, c, token = sum(w), 0, -1
    for v, x in enumerate(w):
        c += x
        if x:
            token = v
            if c * den > num * total:
                break
    return token


def verify(probs, cand, parent, u, max_depth):
    B, N = cand.shape
    accept, best, nxt = np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    path = np.full((B, max_depth + 1), -1, np.int32)
    for b in range(B):
        node, d = 0, 0
        path[b, 0] = 0
        while True:
            t = draw(probs[b, node], float(u[b, d]))
            kids = [j for j in range(node + 1, N) if parent[j] == node and t >= 0 and cand[b, j] == t]
            if not kids or d == max_depth:
                break
            node, d = kids[0], d + 1
            path[b, d] = node
        accept[b], best[b], nxt[b] = d, node, t
    return dict(accept_len=accept, best_node=best, path_nodes=path, next_tok=nxt)
