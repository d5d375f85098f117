"""Plain definitions of the 8-bit paged cache's operators, in float64 and in
sequential Python, written from the header's text (include/medusa.h, part 6).
They share nothing with the library."""
import math

import numpy as np

# ---------------------------------------------------------------------------
# e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities, 0x7f is NaN
_MAG = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])
VALUES = np.concatenate([_MAG, [np.nan], -_MAG, [np.nan]])


def decode(codes):
    return VALUES[np.asarray(codes)]


def encode(x):
    """Nearest e4m3 code, ties to the even code, held at 448, NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 448.0)
    hi = np.clip(np.searchsorted(_MAG, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _MAG[hi] - a, a - _MAG[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.isnan(x), 127, c + 128 * np.signbit(x))
    return c.astype(np.uint8)


def page_scale(values):
    """The smallest 2^e, e in [-64, 64], with |x| <= 448 * 2^e for the finite values."""
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    top = v.max() if v.size else 0.0
    e = -64
    while e < 64 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def page_scales(x):
    """page_scale of every [n, Hkv] block of x [n, Hkv, P, D]."""
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max((2, 3))
    e = np.full(top.shape, -64.0)
    for _ in range(128):
        e = np.where((e < 64) & (top > 448.0 * 2.0 ** e), e + 1, e)
    return 2.0 ** e


def readable(s):
    return bool(2.0 ** -64 <= s <= 2.0 ** 64)


# ---------------------------------------------------------------------------
def prefix(pages, scale, other_scale, table, L, h):
    """Values [n, D] of one head's readable prefix keys (the slots whose page and
    scales count)."""
    n_pages, _, P, D = pages.shape
    rows = [np.zeros((0, D))]
    for j in range(-(-L // P)):
        p = int(table[j])
        if 0 <= p < n_pages and readable(scale[p, h]) and readable(other_scale[p, h]):
            rows.append(decode(pages[p, h, : min(P, L - j * P)]) * float(scale[p, h]))
    return np.concatenate(rows)


def sees(mask, N):
    m = np.asarray(mask).view(np.uint64).reshape(N, -1)
    k = np.arange(N)
    return ((m[:, k >> 6] >> (k & 63).astype(np.uint64)) & np.uint64(1)).astype(bool)


def attention(q, k_tree, v_tree, k_pages, v_pages, k_scale, v_scale, table, kv_len, mask, scale):
    """(out, spread, score bounds): out [B,N,Hq,D]; spread = sum_j p_j |v_j|, the
    scale of a relative error of the weights; bounds [B,N,Hq,2] =
    max_j scale * sum_d |q_d k_jd| and max_j scale * sum_d |k_jd|."""
    B, N, Hq, D = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    G, cap = Hq // Hkv, table.shape[1] * P
    seen = sees(mask, N)
    out, spread, bounds = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, 2))
    for b in range(B):
        L = min(max(int(kv_len[b]), 0), cap)
        for h in range(Hkv):
            kp = prefix(k_pages, k_scale, v_scale, table[b], L, h)
            vp = prefix(v_pages, v_scale, k_scale, table[b], L, h)
            k, v = np.concatenate([kp, k_tree[b, :, h]]), np.concatenate([vp, v_tree[b, :, h]])
            vis = np.concatenate([np.ones((N, len(kp)), bool), seen], 1)
            some = vis.any(1)
            for g in range(h * G, h * G + G):
                z = np.where(vis, q[b, :, g] @ k.T * scale, -np.inf)[some]
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[b, some, g], spread[b, some, g] = p @ v, p @ np.abs(v)
                bounds[b, some, g, 0] = np.where(vis, np.abs(q[b, :, g]) @ np.abs(k).T * scale, 0)[some].max(1)
                bounds[b, some, g, 1] = np.where(vis, np.abs(k).sum(1) * scale, 0)[some].max(1)
    return out, spread, bounds


def append(k_rows, v_rows, k_pages, v_pages, k_scale, v_scale, table, kv_len, rows=None, last=None, best=None):
    """Pools, lengths and counts after the call (the pools are copied)."""
    pools = [k_pages.copy(), v_pages.copy(), k_scale.copy(), v_scale.copy()]
    B, T, Hkv, D = k_rows.shape
    n_pages, P, M = k_pages.shape[0], k_pages.shape[2], table.shape[1]
    R = rows.shape[1] if rows is not None else T
    new_len, count = kv_len.copy(), np.zeros(B, np.int32)
    for b in range(B):
        L, n = int(kv_len[b]), (int(last[b]) if last is not None else R - 1) + 1
        ok = 0 <= n <= R and 0 <= L and L + n <= M * P
        ok = ok and all(0 <= table[b, j] < n_pages for j in range(L // P, (L + n - 1) // P + 1 if n else L // P))
        ok = ok and (rows is None or all(0 <= r < T for r in rows[b, :n]))
        ok = ok and (best is None or 0 <= best[b] < T)
        if not ok:
            count[b] = -2
            continue
        take = rows[b, :n] if rows is not None else np.arange(n)
        for codes, scale, src in ((pools[0], pools[2], k_rows), (pools[1], pools[3], v_rows)):
            for h in range(Hkv):
                x, at = np.asarray(src[b, take, h], np.float64), L
                while len(x):
                    p, o = int(table[b, at // P]), at % P
                    y, x = x[: P - o], x[P - o:]
                    at += len(y)
                    s0 = float(scale[p, h])
                    fin = np.abs(y[np.isfinite(y)])
                    if o and not readable(s0):
                        continue
                    if o and (fin.max() if fin.size else 0.0) <= 448.0 * s0:
                        s1 = s0
                    else:
                        s1 = page_scale(y)
                        if o:
                            codes[p, h, :o] = encode(decode(codes[p, h, :o]) * s0 / s1)
                    scale[p, h] = s1
                    codes[p, h, o:o + len(y)] = encode(y / s1)
        new_len[b], count[b] = L + n, n
    return (*pools, new_len, count)


def fork(table, kv_len, n_pages, P, src=None, need=None, held=None):
    """(table, kv_len, refs, taken, copies): copies = [(from page, to page, rows)]."""
    B, M = table.shape
    src = list(range(B)) if src is None else [int(x) for x in src]
    need = [0] * B if need is None else [max(int(x), 0) for x in need]
    run = []
    for b in range(B):
        j = 0
        while j < M and 0 <= table[b, j] < n_pages:
            j += 1
        run.append(j)
    taken, bad = [0] * B, [False] * B
    for b in range(B):
        s = src[b]
        if s == -1:
            continue
        bad[b] = s < -1 or s >= B or not 0 <= kv_len[s] <= M * P or math.ceil(kv_len[s] / P) > run[s]
        if bad[b]:
            taken[b] = -2
    rows = [[] for _ in range(B)]
    length, copies, keeper = [0] * B, [], {}
    for b in range(B):
        s = src[b]
        if s >= 0 and not bad[b] and (s not in keeper or s == b):
            keeper[s] = b
    refs = np.zeros(n_pages, np.int64) + (0 if held is None else np.maximum(held, 0))
    for b in range(B):
        s = src[b]
        if s < 0 or bad[b]:
            continue
        length[b] = int(kv_len[s])
        rows[b] = [int(x) for x in table[s, : run[s] if keeper[s] == b else length[b] // P]]
        for p in rows[b]:
            refs[p] += 1
    free = [p for p in range(n_pages) if refs[p] == 0]
    asked = 0
    for b in range(B):
        s = src[b]
        if s < 0 or bad[b]:
            continue
        copy = keeper[s] != b and length[b] % P != 0
        want = -(-(length[b] + need[b]) // P)
        n = max(want - len(rows[b]), 1 if copy else 0) if want <= M else 0
        if want > M or (n and asked + n > len(free)):
            taken[b] = -1
            if copy:
                length[b] = length[b] // P * P
        else:
            new = free[asked: asked + n]
            if copy:
                copies.append((int(table[s, length[b] // P]), new[0], length[b] % P))
            for p in new:
                refs[p] += 1
            rows[b] += new
            taken[b] = n
        asked += n
    out = np.full((B, M), -1, np.int32)
    for b in range(B):
        out[b, : len(rows[b])] = rows[b]
    i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return out, i32(length), i32(refs), i32(taken), copies


def compact(table, n_pages, held=None):
    """(table, new_page, live, moves)."""
    ok = (table >= 0) & (table < n_pages)
    used = sorted(set(table[ok].tolist()) | (set() if held is None else set(np.flatnonzero(held > 0).tolist())))
    live = len(used)
    holes = [p for p in range(live) if p not in set(used)]
    new = np.full(n_pages, -1, np.int32)
    moves, k = [], 0
    for p in used:
        new[p] = p
        if p >= live:
            new[p] = holes[k]
            moves.append((p, holes[k]))
            k += 1
    return np.where(ok, new[np.clip(table, 0, n_pages - 1)], -1).astype(np.int32), new, live, moves
