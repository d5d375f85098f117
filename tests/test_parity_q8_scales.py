"""GPU parity of the paged tree attention where V's scales differ between the pages of
one head, against the definition in float64 with tolerances in terms of what a row sums
up (no term in the largest scale of the cache): a page that hardly counts for a row,
however large its scale, takes nothing from the others."""
import numpy as np
import pytest

import q8_ref as R
from test_parity_q8 import U, as_dtype, attend, attention_case

pytestmark = pytest.mark.gpu


def definition(c):
    """(out, tol), [B,N,Hq,D].

    With p the weights and w = p * (V scale) of the keys of pages, rounding may make of
    each output
      sum_j p_j |v_j| (e_j + r_j) + sum_j p_j e_j * sum_j p_j |v_j|
      + float32 sums over the keys: (2 keys + 64) 2^-24 sum_j p_j |v_j|
      + the output's own rounding, and in bf16 keys * 2^-26 * 448 * max_j w_j:
    e_j, the score's error: D products summed in float32, relative to sum |q||k|; the
    arguments of exp2, up to 2^7 in float32; in bf16, q to 2^-17 of the largest |q|.
    (A weight off by the factor e^e is off by less than 1.01 e for e < 0.01.)
    r_j, in bf16: 2^-9 + 2^-11 for a key of a page (f16, of which three planes cut off or
    round what is behind 2^-9), 2^-8 for a tree row.  The planes' least step is 2^-16, a
    weight is off by half of it at most, and the largest w is held as 2^9 at least."""
    q, N, scale, bf16 = c["q"], c["q"].shape[1], c["scale"], c["dtype"] == "bf16"
    B, _, Hq, D = q.shape
    Hkv, P = c["k_pages"].shape[1], c["k_pages"].shape[2]
    seen = R.sees(c["mask"], N)
    out, tol = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    for b in range(B):
        L = min(max(int(c["kv_len"][b]), 0), c["table"].shape[1] * P)
        for h in range(Hkv):
            kp = R.prefix(c["k_pages"], c["k_scale"], c["v_scale"], c["table"][b], L, h)
            vp = R.prefix(c["v_pages"], c["v_scale"], c["k_scale"], c["table"][b], L, h)
            ones = R.prefix(np.full_like(c["v_pages"], 0x38), c["v_scale"], c["k_scale"], c["table"][b], L, h)  # 0x38: 1
            vs, n = ones[:, 0], len(kp)
            k, v = np.concatenate([kp, c["k_tree"][b, :, h]]), np.concatenate([vp, c["v_tree"][b, :, h]])
            vis = np.concatenate([np.ones((N, n), bool), seen], 1)
            some = vis.any(1)
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = np.where(vis, q[b, :, g] @ k.T * scale, -np.inf)[some]
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                e = (D + 8) * U * (np.abs(q[b, :, g]) @ np.abs(k).T * scale)[some] + 8 * U * 128
                r = np.zeros(n + N)
                if bf16:
                    e = e + 2.0 ** -17 * np.abs(q).max() * np.abs(k).sum(1) * scale
                    r[:n], r[n:] = 2.0 ** -9 + 2.0 ** -11, 2.0 ** -8
                spread = p @ np.abs(v)
                out[b, some, g] = o = p @ v
                t = (p * (1.01 * e + r)) @ np.abs(v) + (p * 1.01 * e).sum(1, keepdims=True) * spread
                t = t + (2 * (n + N) + 64) * U * spread + (2.0 ** -8 if bf16 else U) * np.abs(o)
                if bf16 and n:
                    t = t + (n + N) * 2.0 ** -26 * 448 * (p[:, :n] * vs).max(1, keepdims=True)
                tol[b, some, g] = t
    return out, tol


def check(c, got):
    out, tol = definition(c)
    over = np.abs(got - out) - tol
    assert np.isfinite(got).all() and over.max() <= 0, (over.max(), np.abs(got - out).max(), np.abs(out).max())


SHAPES = [(1, 4, 2, 64, 16), (20, 2, 2, 128, 32), (64, 1, 1, 64, 64), (90, 2, 1, 128, 16), (200, 1, 1, 64, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("r", [0, 12, 20, 28, 60])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", SHAPES)
def test_a_page_that_hardly_counts_takes_nothing_from_the_others(medusa, N, Hq, Hkv, D, P, r, dtype):
    """One page of V scale 2^r, first, in the middle or last, with scores so far below
    the others that its share of the output is under 2^-30."""
    rng = np.random.default_rng(N + r)
    c = attention_case(60 + N, 3, N, Hq, Hkv, D, P, [700, 645, 390], dtype)
    base = rng.normal(0, 1, D)
    c["q"] = as_dtype(base + 0.2 * c["q"], dtype)
    # K of that page: -a * base, scores of about -a |base|^2 / sqrt(D) (the spread of the others is under 10)
    a = (30 + 0.7 * (r + 30)) / (base @ base * c["scale"])
    ks = R.page_scale(a * np.abs(base))
    for b, j in enumerate((0, 190 // P, 389 // P)):
        p = c["table"][b, j]
        c["k_pages"][p], c["k_scale"][p] = R.encode(np.broadcast_to(-a * base / ks, c["k_pages"][p].shape)), ks
        c["v_scale"][p] = 2.0 ** r
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", SHAPES)
@pytest.mark.parametrize("spread", [8, 32])
def test_scales_that_jump_from_page_to_page(medusa, N, Hq, Hkv, D, P, spread, dtype):
    """V scales of every head and page anywhere in [2^-spread, 2^spread]."""
    c = attention_case(70 + N, 2, N, Hq, Hkv, D, P, [900, 333], dtype)
    c["v_scale"] *= np.exp2(np.random.default_rng(N).integers(-spread, spread + 1, c["v_scale"].shape)).astype(np.float32)
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", SHAPES)
def test_pages_of_zeros(medusa, N, Hq, Hkv, D, P, dtype):
    """V rows that are all zero, under the smallest scale, as the append writes them: in
    front, between others, and in every page of one sequence."""
    c = attention_case(80 + N, 3, N, Hq, Hkv, D, P, [700, 650, 200], dtype)
    for b, pages in enumerate((range(0, -(-300 // P)), range(1, 650 // P, 2), range(-(-200 // P)))):
        for j in pages:
            c["v_pages"][c["table"][b, j]], c["v_scale"][c["table"][b, j]] = 0, 2.0 ** -64
    check(c, attend(medusa, c))


@pytest.mark.parametrize("N,Hq,Hkv,D,P", SHAPES)
def test_weights_of_pages_have_nine_bits(medusa, N, Hq, Hkv, D, P):
    """No tree row is seen: what rounds are the weights of the pages and the output."""
    c = attention_case(90 + N, 2, N, Hq, Hkv, D, P, [700, 77], "bf16")
    c["mask"][:] = 0
    check(c, attend(medusa, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,P", SHAPES)
def test_scales_over_the_whole_readable_range(medusa, N, Hq, Hkv, D, P, dtype):
    """All pages of a sequence at one end of what a scale may be, the sequences apart."""
    c = attention_case(100 + N, 2, N, Hq, Hkv, D, P, [500, 345], dtype)
    c["mask"][:] = 0
    for b, s in enumerate((2.0 ** 64, 2.0 ** -64)):
        c["v_scale"][c["table"][b][c["table"][b] >= 0]] = s
    check(c, attend(medusa, c))
