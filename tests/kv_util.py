"""The 8-bit key/value cache and the attention over it, restated in 64 bits on the CPU for
the tests: the code's values from its definition, the quantiser by search over them, the
attention row by row. Nothing here calls the library."""
import math

import numpy as np
import torch

MIN_EXP, ZERO_EXP = -100, -60


def e4m3_values():
    """The 256 values of the code: sign, 4 bits of exponent (bias 7), 3 of fraction; two NaNs, no infinity."""
    v = np.empty(256)
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        x = math.nan if e == 15 and f == 7 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        v[b] = -x if b & 128 else x
    return v


VALUES = e4m3_values()


def quantise(x):
    """(codes uint8, exponent bytes uint8) of vectors x [..., D] (float64)."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, dtype=np.uint8)
    exps = np.zeros(x.shape[:-1], dtype=np.uint8)
    grid = VALUES[:127]
    for i in np.ndindex(exps.shape):
        m = np.abs(x[i]).max() if np.isfinite(x[i]).all() else math.inf
        if m == math.inf:
            exps[i] = 255
            continue
        e = ZERO_EXP
        if m > 0:
            e = MIN_EXP
            while m > 448 * 2.0 ** e:
                e += 1
        y = np.abs(x[i]) * 2.0 ** -e
        hi = np.clip(np.searchsorted(grid, y), 1, 126)
        down, up = y - grid[hi - 1], grid[hi] - y
        c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
        codes[i] = c + 128 * np.signbit(x[i])
        exps[i] = e + 127
    return codes, exps


def dequantise(codes, exps):
    codes, exps = np.asarray(codes), np.asarray(exps)
    scale = np.where(exps == 255, math.nan, 2.0 ** (exps.astype(np.float64) - 127))
    return VALUES[codes] * scale[..., None]


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def visible(rows, length, parent=None):
    """[rows, length] bool: what row i of a round of `rows` rows sees of its sequence's first `length` tokens."""
    out = np.zeros((rows, length), dtype=bool)
    ctx = length - rows
    for i in range(rows):
        anc = {i}
        if parent is None:
            anc = set(range(i + 1))
        else:
            j = i
            while j > 0:
                j = parent[j - 1] + 1
                anc.add(j)
            anc.add(0)
        for t in range(length):
            out[i, t] = t < ctx or (t - ctx) in anc
    return out


def attention(q, cache, table, kv_len, rows, *, parent=None, scale=None, prefix_table=None, prefix_len=0):
    """(o, lse, spread, dx) in float64. q [R, H, D] numpy; table, kv_len host arrays; rows: rows of
    each sequence. spread = sum_t p_t |v_t| per output, what roundings of the weights are relative
    to; dx = scale * max_t sum_d |q_d k_td| and scale * max|q| * max_t sum_d |k_td|, per (row, head),
    what errors of the scores are relative to."""
    R, H, D = q.shape
    kc, vc = raw(cache.k), raw(cache.v)
    ke, ve = raw(cache.k_exp), raw(cache.v_exp)
    _, Hk, S, _ = kc.shape
    G = H // Hk
    scale = D ** -0.5 if scale is None else scale
    o, spread = np.zeros((R, H, D)), np.zeros((R, H, D))
    lse = np.full((R, H), -math.inf)
    dx = np.zeros((2, R, H))

    def tokens(pages, n, h):
        pages = np.asarray(pages[:-(-n // S)], dtype=np.int64)
        k = dequantise(kc[pages, h], ke[pages, h]).reshape(-1, D)[:n]
        v = dequantise(vc[pages, h], ve[pages, h]).reshape(-1, D)[:n]
        return k, v

    for h in range(Hk):
        pk, pv = tokens(prefix_table, prefix_len, h) if prefix_len else (np.zeros((0, D)),) * 2
        r = 0
        for b, n_rows in enumerate(rows):
            n = int(kv_len[b])
            k, v = tokens(table[b], n, h)
            k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
            vis = np.concatenate([np.ones((n_rows, prefix_len), dtype=bool), visible(n_rows, n, parent)], axis=1)
            if k.shape[0]:
                qq = q[r:r + n_rows, h * G:(h + 1) * G].reshape(n_rows * G, D)
                s = (qq @ np.where(np.isnan(k), 0, k).T) * scale
                see = np.repeat(vis, G, axis=0)
                hurt = np.isnan(k).any(-1) | np.isnan(v).any(-1)
                s = np.where(see, s, -math.inf)
                m = s.max(-1, keepdims=True)
                m = np.where(m == -math.inf, 0, m)
                with np.errstate(invalid="ignore"):
                    p = np.exp(s - m)
                l = p.sum(-1, keepdims=True)
                with np.errstate(invalid="ignore", divide="ignore"):
                    w = np.where(l > 0, p / l, 0)
                    y = np.where(l > 0, m + np.log(l), -math.inf)[:, 0]
                clean = np.where(np.isnan(v), 0, v)
                a, sp = w @ clean, w @ np.abs(clean)
                dead = (see & hurt).any(-1) | ~np.isfinite(qq).all(-1) & see.any(-1)
                a[dead], y[dead] = math.nan, math.nan
                mk = np.abs(np.where(np.isnan(k), 0, k))
                dx[0, r:r + n_rows, h * G:(h + 1) * G] = (scale * (np.abs(qq) @ mk.T).max(-1)).reshape(n_rows, G)
                dx[1, r:r + n_rows, h * G:(h + 1) * G] = (scale * np.abs(qq).max(-1) * mk.sum(-1).max()).reshape(n_rows, G)
                o[r:r + n_rows, h * G:(h + 1) * G] = a.reshape(n_rows, G, D)
                spread[r:r + n_rows, h * G:(h + 1) * G] = sp.reshape(n_rows, G, D)
                lse[r:r + n_rows, h * G:(h + 1) * G] = y.reshape(n_rows, G)
            r += n_rows
    return o, lse, spread, dx


def bounds(o, spread, dx, dtype, tokens):
    """How far o and lse may be off, per element.

    bf16 queries: the weights are rounded to 16-bit floats (2^-11 of each), the scores' sums are in
    fp32 (2^-24 a step, 128 steps at most: 2^-17 of sum |q k|) over queries held to 2^-17 of their
    largest element, an exponent's error enters numerator and sum, the sums over the tokens are in
    fp32, and the output is rounded to bf16 (2^-8). fp32 queries: fp32 throughout."""
    u = 2.0 ** -24
    if dtype == torch.bfloat16:
        x = 2.0 ** -17 * (dx[0] + dx[1]) + 2.0 ** -20
        rel, out = 2.0 ** -11 + tokens * u, 2.0 ** -8
    else:
        x = 130 * u * dx[0] + 8 * u
        rel, out = (tokens + 16) * u, u
    spread = np.nan_to_num(spread)
    x = np.nan_to_num(x)
    return out * np.abs(o) + (rel + 2 * x)[..., None] * 1.01 * spread + 1e-30, 1.01 * x + (tokens + 16) * u


def compare(got, lse, ref, dtype, tokens):
    o, ref_lse, spread, dx = ref
    bo, bl = bounds(np.nan_to_num(o), spread, dx, dtype, tokens)
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(o)), "NaN rows differ"
    ok = ~np.isnan(o)
    off = np.abs(got - o)[ok]
    assert (off <= bo[ok]).all(), f"off by {off.max():.3g}, {(off / bo[ok]).max():.3g} of the bound"
    if lse is not None:
        lse = lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(lse), np.isnan(ref_lse)) and np.array_equal(lse == -math.inf, ref_lse == -math.inf)
        f = np.isfinite(ref_lse)
        d = np.abs(lse[f] - ref_lse[f])
        lim = bl[f] + 2.0 ** -23 * np.abs(ref_lse[f])
        assert (d <= lim).all(), f"lse off by {d.max():.3g}, {(d / lim).max():.3g} of the bound"


def pages_for(lens, page, rng, extra=2, first=0):
    """(table [B, width] int32, number of pages): each sequence's pages in any order of the pool; places past its end
    name a page outside the cache, which nothing may look at."""
    need = [-(-int(n) // page) for n in lens]
    total = sum(need) + extra + first
    perm = rng.permutation(np.arange(first, total)).astype(np.int32)
    table = np.full((len(need), max(1, max(need, default=1))), 1 << 30, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total
