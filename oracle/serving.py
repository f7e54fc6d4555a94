"""Oracle for the serving operators (fp64, CPU): rotary positions in every
layout and scaling, rows of the 8-bit cache, attention of draft trees.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Formulas as the C
header states them; each function is the plain definition.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
KV_MAX = {"e4m3": 448.0, "i8": 127.0}


def rope_frequencies(rot_dim, theta=5e5, factor=1.0, low=0.0, high=0.0, original=0):
    """Radians per position of each pair."""
    f = float(theta) ** (-2.0 * np.arange(rot_dim // 2) / rot_dim)
    if factor == 1.0:
        return f
    if original == 0:
        return f / factor
    r = original * f / (2.0 * np.pi)
    g = np.clip((r - low) / (high - low), 0.0, 1.0)
    return f * (g + (1.0 - g) / factor)


def rope(x, positions, rot_dim, layout="half", amplitude=1.0, **scaling):
    """x [T][n][head_dim] (float64) rotated by positions [T]."""
    out = np.array(x, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * rope_frequencies(rot_dim, **scaling)
    c, s = np.cos(ang)[:, None] * amplitude, np.sin(ang)[:, None] * amplitude
    h = rot_dim // 2
    ia, ib = (np.arange(h), np.arange(h) + h) if layout == "half" else \
        (2 * np.arange(h), 2 * np.arange(h) + 1)
    a, b = out[..., ia], out[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def _e4m3_grid():
    """The non-negative e4m3 numbers in order, code 0 .. 126."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


def kv_encode(x, kind):
    """(codes, scale bytes) of rows x [..., 128] (float64): the smallest power
    of two >= 2^-124 that the block's largest magnitude does not overflow, the
    nearest code, ties to the even one.  Codes are e4m3 bit patterns (uint8)
    or int8."""
    b = np.asarray(x, dtype=np.float64).reshape(*np.shape(x)[:-1], np.shape(x)[-1] // BLOCK, BLOCK)
    top = np.max(np.abs(b), axis=-1)
    bad = ~np.isfinite(top)
    e = np.full(top.shape, -124)
    safe = np.where(bad | (top == 0), 1.0, top)
    for cand in range(-123, 129):              # the definition: try every scale
        e = np.where(safe > KV_MAX[kind] * 2.0 ** (cand - 1), cand, e)
    y = np.where(bad[..., None], 0.0, b) * 2.0 ** (-e[..., None].astype(float))
    if kind == "i8":
        codes = np.rint(y).astype(np.int8)
    else:
        grid = _e4m3_grid()
        mag = np.abs(y)
        hi = np.clip(np.searchsorted(grid, mag), 0, 126)
        lo = np.maximum(hi - 1, 0)
        up, down = grid[hi] - mag, mag - grid[lo]
        code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        codes = (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)
    byte = np.where(bad, 255, np.where(top == 0, 0, e + 127)).astype(np.uint8)
    return codes.reshape(np.shape(x)), byte


def kv_decode(codes, byte, kind):
    """The numbers that codes and scale bytes stand for (float64)."""
    if kind == "i8":
        v = codes.astype(np.float64)
    else:
        c = codes.astype(np.int64)
        v = np.append(_e4m3_grid(), np.nan)[c & 127] * np.where(c & 128, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127.0))
    return (v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK) * s[..., None]).reshape(v.shape)


def tree_matrix(words, n):
    """Mask words [..., ceil(n / 32)] (uint32) as truth values [..., n]."""
    i = np.arange(n)
    return ((words[..., i // 32] >> (i % 32).astype(np.uint32)) & 1).astype(bool)


def attn_tree(q, k, v, cache_len, draft_len, tree, heads, scale, out):
    """Attention of draft trees.  q [S][N][n_q][d], k and v [S][n_kv][cap][d]
    (float64), tree [S][N][N] and heads [S][N][n_kv] truth values; fills `out`
    [S][N][n_q][d] where there are tokens and returns (out, spread) with
    spread = sum_p weight_p |v_p| and reach = sum_d |q_d k_d| maximal over p,
    the magnitudes an error bound needs."""
    S, N, n_q, _ = q.shape
    rep = n_q // k.shape[1]
    spread, reach = np.zeros_like(out), np.zeros(out.shape[:3])
    for s in range(S):
        c, m = int(cache_len[s]), int(draft_len[s])
        for t in range(m):
            see = np.concatenate([np.ones(c, bool), tree[s, t, :m]])
            at = np.flatnonzero(see)
            for h in range(n_q):
                j = h // rep
                out[s, t, h] = 0.0
                if not heads[s, t, j] or len(at) == 0:
                    continue
                kk, vv = k[s, j, at], v[s, j, at]
                x = scale * (kk @ q[s, t, h])
                w = np.exp(x - np.max(x))
                w /= np.sum(w)
                out[s, t, h] = w @ vv
                spread[s, t, h] = w @ np.abs(vv)
                reach[s, t, h] = scale * np.max(np.abs(kk) @ np.abs(q[s, t, h]))
    return out, spread, reach
