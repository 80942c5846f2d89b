"""fp64 oracle of attention over positions, and of the quantised cache (TEST INFRASTRUCTURE ONLY).

Plain numpy from the definitions; the CUDA library shares nothing with it.

  attend       one head's rows at given positions: causal, optionally a sliding window whose first
               keys (sinks) stay visible; also returns what bounds a kernel's rounding
  attend_paged the new tokens of every sequence over its paged cache
  quantise     a row's power-of-two scale and E4M3 values
"""
from collections import namedtuple

import numpy as np

Rows = namedtuple("Rows", ["o", "lse", "pv", "v", "score", "top"])
Rows.__doc__ = """Per query row: o [n, d], lse [n], and the sizes a rounding bound is made of:
pv [n, d] = sum_j p_j |v_j|, v [n, d] = sum of |v_j| over the visible keys, score [n] = the largest
scale * sum_c |q_c k_jc| over them, top [n] = the largest weight p_j."""


def visible(pos, n_keys, window=-1, sinks=0):
    """[rows, keys] mask of what the rows at positions pos see."""
    p = np.asarray(pos, dtype=np.int64)[:, None]
    j = np.arange(n_keys, dtype=np.int64)[None, :]
    m = j <= p
    if window >= 0:
        m &= (p - j <= window) | (j < sinks)
    return m


def attend(q, k, v, pos, scale, window=-1, sinks=0):
    """Rows of one head: q [n, d] at cache positions pos [n] over k, v [L, d] (float64).  A row that
    sees no key has o = 0 and lse = -inf.  Keys no row sees do not enter, whatever they hold."""
    n, d = q.shape
    vis = visible(pos, len(k), window, sinks)
    used = vis.any(axis=0)
    k = np.where(used[:, None], k, 0.0)
    v = np.where(used[:, None], v, 0.0)
    s = np.where(vis, scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    live = np.isfinite(m)
    e = np.where(vis, np.exp(s - np.where(live, m, 0.0)[:, None]), 0.0)
    l = e.sum(axis=1)
    p = e / np.where(l > 0, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(live, m + np.log(l), -np.inf)
    size = np.where(vis, scale * (np.abs(q) @ np.abs(k).T), 0.0).max(axis=1, initial=0.0)
    return Rows(p @ v, lse, p @ np.abs(v), vis.astype(np.float64) @ np.abs(v), size,
                p.max(axis=1, initial=0.0))


def attend_paged(q, cu_q, seqs_k, seqs_v, scale, window=-1, sinks=0):
    """q [T, Hq, d] packed new tokens (float64), seqs_k[b], seqs_v[b] [L_b, Hkv, d]: the tokens of
    sequence b's cache in order.  Returns Rows with arrays [T, Hq, ...]; rows outside the packed
    sequences are NaN."""
    T, Hq, d = q.shape
    out = Rows(*(np.full(s, np.nan) for s in ((T, Hq, d), (T, Hq), (T, Hq, d), (T, Hq, d), (T, Hq),
                                              (T, Hq))))
    for b, (k, v) in enumerate(zip(seqs_k, seqs_v)):
        r = slice(int(cu_q[b]), int(cu_q[b + 1]))
        n = r.stop - r.start
        if n == 0:
            continue
        G = Hq // k.shape[1]
        pos = np.arange(n) + len(k) - n
        for h in range(Hq):
            x = attend(q[r, h], k[:, h // G], v[:, h // G], pos, scale, window, sinks)
            for dst, src in zip(out, x):
                dst[r, h] = src
    return out


def row_tolerance(rows, eps_p, eps_o, tiny_p, extra_score=0.0):
    """(elements, lse) bounds of a kernel that rounds the weights to a type of spacing eps_p at 1
    (subnormal spacing tiny_p) before the second product and o to one of spacing eps_o, everything
    else in fp32.

    Scores: a sum of d fp32 products and its scaling, off by at most 2^-20 of sum |q_c k_c| (d = 128
    terms of 2^-24 each would be 2^-17 if all went the same way; the tensor cores add in blocks),
    plus extra_score.  A score off by t moves every p_j and l by a factor within e^(2t).  Weights:
    half a step, eps_p / 2 relative or tiny_p / 2 absolute; relative to the running maximum, which
    the largest weight is at least.  o: half a step.  exp2, sums and the division: 2^-17 together.

    Where the scores' error says nothing about the weights (e^(2t) past float64) the bound is infinite,
    of values that have no weight at all too."""
    t = 2.0 ** -20 * rows.score + extra_score
    with np.errstate(over="ignore", invalid="ignore"):
        rel = np.expm1(2.0 * t)[..., None] + 0.5 * eps_p + 2.0 ** -17
        moved = np.where(np.isposinf(rel), np.inf, rel * rows.pv)
    el = moved + 0.5 * tiny_p * rows.top[..., None] * rows.v
    el = el + 0.5 * eps_o * (np.abs(rows.o) + el) + 2.0 ** -25  # half an fp16 subnormal step
    lse = 2.0 * t + 2.0 ** -18 + 2.0 ** -21 * np.abs(np.where(np.isfinite(rows.lse), rows.lse, 0.0))
    return el, lse


def check(o, lse, rows, tol, what=""):
    """Asserts o and lse lie within tol = row_tolerance(...) of the oracle's rows; rows without keys
    exactly 0 and -inf."""
    o, lse = np.asarray(o, dtype=np.float64), np.asarray(lse, dtype=np.float64)
    empty = np.isneginf(rows.lse)
    assert np.all(lse[empty] == -np.inf) and np.all(o[empty] == 0.0), f"{what}: rows without keys"
    live = ~empty
    for name, got, ref, lim in (("o", o[live], rows.o[live], tol[0][live]),
                                ("lse", lse[live], rows.lse[live], tol[1][live])):
        assert np.all(np.isfinite(got)), f"{what}: non-finite {name}"
        assert not np.any(np.isnan(lim)), f"{what}: a tolerance of {name} that is not a number"
        r = np.abs(got - ref) / lim
        if not np.all(r <= 1.0):
            at = np.unravel_index(int(np.argmax(r)), r.shape)
            raise AssertionError(f"{what}: {name} at {tuple(map(int, at))} of the live rows: "
                                 f"{got[at]!r} for {ref[at]!r}, {r[at]:.2f} times the tolerance "
                                 f"({int((r > 1).sum())} values)")


def e4m3_values():
    """The 127 finite non-negative E4M3 values in order of their codes."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    return np.array((sub + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:-1])


def quantise(x):
    """x [..., d] float64 -> (scale [...], values [..., d]): the scale 2^e, e the smallest integer
    >= -126 with max |x| <= 448 * 2^e over the finite values (0 for none or zero), and the E4M3 value
    nearest to x / scale, ties to the even code; NaN for a value that is not finite."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0).max(axis=-1)
    e = np.zeros(a.shape, dtype=np.int64)
    for i in np.ndindex(a.shape):
        if a[i] > 0:
            n = -126
            while a[i] > 448.0 * 2.0 ** n:
                n += 1
            e[i] = n
    scale = 2.0 ** e.astype(np.float64)
    grid = e4m3_values()
    y = np.where(fine, np.abs(x), 0.0) / scale[..., None]
    hi = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    up, down = grid[hi] - y, y - grid[hi - 1]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    val = np.where(take_hi, grid[hi], grid[hi - 1]) * np.where(x < 0, -1.0, 1.0)
    return scale, np.where(fine, val, np.nan)
