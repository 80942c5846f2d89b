"""fp64 oracle of the page lists and of the 4-bit cache (TEST INFRASTRUCTURE ONLY).

Plain Python and numpy from the definitions; the CUDA library shares nothing with it.

  Lists     a block table, lengths and a free list, extended and trimmed token by token
  quantise  what the cache holds of 16-bit rows: codes, scale bytes and values
  values    the values that codes and scale bytes stand for
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# five exponent and three mantissa bits; the last 8 of the 256 (fp16's infinity and NaNs) are left out
E5M3 = np.array([m * 2.0 ** -17 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)])
MAX_SCALE = int(np.searchsorted(E5M3, 10240.0))
NAN_SCALE = 255


class Lists:
    """table: a list of pages per sequence; free: the stack, its top last."""

    def __init__(self, B, free, page):
        self.table, self.len = [[] for _ in range(B)], [0] * B
        self.free, self.page = list(free), page

    def extend(self, n):
        """Slots of the n[b] new tokens of each sequence, packed; None where the list is too short."""
        need = sum(-(-(L + x) // self.page) - -(-L // self.page) for L, x in zip(self.len, n))
        if need > len(self.free):
            return None
        slots = []
        for b, x in enumerate(n):
            for t in range(self.len[b], self.len[b] + x):
                if t % self.page == 0:
                    self.table[b].append(self.free.pop())
                slots.append(self.table[b][t // self.page] * self.page + t % self.page)
            self.len[b] += x
        return slots

    def trim(self, keep):
        for b in reversed(range(len(keep))):
            while len(self.table[b]) > -(-keep[b] // self.page):
                self.free.append(self.table[b].pop())
            self.len[b] = keep[b]


def nearest(x, grid):
    """Places in the ascending grid of the values nearest to x >= 0, the even one of two as near."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    up, down = grid[hi] - x, x - grid[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x):
    """x [..., d] float64 -> (codes [..., d/2], scale bytes [..., d/16], values [..., d])."""
    x = np.asarray(x, dtype=np.float64)
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    fine = np.isfinite(y).all(-1)
    a = np.where(fine, np.abs(np.where(np.isfinite(y), y, 0.0)).max(-1), 0.0)
    by = np.minimum(nearest(a / 6.0, E5M3), MAX_SCALE)
    by = np.where((a > 0) & (by == 0), 1, by)
    f = E5M3[by][..., None]
    code = nearest(np.where(fine[..., None], np.abs(y), 0.0) / np.where(f > 0, f, 1.0), E2M1)
    val = np.where(y < 0, -1.0, 1.0) * E2M1[code] * f
    # a zero of either sign, a zero block and one that is not finite hold codes of 0
    code = np.where((by == 0)[..., None] | ~fine[..., None], 0, code + 8 * (y < 0))
    code = code.reshape(x.shape)
    return ((code[..., 0::2] + 16 * code[..., 1::2]).astype(np.uint8),
            np.where(fine, by, NAN_SCALE).astype(np.uint8),
            np.where(fine[..., None], val, np.nan).reshape(x.shape))


def values(codes, scales):
    """[..., d/2] codes and [..., d/16] scale bytes -> [..., d] float64."""
    codes, scales = np.asarray(codes).astype(np.int64), np.asarray(scales).astype(np.int64)
    v = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(v & 8, -1.0, 1.0) * E2M1[v & 7]
    f = np.where(scales == NAN_SCALE, np.nan, E5M3[np.minimum(scales, len(E5M3) - 1)])
    return v * np.repeat(f, 16, axis=-1)
