"""The 8-bit K/V cache and its attention from their definitions, in numpy: 64-bit
arithmetic, and binary32 where the cache's format prescribes it (scales, their
reciprocals and ratios, and the products that are rounded to codes: bf16 values
often lie exactly on a rounding border of the quotient, where only the same
products give the same code)."""
import numpy as np

PAGE = 16


def bf16(x):
    """Round to bf16 (nearest even); returns (bits uint16, value float64)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    bits = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return bits, (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rotate(x, pos, theta):
    """x [rows][heads][d] at positions pos [rows]; theta 0: as it is."""
    if not theta:
        return x
    h = x.shape[2] // 2
    a = np.asarray(pos, np.float64)[:, None] * theta ** (-np.arange(h) / h)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    return np.concatenate((x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s), -1)


class Cache:
    """One layer: codes [pages][heads][2][PAGE][d] as float64, scales [pages][heads][2] binary32."""

    def __init__(self, pages, heads, d, theta):
        self.codes = np.zeros((pages, heads, 2, PAGE, d))
        self.scales = np.zeros((pages, heads, 2), np.float32)
        self.theta = theta

    def append(self, pages, pos0, k, v):
        """k, v [n][heads][d]: one session's rows at pos0..; pages: its page ids."""
        n = k.shape[0]
        x = np.stack((rotate(k, pos0 + np.arange(n), self.theta), v), 2)  # [n][heads][2][d]
        for p in range(pos0 // PAGE, (pos0 + n - 1) // PAGE + 1 if n else 0):
            lo, hi = max(pos0, p * PAGE), min(pos0 + n, (p + 1) * PAGE)
            pg, first = pages[p], lo - p * PAGE
            new = x[lo - pos0:hi - pos0]
            s = (np.abs(new).max((0, 3)).astype(np.float32) / np.float32(127)).astype(np.float32)
            s[s < 2.0 ** -100] = 0
            old = self.scales[pg].copy() if first else np.zeros_like(s)
            s = np.maximum(s, old)
            with np.errstate(divide="ignore", invalid="ignore"):
                r = np.where(old > 0, old / s, np.float32(1))
                self.codes[pg, :, :, :first] = np.rint(self.codes[pg, :, :, :first].astype(np.float32) * r[..., None, None])
                inv = np.where(s > 0, np.float32(1) / s, np.float32(0))
                q = new.astype(np.float32) * inv[..., None]
            self.codes[pg, :, :, first:hi - p * PAGE] = np.clip(np.rint(q), -127, 127).transpose(1, 2, 0, 3)
            self.scales[pg] = s

    def values(self, pages, n):
        """(K, V) [n][heads][d] and the step (scale) of each value, of positions 0..n-1."""
        pg = np.asarray(pages[:(n + PAGE - 1) // PAGE], int)
        x = self.codes[pg] * self.scales[pg][..., None, None].astype(np.float64)
        x = x.transpose(2, 0, 3, 1, 4).reshape(2, -1, x.shape[1], x.shape[4])[:, :n]
        st = np.repeat(self.scales[pg], PAGE, 0)[:n].transpose(2, 0, 1)[..., None].astype(np.float64)
        return x[0], x[1], st[0], st[1]


def attention(q, k, v, pos0, scale, theta):
    """q [n][nq][d] at pos0.., k, v [pos0 + n][heads][d]: (out [n][nq][d], the
    rotated queries). Causal."""
    n, nq, d = q.shape
    group = nq // k.shape[1]
    q = rotate(q, pos0 + np.arange(n), theta)
    out = np.zeros_like(q)
    unseen = np.arange(k.shape[0])[None] > pos0 + np.arange(n)[:, None]
    for h in range(nq):
        x = q[:, h] @ k[:, h // group].T * scale
        x[unseen] = -np.inf
        p = np.exp(x - x.max(1, keepdims=True))
        out[:, h] = p @ np.where(np.isnan(v[:, h // group]), 0, v[:, h // group]) / p.sum(1, keepdims=True)
    return out, q
