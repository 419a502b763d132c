"""Plain 64-bit statement of the paged 8-bit cache and of the prompt attention, for the tests.

Nothing here shares code with the kernels: numpy and Python lists, one token, block or row
at a time.
"""

import math

import numpy as np
import torch

TOP = {"int8": 127.0, "e4m3": 448.0}
# half a step of each 16-bit type, relative to the value
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def e4m3(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even) of float64 values of magnitude <= 448 (1 + 2^-20)."""
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def block_values(x: np.ndarray, fmt: str) -> np.ndarray:
    """Values one block of one head stands for, binary32; x [tokens][d] float64."""
    if not np.isfinite(x).all():
        return np.full(x.shape, np.nan, np.float32)
    amax = np.float32(np.abs(x).max())
    scale = np.float32(1.0) if amax == 0 else max(np.float32(amax / np.float32(TOP[fmt])), np.float32(2.0 ** -126))
    y = (x.astype(np.float32) / scale).astype(np.float64)  # the quotient is binary32
    q = np.clip(np.rint(y), -127, 127) if fmt == "int8" else e4m3(y)
    return q.astype(np.float32) * scale


def cached_values(x: np.ndarray, bt: int, fmt: str) -> np.ndarray:
    """What the cache holds of one request: x [tokens][heads][d] float64 -> binary32."""
    out = x.astype(np.float32)
    for b in range(x.shape[0] // bt):
        for h in range(x.shape[1]):
            out[b * bt:(b + 1) * bt, h] = block_values(x[b * bt:(b + 1) * bt, h], fmt)
    return out


class Tables:
    """The request state as Python lists."""

    def __init__(self, n_blocks, bt, n_requests):
        self.bt, self.lens = bt, [0] * n_requests
        self.free = list(range(n_blocks - 1, -1, -1))
        self.rows = [[] for _ in range(n_requests)]

    def step(self, new):
        """(q_start, positions, slots) of a step; the state moves on."""
        for i, n in enumerate(new):
            if n < 0:
                self.free += self.rows[i]
                self.rows[i], self.lens[i] = [], 0
        q_start, positions, slots = [0], [], []
        for i, n in enumerate(new):
            n = max(n, 0)
            after = self.lens[i] + n
            while len(self.rows[i]) < after // self.bt:
                self.rows[i].append(self.free.pop())
            for p in range(self.lens[i], after):
                positions.append(p)
                slots.append(self.slot(i, p, after))
            self.lens[i] = after
            q_start.append(q_start[-1] + n)
        return q_start, positions, slots

    def slot(self, i, p, n):
        bt = self.bt
        return self.rows[i][p // bt] * bt + p % bt if p // bt < n // bt else -1 - (i * bt + p % bt)


def attention(q, k, v, scale, see=None):
    """Rows of softmax attention in float64: q [n][d], k, v [m][d]; row i sees the first see[i]
    keys (None: all). Returns out, lse and two error scales per row: the weighted mean of |v|
    and the sum of |q_c k_c| of the worst key (what binary32 accumulation rounds)."""
    n, m = q.shape[0], k.shape[0]
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    mean_abs, worst = np.zeros((n, v.shape[1])), np.zeros(n)
    for i in range(n):
        j = m if see is None else min(max(see[i], 0), m)
        if j == 0:
            continue
        s = (k[:j] @ q[i]) * scale
        top = s.max()
        p = np.exp(s - top)
        lse[i] = top + math.log(p.sum())
        p /= p.sum()
        out[i], mean_abs[i] = p @ v[:j], p @ np.abs(v[:j])
        worst[i] = (np.abs(k[:j]) @ np.abs(q[i])).max() * abs(scale)
    return out, lse, mean_abs, worst


def tolerance(out, mean_abs, worst, dtype, weight_step):
    """Bound of |kernel - exact| per entry.

    A score is a sum of d = 128 products in binary32 (any order, each addition off by at most
    2^-23 of the partial sums' magnitude): |ds| <= (128 + 8) 2^-23 sum|q_c k_c| with a few
    roundings for the scale. A weight is then off by ds, the exponential (2^-21) and its
    rounding to the 16-bit operand (weight_step), in numerator or denominator; outputs are
    rounded once to `dtype` (below 2^-14 binary16 is spaced 2^-24)."""
    ds = 136 * 2.0 ** -23 * worst[:, None]
    return mean_abs * (2 * ds + weight_step + 2.0 ** -19) + HALF_STEP[dtype] * np.abs(out) + 2.0 ** -24


def lse_tolerance(lse, worst):
    return 136 * 2.0 ** -23 * worst + 2.0 ** -19 + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
