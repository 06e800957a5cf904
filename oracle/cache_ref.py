"""Float64 oracle of the cache side of a verify cycle: rotary embedding with the append to a
paged cache, and the attention of the new tokens over it. Plain NumPy, one sequence, one token
and one head at a time, in the order the operators are stated; it shares no code with the CUDA
path.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np


def frequencies(R, theta, scaling=None, factor=1.0, trained=8192.0, low=1.0, high=4.0):
    """(frequencies [R/2], magnitude) of the rotary embedding, stated per pair."""
    out = []
    for i in range(R // 2):
        base = theta * factor ** (R / (R - 2)) if scaling == "ntk" else theta
        f = base ** (-2.0 * i / R)
        turns = trained * f / (2 * math.pi)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            def index(t):  # where a pair makes t turns in the trained context
                return R * math.log(trained / (t * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), R - 1)
            g = min(max((i - a) / (b - a if b > a else 0.001), 0.0), 1.0)
            f = f * (1 - g) + f / factor * g
        elif scaling == "bands":
            g = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = f * g + f / factor * (1 - g)
        out.append(f)
    return np.array(out), 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0


def rotate(x, pos, inv_freq, interleaved=False, magnitude=1.0):
    """x [heads, D] at position pos; inv_freq [R/2]. Returns (y, |x1| + |x2| per element, 0 where
    the element is only copied)."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.zeros_like(x)
    R = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a = pos * float(f)
        c, s = magnitude * math.cos(a), magnitude * math.sin(a)
        d1, d2 = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y[:, d1] = x[:, d1] * c - x[:, d2] * s
        y[:, d2] = x[:, d2] * c + x[:, d1] * s
        size[:, d1] = size[:, d2] = abs(magnitude) * (np.abs(x[:, d1]) + np.abs(x[:, d2]))
    return y, size


def gather(pages, table_row, L):
    """The L cached rows [L, heads, D] of a sequence, page by page; NaN where the page id is out
    of range."""
    n_pages, ps = pages.shape[0], pages.shape[1]
    out = np.full((L,) + pages.shape[2:], np.nan)
    for t in range(L):
        page = int(table_row[t // ps])
        if 0 <= page < n_pages:
            out[t] = pages[page, t % ps]
    return out


@dataclass
class Attended:
    out: np.ndarray     # [n, Hq, D]
    lse: np.ndarray     # [n, Hq]
    wabs: np.ndarray    # [n, Hq, D]: sum of w |v|, what a relative error of the weights scales
    qk: np.ndarray      # [n, Hq]: the largest sum of |q| |k| over the seen positions, scaled
    seen: np.ndarray    # [n]: how many positions the token sees


def attend(q, K, V, n, scale, causal=True, window=None):
    """q [n, Hq, D] over K, V [L, Hkv, D]: new token i sits at position L - n + i."""
    L, Hkv, D = K.shape
    Hq = q.shape[1]
    r = Attended(np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D)),
                 np.zeros((n, Hq)), np.zeros(n, dtype=np.int64))
    for i in range(n):
        p = L - n + i
        lo = 0 if window is None else max(0, p - window + 1)
        hi = min(L, p + 1) if causal else L
        r.seen[i] = max(0, hi - lo)
        if hi <= lo:
            continue
        for h in range(Hq):
            k, v = K[lo:hi, h // (Hq // Hkv)], V[lo:hi, h // (Hq // Hkv)]
            z = scale * (k @ q[i, h])
            m = z.max()
            e = np.exp(z - m)
            w = e / e.sum()
            r.out[i, h] = w @ v
            r.lse[i, h] = m + math.log(e.sum()) if np.isfinite(m) else np.nan
            r.wabs[i, h] = w @ np.abs(v)
            r.qk[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return r
