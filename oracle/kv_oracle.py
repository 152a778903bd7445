"""float64 oracle of the caller's paged cache: rotary positions, 4-bit storage, attention over a
request's keys, the accepted path.  Plain numpy, request by request; shares no code with the
library."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x):
    """Values rounded to bf16 (nearest, ties to even), as float64."""
    f = np.ascontiguousarray(np.asarray(x, np.float32))
    u = f.view(np.uint32).astype(np.uint64)
    r = (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(f), np.nan, r).astype(np.float64)


def e4m3_grid():
    g = []
    for e in range(16):
        for m in range(8):
            if e == 15 and m == 7:
                continue   # NaN
            g.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(g)


E4M3 = e4m3_grid()   # index = code


def nearest(x, grid):
    """Index of the nearest grid value of x >= 0 (ascending grid; ties to the even index)."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(x >= grid[-1], len(grid) - 1, pick)


def rotary(x, positions, inv_freq, interleaved=False, amplitude=1.0):
    """x [N, H, hd] float64; inv_freq [rot / 2]."""
    x = np.array(x, np.float64)
    y = x.copy()
    w = np.asarray(inv_freq, np.float64)
    half = len(w)
    ang = np.asarray(positions, np.float64)[:, None] * w[None, :]
    c, s = amplitude * np.cos(ang)[:, None, :], amplitude * np.sin(ang)[:, None, :]
    a = np.arange(half) * (2 if interleaved else 1)
    b = a + (1 if interleaved else half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise(x, glob):
    """bf16 values [..., hd] -> (codes [..., hd], scale codes [..., hd / 16], the values they
    stand for)."""
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    sc = nearest(np.minimum(np.abs(g).max(-1) / (6.0 * glob), 448.0), E4M3)
    unit = (E4M3[sc] * glob)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        mag = np.where(unit > 0, np.abs(g) / unit, 0.0)
    code = nearest(np.minimum(mag, 6.0), E2M1)
    val = np.copysign(E2M1[code] * unit, g)
    code = code + 8 * (np.signbit(g) & (unit > 0))
    return code.reshape(x.shape), sc, val.reshape(x.shape)


def attention(q, K, V, see, scale):
    """One request: q [R, Hq, hd], K / V [L, Hkv, hd], see [R, L] bool.  Returns out, lse, and for
    error bounds per (row, head): sum p |v| / sum p, the largest seen sum |q k| scale, sum |v|."""
    R, Hq, hd = q.shape
    G = Hq // K.shape[1]
    out = np.zeros((R, Hq, hd))
    lse = np.full((R, Hq), -np.inf)
    mag = np.zeros((R, Hq, hd))
    qk = np.zeros((R, Hq))
    vsum = np.zeros((R, Hq, hd))
    for i in range(R):
        idx = np.nonzero(see[i])[0]
        if len(idx) == 0:
            continue
        for h in range(Hq):
            k, v = K[idx, h // G], V[idx, h // G]
            s = k @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            out[i, h] = p @ v / p.sum()
            lse[i, h] = m + np.log(p.sum())
            mag[i, h] = p @ np.abs(v) / p.sum()
            vsum[i, h] = np.abs(v).sum(0)
            qk[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * scale
    return out, lse, mag, qk, vsum
