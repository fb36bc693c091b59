"""fp64 CPU oracle of the cache calls -- test infrastructure only: the rotation with the page
write, the 4-bit values and attention over pages, written from their definitions in
``include/specdec.h``, one sequence, one head and one slot at a time where that is affordable."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    """The values of E4M3 bytes 0..126 (byte 127 is NaN): subnormals m * 2^-9, then (1 + m/8) 2^(e-7)."""
    return np.array([(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def to_e4m3(x: float) -> int:
    """The byte of the nearest E4M3 value of x >= 0, ties to the even byte, saturated at 448."""
    v = e4m3_values()
    d = np.abs(v - min(float(x), 448.0))
    near = np.flatnonzero(d == d.min())
    return int(near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1])


def quantise_group(x, tensor_scale: float):
    """Codes (16) and scale byte of 16 values: divisions and the product in fp32, as defined."""
    y = np.asarray(x, np.float32) * (np.float32(1.0) / np.float32(tensor_scale))
    if not np.isfinite(y).all():
        return np.zeros(16, np.uint8), 127
    byte = to_e4m3(float(np.abs(y).max() / np.float32(6.0)))
    s = np.float32(e4m3_values()[byte])
    codes = np.zeros(16, np.uint8)
    if s > 0:
        for i, v in enumerate(y):
            t = float(np.float32(v) / s)
            d = np.abs(E2M1 - min(abs(t), 6.0))
            near = np.flatnonzero(d == d.min())
            codes[i] = (near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]) + (8 if np.signbit(t) else 0)
    return codes, byte


def dequantise(codes, scales, tensor_scale: float) -> np.ndarray:
    """Rows of packed codes [..., D/2] and scale bytes [..., D/16] as float64 values [..., D]."""
    codes, scales = np.asarray(codes), np.asarray(scales).astype(int)
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    table = np.concatenate((e4m3_values(), [np.nan]))
    s = np.where(scales & 128, -1.0, 1.0) * table[scales & 127]
    return v * np.repeat(s, 16, -1) * np.float32(tensor_scale)


def rotate(x, pos: int, inv_freq, weight=None, eps: float = 1e-6, interleaved: bool = False):
    """One head's vector, normed (weight given) and rotated."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean() + eps) * np.asarray(weight, np.float64)
    y = x.copy()
    half = len(inv_freq)
    for j, f in enumerate(inv_freq):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        t = np.longdouble(pos) * np.longdouble(f)
        c, s = float(np.cos(t)), float(np.sin(t))
        y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y


def visible(n: int, nq: int, length: int, window: int, sinks: int, tree_mask=None, depth=None) -> np.ndarray:
    """[n, length] bool: whether query i sees slot s (queries past nq see nothing)."""
    P = length - nq
    sees = np.zeros((n, length), bool)
    for i in range(nq):
        pi = P + (i if depth is None else int(depth[i]))
        for s in range(length):
            j = s - P
            ok = j <= i if tree_mask is None else (j < 0 or bool(tree_mask[i][j]))
            ps = s if j < 0 or depth is None else P + int(depth[j])
            if window > 0:
                ok = ok and (pi - ps < window or ps < sinks)
            sees[i, s] = ok
    return sees


def attend(q, k, v, sees, scale: float):
    """One sequence: q [n, Hq, D], k and v [L, Hkv, D] float64, sees [n, L].  Returns out, lse and
    what the tolerances are made of: sum p |v| and sum of visible |v| per output element, and the
    largest sum |q_d k_d| of a row's visible slots."""
    n, hq, D = q.shape
    G = hq // k.shape[1]
    out, lse = np.zeros((n, hq, D)), np.full((n, hq), -np.inf)
    pv, av, qk = np.zeros((n, hq, D)), np.zeros((n, hq, D)), np.zeros((n, hq))
    for i in range(n):
        idx = np.flatnonzero(sees[i])
        if not len(idx):
            continue
        for h in range(hq):
            kk, vv = k[idx, h // G], v[idx, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                s = (kk @ q[i, h]) * scale
                m = s.max()
                e = np.exp(s - m)
                lse[i, h] = m + np.log(e.sum())
                p = e / e.sum()
                out[i, h] = p @ vv
                pv[i, h], av[i, h] = p @ np.abs(vv), np.abs(vv).sum(0)
                qk[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, pv, av, qk
