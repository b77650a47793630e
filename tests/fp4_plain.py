"""The 4-bit cache's definitions in 64 bits (numpy), shared by its tests.

Nothing here uses the library: E2M1 and E4M3 are tables of their values, a
rounding picks the nearest value by exact comparison (ties to the even code),
attention is a plain softmax.
"""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16)
                                                       for m in range(8)][:-1])  # codes 0 .. 126
D, GROUP = 128, 16


def nearest(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Code of the value nearest to each x >= 0 (exact comparison of x with the middle of two neighbours)."""
    mid = (values[1:] + values[:-1]) / 2  # exact: few bits
    lo = np.searchsorted(mid, x, side="left")   # a tie goes down ...
    hi = np.searchsorted(mid, x, side="right")  # ... or up:
    return np.where(lo % 2 == 0, lo, hi)        # to the even code


def quantise(x: torch.Tensor, S: float):
    """(codes uint8 [.., 64], groups uint8 [.., 8], values float64 [.., 128]) of bf16 rows [.., 128]."""
    v = x.double().cpu().numpy()
    shape = v.shape
    v = v.reshape(-1, D // GROUP, GROUP)
    fine = np.isfinite(v).all(-1)
    top = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0)).max(-1), 0.0)
    byte = nearest(top / (6 * S), E4M3)
    s = E4M3[byte]
    use = fine & (s > 0)
    t = np.abs(np.where(use[..., None], v, 0)) / (np.where(use, s, 1.0) * S)[..., None]
    code = nearest(t, E2M1) + 8 * np.signbit(v)
    code = np.where(use[..., None], code, 0).astype(np.uint8).reshape(-1, D)
    group = np.where(fine, byte, 0x7F).astype(np.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    lead = shape[:-1]
    return (codes.reshape(*lead, D // 2), group.reshape(*lead, D // GROUP),
            values(codes, group, S).reshape(shape))


def values(codes: np.ndarray, groups: np.ndarray, S: float) -> np.ndarray:
    """The numbers that codes and group scales stand for, in 64 bits."""
    table = np.concatenate([E2M1, -E2M1])
    e4m3 = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    full = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D)
    return table[full] * np.repeat(e4m3[groups] * S, GROUP, -1)


def attend(q: torch.Tensor, k: np.ndarray, v: np.ndarray, entries: np.ndarray) -> np.ndarray:
    """softmax(q k / sqrt(d)) v of one row: q [H_q, 128], k and v [tokens, H_kv, 128] in 64 bits, over the entries that
    are not -1 (each as often as it stands there); zeros where there is none."""
    qd = q.double().cpu().numpy()
    H, K = qd.shape[0], k.shape[1]
    e = entries[entries >= 0]
    out = np.zeros((H, D))
    if len(e) == 0:
        return out
    for h in range(H):
        kv = h // (H // K)
        with np.errstate(all="ignore"):
            z = k[e, kv] @ qd[h] / np.sqrt(D)
            p = np.exp(z - z.max())
            out[h] = (p / p.sum()) @ v[e, kv]
    return out
