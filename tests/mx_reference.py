"""Plain 64-bit implementations of the microscaled format and the expert
routing, written from their formulas in include/q4.h and sharing no code with
the library."""
from __future__ import annotations

import numpy as np
import torch

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
POWERS = np.array([2.0 ** (b - 127) for b in range(255)] + [np.nan])


def _up(n, m):
    return -(-n // m) * m


def scale_at(r, g):
    return (r % 32) * 16 + (r // 32) * 4 + g


def pack(w):
    """(codes [Nb, Kb, 128, 64], scales [Nb, Kb, 512]) of w [N, K]."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    Np, Kp = _up(N, 128), _up(K, 128)
    full = np.zeros((Np, Kp))
    full[:N, :K] = w
    groups = full.reshape(Np, Kp // 32, 32)
    top = np.abs(groups).max(-1)
    finite = np.isfinite(groups).all(-1)
    with np.errstate(invalid="ignore"):
        exponent = np.where(finite & (top > 0), np.frexp(np.where(finite, top, 1.0))[1] - 1 - 2, -127)
    byte = np.where(finite, np.maximum(exponent, -127) + 127, 255)
    a = np.where(finite[..., None], np.abs(groups) / POWERS[np.minimum(byte, 254)][..., None], 0.0)
    code = np.zeros(a.shape, dtype=np.uint8)
    best = np.full(a.shape, np.inf)
    for i, v in enumerate(GRID):          # nearest, ties to the even code, beyond 6 to 6
        d = np.abs(np.minimum(a, 6.0) - v)
        take = (d < best) | ((d == best) & (i % 2 == 0))
        code[take] = i
        best = np.minimum(best, d)
    code |= np.where(np.signbit(groups) & finite[..., None], 8, 0).astype(np.uint8)
    code = code.reshape(Np, Kp)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    codes = packed.reshape(Np // 128, 128, Kp // 128, 64).transpose(0, 2, 1, 3).copy()
    scales = np.zeros((Np // 128, Kp // 128, 512), dtype=np.uint8)
    byte = byte.astype(np.uint8).reshape(Np // 128, 128, Kp // 128, 4)
    for r in range(128):
        for g in range(4):
            scales[:, :, scale_at(r, g)] = byte[:, r, :, g]
    return codes, scales


def unpack(codes, scales, N, K):
    """W [N, K] in 64 bits."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    nb, kb = codes.shape[:2]
    code = np.stack([codes & 15, codes >> 4], -1).reshape(nb, kb, 128, 128)
    value = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    spot = np.array([[scale_at(r, g) for g in range(4)] for r in range(128)])
    factor = POWERS[scales[:, :, spot]]
    w = (value.reshape(nb, kb, 128, 4, 32) * factor[..., None]).reshape(nb, kb, 128, 128)
    return w.transpose(0, 2, 1, 3).reshape(nb * 128, kb * 128)[:N, :K]


def tolerance(w, x, out_dtype):
    """Bound on |y - exact| per element, [M, N], for W [N, K] and x [M, K] in 64 bits.

    A step of the tensor core adds 32 exact products to its accumulator, all
    aligned to the largest of the 33 and cut below 2^-24 of it: at most
    33 * 2^-24 * sum |W x|.  The accumulator is read out every 8 blocks of
    128 k (32 steps) for a binary32 y and every 64 (256 steps) for bfloat16,
    and what is read out is added in binary32: 2^-24 * sum |W x| each time.
    x's two parts miss at most 2^-22 of their group's largest |x|: half of the
    low part's smallest step, 2^-9 * (s / 32) / 2 = 2^-15 s, with that largest
    at least 128 s.  bfloat16 rounds once more, by half a step, 2^-8 of the
    value at most.
    """
    K = w.shape[1]
    absw = np.abs(w)
    total = np.abs(x) @ absw.T
    top = np.abs(np.pad(x, ((0, 0), (0, -K % 32)))).reshape(x.shape[0], -1, 32).max(-1)
    split = np.repeat(top, 32, axis=1)[:, :K] @ absw.T * 2.0 ** -22
    flush = 8 if out_dtype == torch.float32 else 64
    steps = min(-(-K // 32), 4 * flush)
    rounds = -(-K // (128 * flush)) + 64      # read-outs, and parts of a tile
    bound = total * 2.0 ** -24 * (33 * steps + rounds) + split + 1e-37
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(x @ w.T) + bound)
    return bound


def sort(ids, E):
    """(offsets [E + 1], rows [T], places [M, top]) of the choices ids [M, top]."""
    ids = np.asarray(ids)
    M, top = ids.shape
    buckets = [[] for _ in range(E + 1)]
    for slot, i in enumerate(ids.reshape(-1).tolist()):
        buckets[i if 0 <= i < E else E].append(slot)
    offsets = np.cumsum([0] + [len(b) for b in buckets[:E]])
    rows = np.full(M * top, -1)
    places = np.zeros(M * top, dtype=np.int64)
    p = 0
    for e, b in enumerate(buckets):
        for slot in b:
            if e < E:
                rows[p] = slot // top
            places[slot] = p if e < E else -1 - p
            p += 1
    return offsets, rows, places.reshape(M, top)
