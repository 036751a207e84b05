"""64-bit definitions of the sort by expert and back and of the MXFP4 operators (CPU), for the tests."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# half the spacing of the smallest values (subnormals) of each type
HALF_MIN = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
U32 = 2.0 ** -24


def sort(ids, E):
    """offsets [E+1], sorted_routes [R], route_rows [T, k] from the definition."""
    ids = np.asarray(ids)
    flat = [int(e) if 0 <= e < E else E for e in ids.reshape(-1)]
    order = sorted(range(len(flat)), key=lambda r: (flat[r], r))
    offsets = [sum(1 for e in flat if e < x) for x in range(E + 1)]
    row = [0] * len(flat)
    for j, r in enumerate(order):
        row[r] = j if flat[r] < E else -1 - j
    return np.array(offsets), np.array(order, dtype=np.int64), np.array(row).reshape(ids.shape)


def unpermute(rows, route_rows, weights):
    """(sum of weight * row, sum of |weight * row|) in float64; negative rows add nothing."""
    T, k = route_rows.shape
    out = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for s in range(k):
            j = route_rows[t, s]
            if j >= 0:
                v = rows[j] * (1.0 if weights is None else weights[t, s])
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def e2m1_code(m):
    """Code 0..7 of the e2m1 value nearest to m >= 0, ties to the even code, 6 at most."""
    d = np.abs(np.asarray(m)[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    tied = d == best
    first = tied.argmax(-1)
    return np.where((tied.sum(-1) == 2) & (first % 2 == 1), first + 1, first)


def quantize(x):
    """codes (one per value, sign in bit 3) and scale bytes of x [..., K] (float64 holding the
    inputs exactly), blocks along the last axis."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    finite = np.isfinite(b).all(-1)
    safe = np.where(finite[..., None], b, 0.0)
    top = np.abs(safe).max(-1)
    e = np.frexp(top)[1] - 1  # floor(log2 top) where top > 0
    e = np.where(top > 0, np.maximum(e - 2, -127), -127)
    code = e2m1_code(np.abs(safe) / np.ldexp(1.0, e)[..., None])
    code = np.where(np.signbit(safe), code + 8, code)
    code = np.where(finite[..., None], code, 0)
    scale = np.where(finite, e + 127, 255)
    return code.reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def values(codes, scales):
    """float64 values of packed codes [..., K/2] with scale bytes [..., K/32]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(*codes.shape[:-1], -1)
