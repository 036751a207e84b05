"""64-bit definitions of routing by scores, 8-bit floating point in blocks of 128 and the gated activation
(CPU), for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests._expert_ref import HALF_MIN, HALF_STEP, U32  # noqa: F401

BLOCK = 128
# the 127 finite magnitudes of e4m3 by code: exponent bits e, mantissa bits m
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


# ---------------------------------------------------------------- routing by scores
def scores(logits, sigmoid):
    """Scores of one row in float64; NaN for the whole row where softmax has none."""
    x = logits.astype(np.float64)
    with np.errstate(all="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-x))
        if np.isneginf(x).all():
            return np.zeros_like(x)
        p = np.exp(x - x.max())
        return p / p.sum()


def choose(logits, bias, top_k, sigmoid, n_groups=1, top_groups=1, group_top=1):
    """Ids of one row: one sort by (choice down, index up)."""
    c = scores(logits, sigmoid)
    if bias is not None:
        c = c + bias.astype(np.float64)
    c = np.where(np.isneginf(logits), -np.inf, c)
    order = lambda v: sorted(range(len(v)), key=lambda i: (0 if np.isnan(v[i]) else 1, -v[i] if not np.isnan(v[i]) else 0, i))  # noqa: E731
    if top_groups < n_groups:
        rank = []
        for g in c.reshape(n_groups, -1):
            best = [g[i] for i in order(g)[:group_top]]
            rank.append(best[0] + sum(v for v in best[1:] if not np.isneginf(v)))
        lost = order(np.array(rank))[top_groups:]
        c = c.reshape(n_groups, -1).copy()
        c[lost] = -np.inf
        c = c.reshape(-1)
    ids = [i for i in order(c)[:top_k] if not np.isneginf(c[i])]
    return np.array(ids + [-1] * (top_k - len(ids)))


def _log_scores(l, sigmoid):
    return -np.logaddexp(0.0, -l) if sigmoid else l


def weights(logits, ids, sigmoid, normalize, scale):
    """Weights of one row's ids in float64, also where the scores themselves are 0 to it."""
    out = np.zeros(len(ids))
    at = ids[ids >= 0]
    l = logits.astype(np.float64)
    if normalize and len(at):
        v = _log_scores(l[at], sigmoid)
        e = np.exp(v - v.max())
        out[ids >= 0] = e / e.sum()
    elif len(at):
        out[ids >= 0] = scores(logits, sigmoid)[at]
    return out * scale


def route_grad(logits, ids, grad, sigmoid, normalize, scale):
    """(gradient of one row's logits, its terms' magnitudes) in float64."""
    E = len(logits)
    out, mag = np.zeros(E), np.zeros(E)
    kept = (ids >= 0) & (ids < E)
    kept &= ~np.isneginf(logits[np.where(kept, ids, 0)])
    at, g = ids[kept], grad[kept].astype(np.float64) * scale
    if not len(at) and (normalize or sigmoid):
        return out, mag
    w = weights(logits, at, sigmoid, normalize, 1.0)
    rest = 1.0 / (1.0 + np.exp(logits[at].astype(np.float64)))  # 1 - sigmoid
    if normalize:
        v = w * (g - (g * w).sum()) * (rest if sigmoid else 1.0)
        a = w * (np.abs(g) + np.abs(g * w).sum()) * (rest if sigmoid else 1.0)
    elif sigmoid:
        v = g * w * rest
        a = np.abs(v)
    else:
        p = scores(logits, False)
        full, size = np.zeros(E), np.zeros(E)
        np.add.at(full, at, g)
        np.add.at(size, at, np.abs(g))
        return p * (full - (g * w).sum()), p * (size + np.abs(g * w).sum())
    np.add.at(out, at, v)
    np.add.at(mag, at, a)
    return out, mag


def weight_error(logits, ids, E):
    """Relative error of a weight in float32, in units of 2^-24.  exp(l - m) turns the rounding of l - m into
    |l - m| units, and is good to 2 more; a sigmoid over another takes 2 exponentials (3 each), 2 sums, 2
    quotients; a sum over k slots or E experts adds in trees of at most 6 levels, behind 16 experts a lane;
    quotient and scale 1 each.  A quotient carries the error of both of its sides."""
    finite = logits[np.isfinite(logits)]
    spread = float(finite.max() - finite.min()) if finite.size else 0.0
    spread = max(spread, float(np.abs(finite).max()) if finite.size else 0.0)
    return 2 * (spread + 14) + 22 + 4


# ---------------------------------------------------------------- 8-bit floating point
def scale_of(top):
    """The least power of two, at least 2^-126, with top <= 448 scale."""
    if not np.isfinite(top):
        return np.nan
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def code_of(v):
    """Code of the e4m3 value nearest to v (|v| <= 448), ties to the even code."""
    m = np.abs(v)
    mid = (E4M3[:-1] + E4M3[1:]) / 2
    at = np.searchsorted(mid, m, side="left")  # the lower code on a tie
    tie = (at < 126) & (m == mid[np.minimum(at, 125)])
    at = np.where(tie & (at % 2 == 1), at + 1, at)
    return (at + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _block(b):
    s = scale_of(np.abs(b).max() if np.isfinite(b).all() else np.inf)
    return (np.zeros(b.shape, np.uint8) if np.isnan(s) else code_of(b / s)), s


def quantize(x, block_rows):
    """codes and scales of a matrix (float64 holding the inputs exactly)."""
    R, C = x.shape
    codes = np.zeros((R, C), np.uint8)
    scales = np.zeros((-(-R // block_rows), -(-C // BLOCK)))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            codes[at], scales[i, j] = _block(x[at])
    return codes, scales


def code_values(codes):
    c = codes.astype(np.int64)
    v = np.append(E4M3, np.nan)[c & 127]
    return np.where(c & 128, -v, v)


def values(codes, scales, block_rows=1):
    """What codes [R, C] with scales [ceil(R / block_rows), ceil(C / 128)] stand for, in float64."""
    R, C = codes.shape
    s = np.asarray(scales, np.float64)[np.arange(R) // block_rows][:, np.arange(C) // BLOCK]
    return code_values(codes) * s


def matmul(a, w, sa, sw):
    """(product, bound) of codes a [R, K], w [N, K] with scales sa [R, blocks], sw [N/128 rounded up, blocks].  The
    matrix instruction keeps each of eight neighbouring products to 2^-13 of the largest's power of two (a product
    of two mantissas is below 4 of it, and not below it); the other roundings are float32's, a whole unit (2 U32)
    where it may truncate: 16 sums in a block, the scales' product, its product with the sum and one sum a block."""
    x, y = values(a, sa), values(w, sw, BLOCK)
    eights = lambda v: np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 8)))).reshape(v.shape[0], -(-v.shape[1] // 8), 8).max(-1)  # noqa: E731
    want, mag = x @ y.T, np.abs(x) @ np.abs(y.T)
    blocks = -(-a.shape[1] // BLOCK)
    return want, 8 * 2.0 ** -13 * (eights(x) @ eights(y).T) + (2 * 17 + blocks + 3) * U32 * mag


# ---------------------------------------------------------------- gated activation
def gate(g, geglu, alpha=1.0, limit=math.inf):
    """g', s(z), 1 - s(z) and g' dz/dg of gates in float64."""
    g = np.asarray(g, np.float64)
    with np.errstate(all="ignore"):
        if geglu:
            c = 2 * math.sqrt(2 / math.pi)
            h = np.clip(g, -1e3, 1e3)  # far behind where s is 0 or 1
            z, slope = c * (h + 0.044715 * h ** 3), c * h * (1 + 3 * 0.044715 * h * h)
        else:
            g = np.minimum(g, limit)
            z = slope = alpha * g
        s, rest = np.exp(-np.logaddexp(0, -z)), np.exp(-np.logaddexp(0, z))
    return g, s, rest, slope, z


def activate(g, u, geglu, alpha=1.0, beta=0.0, limit=math.inf):
    """(values, error bound of float32 arithmetic) of the activation.  s is good to 8 units and to |z| times the
    relative error of z (1 unit for alpha g, 4 for GELU's polynomial) where the exponential carries it; three
    products follow."""
    gp, s, rest, slope, z = gate(g, geglu, alpha, limit)
    lin = np.asarray(u, np.float64) if geglu else np.clip(u, -limit, limit) + beta
    out = gp * s * lin
    lin_mag = np.abs(lin) if geglu else np.abs(np.clip(u, -limit, limit)) + abs(beta)
    err = (12 + (5 if geglu else 1) * np.minimum(np.abs(z), 150)) * U32 * np.abs(gp) * s * lin_mag
    return out, err + 2.0 ** -120 * (1 + np.abs(gp) * lin_mag)  # an exponential below 2^-126 is 0


def activate_grad(d, g, u, geglu, alpha=1.0, beta=0.0, limit=math.inf):
    """(to gate, its bound, to up, its bound)."""
    gp, s, rest, slope, z = gate(g, geglu, alpha, limit)
    d = np.asarray(d, np.float64)
    lin = np.asarray(u, np.float64) if geglu else np.clip(u, -limit, limit) + beta
    lin_mag = np.abs(lin) if geglu else np.abs(np.clip(u, -limit, limit)) + abs(beta)
    unit = (16 + (5 if geglu else 1) * np.minimum(np.abs(z), 150)) * U32
    slope = np.where(np.abs(z) > 150, np.clip(slope, -1e4, 1e4), slope)  # s or 1 - s is 0 there
    up = d * gp * s
    to_gate = d * lin * s * (1 + slope * rest)
    gate_err = 2 * unit * np.abs(d) * lin_mag * s * (1 + np.abs(slope) * rest)
    if not geglu:
        up = np.where(np.abs(u) > limit, 0.0, up)
        to_gate = np.where(np.asarray(g) > limit, 0.0, to_gate)
    tiny = 2.0 ** -118 * (1 + np.abs(d) * (np.abs(gp) + lin_mag * (1 + np.abs(slope))))
    return to_gate, gate_err + tiny, up, unit * np.abs(d * gp) * s + tiny
