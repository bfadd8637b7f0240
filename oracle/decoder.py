"""Oracle of the operators between a decoding step's projections: norm, 8-bit product, rotary
positions, sampling.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Plain fp64 from the definitions in include/svdq_decoder.h; the contract's fp32 roundings are NumPy's
IEEE float32, and sampling's whole numbers are Python's.
"""
from __future__ import annotations

import math

import numpy as np

from .numerics import round_bf16

UNIT = 1 << 40


# -------------------------------------------------------------------------------------- norm
def rms_norm(x, residual, gamma, eps):
    """(h, y) fp64 [M, K]: h = fl32(x + residual), y = h / sqrt(mean(h^2) + eps) gamma."""
    h = np.asarray(x, np.float32)
    if residual is not None:
        with np.errstate(over="ignore"):
            h = h + np.asarray(residual, np.float32)
    h = h.astype(np.float64)
    g = np.ones(h.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        rms = np.sqrt((h * h).mean(axis=1, keepdims=True) + float(eps))
        y = np.where(h == 0.0, 0.0, h / rms) * g
    return h, y


def rows8(y):
    """(codes fp64 before rounding, scales) of fp64 rows, unrounded: y / s and s = max |y| / 127."""
    s = np.abs(y).max(axis=1) / 127.0
    with np.errstate(invalid="ignore", divide="ignore"):
        return np.where(s[:, None] > 0, y / s[:, None], 0.0), s


def quantize_rows(x, factor):
    """(codes, scales) exactly as stored: fp32 products, scale and quotient."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        y = np.asarray(x, np.float32)
        if factor is not None:
            y = y * np.asarray(factor, np.float32)[None, :]
        s = np.abs(y).max(axis=1) / np.float32(127.0)
        q = np.rint(y / s[:, None])
    ok = (np.isfinite(s) & (s > 0))[:, None]
    return np.where(ok, np.clip(np.where(ok, q, 0.0), -127, 127), 0.0).astype(np.int8), s


# ----------------------------------------------------------------------------------- product
def linear8(qx, sx, qw, sw, bias, bf16):
    """Y exactly as stored, fp64: whole-number sums, then the fp32 roundings in their order."""
    acc = np.asarray(qx, np.int64) @ np.asarray(qw, np.int64).T
    with np.errstate(over="ignore", invalid="ignore"):
        y = (acc.astype(np.float32) * np.asarray(sx, np.float32)[:, None]) * np.asarray(sw, np.float32)[None, :]
        if bias is not None:
            y = y + np.asarray(bias, np.float32)[None, :]
    y = y.astype(np.float64)
    return round_bf16(y) if bf16 else y


# -------------------------------------------------------------------------------------- rope
def rope(x, positions, freqs, interleaved, scale):
    """(out, mag) fp64 [rows, heads, dim]: the turned heads, and |a| + |b| of each channel's pair."""
    out, mag = np.array(x, np.float64), np.zeros(x.shape)
    half = len(freqs)
    for r, pos in enumerate(positions):
        for i, f in enumerate(freqs):
            c, s = math.cos(int(pos) * float(f)) * scale, math.sin(int(pos) * float(f)) * scale
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = x[r, :, p], x[r, :, q]
            out[r, :, p], out[r, :, q] = a * c - b * s, a * s + b * c
            mag[r, :, p] = mag[r, :, q] = (np.abs(a) + np.abs(b)) * abs(scale)
    return out, mag


# ------------------------------------------------------------------------------------ sample
def weights(z, temperature):
    """Whole-number weights of one row (a list), for a temperature > 0."""
    top = max(z)
    out = []
    for v in z:
        if v == -math.inf:
            out.append(0)
        elif top == math.inf:
            out.append(UNIT if v == math.inf else 0)
        else:
            out.append(round(math.exp((v - top) / temperature) * UNIT))
    return out


def sample_row(z, temperature, u, top_k=0, top_p=1.0, min_p=0.0):
    """(token, share) of one row of Python floats."""
    z = [float(v) for v in z]
    if any(math.isnan(v) for v in z) or max(z) == -math.inf:
        return -1, 0.0
    if not temperature > 0:
        return z.index(max(z)), 1.0
    w = weights(z, temperature)
    kept = sorted(range(len(z)), key=lambda i: (-z[i], i))
    if top_k > 0:
        kept = kept[:top_k]
    if top_p < 1:
        least, before, stay = float(top_p) * float(sum(w[i] for i in kept)), 0, []
        for i in kept:
            if float(before) < least or not stay:
                stay.append(i)
            before += w[i]
        kept = stay
    if min_p > 0:
        kept = [i for i in kept if w[i] >= min(min_p, 1.0) * UNIT]
    total = sum(w[i] for i in kept)
    u = min(u, 1 - 2.0 ** -24) if u > 0 else 0.0
    at = min(math.floor(float(total) * u), total - 1)
    run = 0
    for i in sorted(kept):
        run += w[i]
        if run > at:
            return i, w[i] / total
    raise AssertionError("the weights do not add up")
