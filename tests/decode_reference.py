"""Plain 64-bit (and whole-number) references of head norms with rotary positions, e4m3
values and sampling, for their tests."""
from __future__ import annotations

import numpy as np
import torch

from tests import spec_reference as ref

E4M3 = torch.float8_e4m3fn
TOP, ONE, UNIT = 448.0, 1 << 38, 1 << 24


def e4m3_bound(y):
    """Half a step of e4m3 at y: 2^-4 of it, or of the subnormal step 2^-9."""
    return np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10)


# ---- norms and rotary positions ----------------------------------------------------------


def turn(x, positions, inv_freq, interleaved, scale, back=False):
    return ref.rope(torch.from_numpy(x), positions, inv_freq, interleaved, scale, back)


def norm_rope(x, w, eps, positions, inv_freq, interleaved, scale):
    """(value, magnitude of the terms) of the head norm and rotation of x [T, H, D]."""
    x = ref.f64(x)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * ref.f64(w)
    return turn(x, positions, inv_freq, interleaved, scale)


def norm_rope_bound(y, m, D, dtype):
    """One rounding to the type; in fp32 the mean (D squares and sums in a tree: D / 8 + 8
    roundings at most), its root (2 units), two products, sine, cosine, products and sum."""
    return ref.ROUNDOFF.get(dtype, 0.0) * np.abs(y) + (D / 8 + 32) * 2.0 ** -24 * m + 2.0 ** -25


def norm_rope_grad(dy, x, w, eps, positions, inv_freq, interleaved, scale):
    """(dx, dw, magnitudes of both's terms) in 64 bits."""
    g, gm = turn(ref.f64(dy), positions, inv_freq, interleaved, scale, back=True)
    if w is None:
        return g, None, gm, None
    x, w = ref.f64(x), ref.f64(w)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh, h = x * r, g * w
    mean = np.mean(h * xh, -1, keepdims=True)
    dx = r * (h - xh * mean)
    mag = r * (gm * np.abs(w) + np.abs(xh) * np.mean(gm * np.abs(w) * np.abs(xh), -1, keepdims=True))
    return dx, (g * xh).sum((0, 1)), mag, (gm * np.abs(xh)).sum((0, 1))


# ---- sampling ---------------------------------------------------------------------------------


def canonical(logits):
    x = logits.detach().float().cpu().numpy().astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    return np.where(np.isneginf(x), x, np.clip(x, -2.0 ** 126, 2.0 ** 126))


def part(total, fraction):
    """fraction (fp32) of a whole number, in multiples of 2^-24."""
    f = np.float32(fraction)
    f = 0.0 if np.isnan(f) else min(1.0, max(0.0, float(f)))
    return (total * int(f * UNIT)) >> 24


def sample(x, tau, k, p, m, u):
    """(token, kept weights [V] as whole numbers) of one canonical row x."""
    V, w = x.size, np.zeros(x.size, np.int64)
    if np.isneginf(x).all():
        return -1, w
    order = np.lexsort((np.arange(V), -x))
    tau = np.float32(tau)
    if not tau > 0:
        ranked = np.zeros(V, np.int64)
        ranked[0] = ONE
    else:
        with np.errstate(invalid="ignore", over="ignore"):
            ranked = np.floor(np.exp((x[order] - x[order[0]]) / float(tau)) * ONE).astype(np.int64)
    if 0 < k < V:
        ranked[k:] = 0
    p = np.float32(p)
    if not p >= 1:
        before = np.concatenate([[0], np.cumsum(ranked)[:-1]])
        ranked[(before >= part(int(ranked.sum()), p)) & (np.arange(V) > 0)] = 0
    m = np.float32(m)
    least = 0 if np.isnan(m) else int(min(1.0, max(0.0, float(m))) * ONE)
    ranked[ranked < least] = 0
    w[order] = ranked
    run = np.cumsum(w)
    mark = part(int(run[-1]), min(float(u), 1 - 2.0 ** -24))
    return int(np.searchsorted(run, mark, side="right")), w
