"""Plain 64-bit (and exact whole-number) references of the speculative decoding
operators, and builders of small random batches for their tests."""
from __future__ import annotations

import numpy as np
import torch

# unit roundoff of one rounding to the type
ROUNDOFF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
NEG = float("-inf")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- batches -------------------------------------------------------------------------


def random_tree(rng, n, reach=6):
    return [-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, n)] if n else []


def chain(n):
    return list(range(-1, n - 1))


def paged(rng, lens, bs, spare=2):
    """(block_table [B, width] int32, blocks): scattered pages for lens[b] tokens."""
    need = [-(-x // bs) for x in lens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(1, max(need, default=1))), -7, np.int32)  # unused: not an index
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, sum(need) + spare


def slots_of(table, b, positions, bs):
    return [int(table[b, j // bs]) * bs + j % bs for j in positions]


def ptr_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# ---- rotary positions ------------------------------------------------------------------


def rope(x, positions, inv_freq, interleaved, scale, inverse):
    """(value, magnitude) of the rotation of x [T, H, D] in 64 bits; magnitude
    bounds the terms of each output."""
    x = f64(x)
    half = len(inv_freq)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq)  # exact enough: < 2^31 * 2^-53
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
    s = -s if inverse else s
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, m = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    m[..., a] = m[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(scale)
    return y, m


def rope_bound(y, m, dtype):
    """One rounding of the result; the fp32 sine, cosine, products and sum are
    each off by a few 2^-24 of the terms; 2^-25 for results below the normal range."""
    return ROUNDOFF[dtype] * np.abs(y) + 16 * 2.0 ** -24 * m + 2.0 ** -25


# ---- tree attention ----------------------------------------------------------------------


def ancestors(parents):
    """sees[i, j]: node i is j or a descendant of j; none for padding rows."""
    n = len(parents)
    sees = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            if parents[j] == -2:
                break
            sees[i, j] = True
            j = parents[j]
    return sees


def attention(q, k_cache, v_cache, table, prefix, ptr, parents, scale, dtype):
    """(out, lse, bound of out, bound of lse) in 64 bits for the covered rows."""
    q, bs = f64(q), k_cache.shape[1]
    Hq, D, Hkv = q.shape[1], q.shape[2], k_cache.shape[2]
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], NEG)
    tol, ltol = np.full(q.shape, 2.0 ** -25), np.zeros(q.shape[:2])
    u = ROUNDOFF[dtype]
    flat_k, flat_v = k_cache.reshape(-1, Hkv, D), v_cache.reshape(-1, Hkv, D)
    for b in range(len(prefix)):
        t0, t1 = int(ptr[b]), int(ptr[b + 1])
        n, P = t1 - t0, int(prefix[b])
        if n == 0:
            continue
        at = torch.tensor(slots_of(table, b, range(P + n), bs), device=k_cache.device)
        K, V = f64(flat_k[at]), f64(flat_v[at])
        par = chain(n) if parents is None else [int(p) for p in parents[t0:t1]]
        sees = ancestors(par)
        for i in range(n):
            live = np.concatenate([np.full(P, par[i] != -2), sees[i]])
            if not live.any():
                continue
            for h in range(Hq):
                kk, vv, x = K[live, h // (Hq // Hkv)], V[live, h // (Hq // Hkv)], q[t0 + i, h]
                s = scale * (kk @ x)
                # fp32 scores: one rounding per product and sum, of terms no
                # larger than scale |q| |k|; then the exponent's own rounding
                off = (D + 16) * 2.0 ** -24 * float((np.abs(scale) * (np.abs(kk) @ np.abs(x))).max()) + 2.0 ** -20
                m = s.max()
                e = np.exp(s - m)
                l = e.sum()
                out[t0 + i, h] = e @ vv / l
                lse[t0 + i, h] = m + np.log(l)
                mag = e @ np.abs(vv) / l
                # each weight is rounded once to the type (f16 weights below
                # 2^-21 of the largest lose relative accuracy: 2^-24 |v| each), sums
                # in fp32, then the result is rounded once
                tol[t0 + i, h] += (u * np.abs(out[t0 + i, h]) + (u + 2 * off + (len(s) + 64) * 2.0 ** -24) * mag
                                   + (2.0 ** -24 * np.abs(vv).sum(0) / l if dtype == torch.float16 else 0))
                ltol[t0 + i, h] = off + (len(s) + 16) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[t0 + i, h])
    return out, lse, tol, ltol


# ---- verification -------------------------------------------------------------------------

ONE, UNIT = 1 << 38, 1 << 24


def _prob(x):
    return np.nan_to_num(np.clip(np.asarray(x, np.float32), np.float32(0), np.float32(1)), nan=0.0)


def weights(p):
    return (_prob(p) * np.float32(2.0 ** 38)).astype(np.int64)


def _f32(w):
    return np.float32(int(w))  # whole numbers below 2^63, rounded to nearest once


def verify(target, draft, tokens, parents, ptr, accept, sample, max_path):
    B = len(ptr) - 1
    count, path, token = np.zeros(B, np.int32), np.full((B, max_path), -1, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        t0, n = int(ptr[b]), int(ptr[b + 1] - ptr[b])
        if n == 0:
            continue
        par = chain(n) if parents is None else list(parents[t0:t0 + n])
        cur, w, W = 0, weights(target[t0]), ONE
        path[b, 0], count[b] = 0, 1
        for i in range(1, n):
            if par[i] != cur or count[b] == max_path:
                continue
            x = int(tokens[t0 + i])
            q = np.float32(1) if draft is None else _prob(draft[t0 + cur, x])
            if np.float32(np.float32(accept[t0 + i]) * q) * _f32(W) < _f32(w[x]):
                path[b, count[b]] = i
                count[b] += 1
                cur, w, W = i, weights(target[t0 + i]), ONE
            else:
                if draft is None:
                    w = w.copy()
                    w[x] = 0
                else:
                    w = np.maximum(w - (_prob(draft[t0 + cur]) * _f32(W)).astype(np.int64), 0)
                W = int(w.sum())
        if w.sum() == 0:
            w = weights(target[t0 + cur])
        total = int(w.sum())
        if total:
            m = min(max(int(np.float32(sample[b]) * np.float32(UNIT)), 0), UNIT - 1)
            token[b] = int(np.searchsorted(np.cumsum(w), (total * m) >> 24, side="right"))
    return count, path, token


# ---- commit ---------------------------------------------------------------------------------


def commit(cache, table, prefix, path, count):
    """The cache [layers, blocks, bs, H, D] (numpy) after the moves."""
    new, bs = cache.copy(), cache.shape[2]
    for b in range(len(prefix)):
        for d in range(int(count[b])):
            i, j = int(prefix[b]) + d, int(prefix[b]) + int(path[b, d])
            new[:, table[b, i // bs], i % bs] = cache[:, table[b, j // bs], j % bs]
    return new
