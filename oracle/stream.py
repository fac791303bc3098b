"""Float64 CPU oracle of the residual stream's operators: counter-based dropout, the scaled embedding
and its gradient, and the norms around a block with their gradient.

TEST INFRASTRUCTURE ONLY: the CUDA library never calls it and shares no code with it.  Pinned in
tests/test_oracle_stream_pins.py by the generator's published answers, by finite differences and by
torch autograd."""
from __future__ import annotations

import numpy as np

M32 = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., SC 2011): counter [4][...] and key [2] of 32-bit words -> [4][...]."""
    c = [np.asarray(x, dtype=np.uint64) & M32 for x in counter]
    k = [int(x) & 0xFFFFFFFF for x in key]
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & M32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_factors(rows, cols, p, seed, base, offset):
    """0 or 65536 / (65536 - n) for every element of the given rows (an int: all rows below it)."""
    rows = np.arange(rows) if np.ndim(rows) == 0 else np.asarray(rows)
    n = int(np.floor(p * 65536 + 0.5))
    if n == 0:
        return np.ones((len(rows), cols))
    per_row = -(-cols // 8)
    b = rows.astype(np.uint64)[:, None] * np.uint64(per_row) + np.arange(per_row, dtype=np.uint64)[None]
    o, seed = (base + offset) % 2 ** 64, seed % 2 ** 64
    w = philox4x32([b, b >> np.uint64(32), np.full_like(b, o & 0xFFFFFFFF), np.full_like(b, o >> 32)],
                   [seed & 0xFFFFFFFF, seed >> 32])
    u = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], -1)
    u = u.reshape(len(rows), 8 * per_row)[:, :cols]
    return np.where(u >= n, 65536.0 / (65536 - n) if n < 65536 else 0.0, 0.0)


def dropout(x, factors):
    """Dropped elements are 0 whatever they hold."""
    return np.where(factors == 0, 0.0, np.where(factors == 0, 0.0, x) * factors)


def _token_factors(ids, vocab, scale, row_scale):
    f = np.full(len(ids), float(scale)) if row_scale is None else scale * np.asarray(row_scale, dtype=np.float64)
    return np.where((ids >= 0) & (ids < vocab), f, 0.0)[:, None]


def embed(ids, table, scale, row_scale, factors):
    ids = np.asarray(ids)
    ok = ((ids >= 0) & (ids < len(table)))[:, None]
    rows = np.where(ok, table[np.clip(ids, 0, len(table) - 1)], 0.0)
    return dropout(rows * _token_factors(ids, len(table), scale, row_scale), factors)


def embed_backward(ids, d_out, vocab, scale, row_scale, factors):
    """The gradient and, element by element, the sum of its terms' magnitudes."""
    ids = np.asarray(ids)
    f = _token_factors(ids, vocab, scale, row_scale)
    terms = np.where(f == 0, 0.0, dropout(d_out, factors) * f)
    out, mag = np.zeros((vocab, d_out.shape[1])), np.zeros((vocab, d_out.shape[1]))
    ok = (ids >= 0) & (ids < vocab)
    np.add.at(out, ids[ok], terms[ok])
    np.add.at(mag, ids[ok], np.abs(terms[ok]))
    return out, mag


def moments(z, rms, eps):
    mean = np.zeros((len(z), 1)) if rms else z.mean(1, keepdims=True)
    return mean, 1.0 / np.sqrt(((z - mean) ** 2).mean(1, keepdims=True) + eps)


def _affine(z, gamma, beta):
    return z * gamma + (0.0 if beta is None else beta)


def block_norm(x, y, p, factors, eps):
    """p: dict of rms, residual_scale, post_gamma, post_beta, pre_gamma, pre_beta, gate.
    Returns x_out, h (or None) and stats [rows, 4]."""
    stats = np.zeros((len(x), 4))
    u = y
    if p["post_gamma"] is not None:
        m, r = moments(y, p["rms"], eps)
        stats[:, 0:1], stats[:, 1:2] = m, r
        u = _affine((y - m) * r, p["post_gamma"], p["post_beta"])
    u = dropout(u, factors)
    x_out = p["residual_scale"] * x + (u if p["gate"] is None else p["gate"] * u)
    h = None
    if p["pre_gamma"] is not None:
        m, r = moments(x_out, p["rms"], eps)
        stats[:, 2:3], stats[:, 3:4] = m, r
        h = _affine((x_out - m) * r, p["pre_gamma"], p["pre_beta"])
    return x_out, h, stats


def _norm_backward(g, zhat, rstd, rms):
    g0 = 0.0 if rms else g.mean(1, keepdims=True)
    return rstd * (g - g0 - zhat * (g * zhat).mean(1, keepdims=True))


def block_norm_backward(x_out, y, stats, d_x_out, d_h, p, factors):
    """dx, dy and a dict of the parameters' gradients, from the forward's statistics."""
    my, ry, mx, rx = (stats[:, i:i + 1] for i in range(4))
    grads = {}
    G = np.zeros_like(y) if d_x_out is None else d_x_out
    if p["pre_gamma"] is not None:
        xh = (x_out - mx) * rx
        grads["pre_gamma"], grads["pre_beta"] = (d_h * xh).sum(0), d_h.sum(0)
        G = G + _norm_backward(d_h * p["pre_gamma"], xh, rx, p["rms"])
    post = p["post_gamma"] is not None
    yh = (y - my) * ry if post else y
    dn = dropout(G, factors)
    if p["gate"] is not None:
        n = _affine(yh, p["post_gamma"], p["post_beta"]) if post else y
        per_row = dn * dropout(n, np.where(factors == 0, 0.0, 1.0))
        grads["gate"] = per_row if np.ndim(p["gate"]) == 2 else per_row.sum(0)
        dn = dn * p["gate"]
    dy = dn
    if post:
        grads["post_gamma"], grads["post_beta"] = (dn * yh).sum(0), dn.sum(0)
        dy = _norm_backward(dn * p["post_gamma"], yh, ry, p["rms"])
    return p["residual_scale"] * G, dy, grads
