"""Plain float64 definitions of the operators in a dense block: dropout from a
counter-based generator, layer norm with bias, dropout and residual add, 8-bit rows
and their products.  Numpy only; shares no code with the HIP library.
``tests/test_dense_block_cpu.py`` checks the generator against published values and the
gradients against differences."""
from __future__ import annotations

import numpy as np

LOW = np.uint64(0xFFFFFFFF)
SHIFT = np.uint64(32)


def philox4x32(counter, key, rounds=10):
    """Four words (uint32 arrays) of Philox4x32 for four counter words and two key words."""
    c = [np.asarray(x, dtype=np.uint64) & LOW for x in counter]
    k = [int(x) & 0xFFFFFFFF for x in key]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> SHIFT) ^ c[1] ^ np.uint64(k[0]), b & LOW,
             (a >> SHIFT) ^ c[3] ^ np.uint64(k[1]), a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [x.astype(np.uint32) for x in c]


def threshold(p):
    return int(np.floor((1.0 - float(np.float32(p))) * 65536.0 + 0.5))


def keep_factor(M, N, p, seed, offset, draw=0, row_begin=0, col_begin=0):
    """What each element of [M, N] is multiplied by: 65536 / threshold, or 0."""
    t = threshold(p)
    if t >= 65536:
        return np.ones((M, N))
    if t == 0:
        return np.zeros((M, N))
    at = (offset + draw) % 2 ** 64
    rows = (row_begin + np.arange(M, dtype=np.uint64))[:, None]
    cols = (col_begin // 8 + np.arange(-(-N // 8), dtype=np.uint64))[None, :]
    rows, cols = np.broadcast_arrays(rows, cols)
    w = philox4x32((cols, rows, np.full(rows.shape, at % 2 ** 32, np.uint64),
                    np.full(rows.shape, at // 2 ** 32, np.uint64)),
                   (seed % 2 ** 64 % 2 ** 32, seed % 2 ** 64 // 2 ** 32))
    halves = np.stack([h for x in w for h in (x & 0xFFFF, x >> 16)], axis=-1)
    return (halves.reshape(M, -1)[:, :N] < t) * (65536.0 / t)


def layer_norm(block, resid, bias, w, b, factor, eps):
    """(out, y, mean, rstd, mag): mag is the sum of the magnitudes that out is made of."""
    f = 1.0 if factor is None else factor
    z = np.zeros_like(resid if resid is not None else block)
    mag = np.zeros_like(z)
    for x, g in ((block, f), (None if bias is None else np.broadcast_to(bias, z.shape), f), (resid, 1.0)):
        if x is not None:
            # what is dropped is 0 whatever it was
            v = np.where(np.broadcast_to(g, z.shape) == 0, 0.0, x * g)
            z, mag = z + v, mag + np.abs(v)
    if w is None:
        return z, None, None, None, mag
    mean = z.mean(axis=1)
    away = z - mean[:, None]
    rstd = 1.0 / np.sqrt((away * away).mean(axis=1) + eps)
    y = away * rstd[:, None] * w + (0.0 if b is None else b)
    return z, y, mean, rstd, mag


def layer_norm_bwd(d_y, d_out, out, mean, rstd, w, factor):
    """(gradients, magnitudes of their terms): dicts with d_resid, d_block, d_bias and,
    with w, d_w and d_b."""
    f = 1.0 if factor is None else factor
    dz = np.zeros_like(d_out if d_out is not None else d_y)
    mag = np.zeros_like(dz)
    g, m = {}, {}
    if w is not None:
        hat = (out - mean[:, None]) * rstd[:, None]
        t = d_y * w
        m1, m2 = t.mean(axis=1, keepdims=True), (t * hat).mean(axis=1, keepdims=True)
        dz = rstd[:, None] * (t - m1 - hat * m2)
        mag = rstd[:, None] * (np.abs(t) + np.abs(t).mean(axis=1, keepdims=True)
                               + np.abs(hat) * np.abs(t * hat).mean(axis=1, keepdims=True))
        g["d_w"], m["d_w"] = (d_y * hat).sum(axis=0), np.abs(d_y * hat).sum(axis=0)
        g["d_b"], m["d_b"] = d_y.sum(axis=0), np.abs(d_y).sum(axis=0)
    if d_out is not None:
        dz, mag = dz + d_out, mag + np.abs(d_out)
    g["d_resid"], m["d_resid"] = dz, mag
    g["d_block"], m["d_block"] = dz * f, mag * f
    g["d_bias"], m["d_bias"] = (dz * f).sum(axis=0), (mag * f).sum(axis=0)
    return g, m


def quant(x):
    """(q, scale) of the rows of x; scale in float64."""
    top = np.abs(x).max(axis=1, initial=0.0)
    q = np.zeros(x.shape)
    scale = np.zeros(len(x))
    for i, t in enumerate(top):
        if not t < 2.0 ** 120:
            scale[i] = np.nan
        elif t >= 2.0 ** -100:
            q[i] = np.rint(127.0 * x[i] / t)     # halves to even
            scale[i] = t / 127.0
    return q, scale


def act(x, code):
    if code == 1:
        return np.maximum(x, 0)
    if code == 2:
        return 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)))
    return x / (1 + np.exp(-x)) if code == 3 else x


def gemm_i8(A, a_scale, W, w_scale, bias, code):
    """(C, value before the activation, the sum of the magnitudes it is made of)."""
    with np.errstate(invalid="ignore"):
        v = (A.astype(np.float64) @ W.astype(np.float64).T) * (a_scale[:, None] * w_scale)
        mag = np.abs(v)
        if bias is not None:
            v, mag = v + bias, mag + np.abs(bias)
        return act(v, code), v, mag
