"""Plain float64 definitions of the operators around a sparse block: router and
balance loss, norms with gate and residual, 4-bit weights.  Numpy loops and sums
only; shares no code with the HIP library.  ``tests/test_block_cpu.py`` checks the
gradients against differences and the packing against hand-written bytes."""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def _log_sigmoid(x):
    return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))


def _softmax_row(u):
    """Softmax of one row; zeros where every entry is -inf."""
    m = u.max(initial=-np.inf)
    if m == -np.inf:
        return np.zeros_like(u)
    e = np.exp(u - m)
    return e / e.sum()


def gate(x, topk, score, renorm, scale, bias=None, mask=None):
    """(ids, weights, counts [E + 1], prob_sums, loss) of logits x [T, E] (float64)."""
    T, E = x.shape
    ids = np.full((T, topk), -1, np.int64)
    w = np.zeros((T, topk))
    sums = np.zeros(E)
    n = 0
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        n += 1
        u = x[t] if score == SOFTMAX else _log_sigmoid(x[t])
        share = _softmax_row(u)
        sc = share if score == SOFTMAX else _sigmoid(x[t])
        sums += share
        key = x[t] if bias is None else np.where(x[t] == -np.inf, -np.inf, sc + bias)
        order = sorted(range(E), key=lambda e: (-key[e], e))[:topk]
        for k, e in enumerate(order):
            if key[e] > -np.inf:
                ids[t, k] = e
        sel = ids[t][ids[t] >= 0]
        w[t, :len(sel)] = scale * (_softmax_row(u[sel]) if renorm else sc[sel])
    counts = np.array([(ids == e).sum() for e in range(E)] + [n], np.int64)
    loss = E / (topk * float(max(n, 1)) ** 2) * float((counts[:E] * sums).sum())
    return ids, w, counts, sums, loss


def gate_objective(x, ids, score, renorm, scale, mask, d_w, counts, d_loss):
    """sum(weights * d_w) + loss * d_loss with ids and counts held fixed."""
    T, E = x.shape
    total, sums = 0.0, np.zeros(E)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        u = x[t] if score == SOFTMAX else _log_sigmoid(x[t])
        share = _softmax_row(u)
        sums += share
        sc = share if score == SOFTMAX else _sigmoid(x[t])
        k = [i for i, e in enumerate(ids[t]) if 0 <= e < E]
        sel = ids[t][k]
        w = _softmax_row(u[sel]) if renorm else sc[sel]
        if d_w is not None:
            total += scale * float((w * d_w[t][k]).sum())
    if counts is not None and counts[E] > 0:
        total += d_loss * E / (ids.shape[1] * float(counts[E]) ** 2) * float((counts[:E] * sums).sum())
    return total


def gate_bwd(x, ids, score, renorm, scale, mask=None, d_w=None, counts=None, d_loss=0.0):
    """(d_logits, bound): the gradient, and the sum of the magnitudes that it is
    made of, which the rounding error is relative to."""
    T, E = x.shape
    dx, mag = np.zeros((T, E)), np.zeros((T, E))
    a = np.zeros(E)
    if counts is not None and counts[E] > 0:
        a = d_loss * E / (ids.shape[1] * float(counts[E]) ** 2) * counts[:E].astype(np.float64)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        u = x[t] if score == SOFTMAX else _log_sigmoid(x[t])
        p = _softmax_row(u)
        du = p * (a - (p * a).sum())
        m = p * (np.abs(a) + (p * np.abs(a)).sum())
        if d_w is not None:
            k = [i for i, e in enumerate(ids[t]) if 0 <= e < E]
            sel, d = ids[t][k], scale * d_w[t][k]
            if renorm:
                q = _softmax_row(u[sel])
                np.add.at(du, sel, q * (d - (q * d).sum()))
                np.add.at(m, sel, q * (np.abs(d) + (q * np.abs(d)).sum()))
            else:
                w = p[sel] if score == SOFTMAX else _sigmoid(x[t][sel])
                np.add.at(du, sel, w * d)
                np.add.at(m, sel, w * np.abs(d))
                if score == SOFTMAX:
                    du -= p * (w * d).sum()
                    m += p * (w * np.abs(d)).sum()
        f = 1.0 if score == SOFTMAX else _sigmoid(-x[t])
        dx[t], mag[t] = du * f, m * f
    return dx, mag


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def _rows(g, M):
    return np.repeat(g, M // g.shape[0], axis=0)


def norm(block, resid, w_post, w_pre, gate, scale, eps):
    """(out, y, rstd_post, rstd_pre, magnitude of out's terms), None where absent."""
    M = (block if block is not None else resid).shape[0]
    out = np.zeros((block if block is not None else resid).shape)
    mag = np.zeros_like(out)
    rq = rp = y = None
    if block is not None:
        b = block
        if w_post is not None:
            rq = _rstd(block, eps)
            b = block * rq[:, None] * w_post
        if gate is not None:
            b = b * _rows(gate, M)
        out = out + scale * b
        mag = mag + np.abs(scale * b)
    if resid is not None:
        out, mag = out + resid, mag + np.abs(resid)
    if w_pre is not None:
        rp = _rstd(out, eps)
        y = out * rp[:, None] * w_pre
    return out, y, rq, rp, mag


def norm_bwd(d_y, d_out, out, block, w_post, w_pre, gate, scale, rstd_post, rstd_pre):
    """(gradients, magnitudes): dicts of d_resid, d_block, d_w_post, d_w_pre, d_gate."""
    like = d_y if d_y is not None else d_out
    M, N = like.shape
    g, mag = {}, {}
    dz = d_out.copy() if d_out is not None else np.zeros((M, N))
    m = np.abs(dz)
    if w_pre is not None:
        r = rstd_pre[:, None]
        hat, t = out * r, d_y * w_pre
        dz = dz + r * (t - hat * (t * hat).mean(axis=1, keepdims=True))
        m = m + r * (np.abs(t) + np.abs(hat) * np.abs(t * hat).mean(axis=1, keepdims=True))
        g["d_w_pre"], mag["d_w_pre"] = (d_y * hat).sum(axis=0), np.abs(d_y * hat).sum(axis=0)
    g["d_resid"], mag["d_resid"] = dz, m
    r = rstd_post[:, None] if w_post is not None else 1.0
    hat = block * r if block is not None else np.zeros((M, N))
    nrm = hat * w_post if w_post is not None else hat
    d, m = dz * scale, m * abs(scale)
    if gate is not None:
        G = gate.shape[0]
        g["d_gate"] = (d * nrm).reshape(G, M // G, N).sum(axis=1)
        mag["d_gate"] = (m * np.abs(nrm)).reshape(G, M // G, N).sum(axis=1)
        d, m = d * _rows(gate, M), m * np.abs(_rows(gate, M))
    if w_post is not None:
        g["d_w_post"], mag["d_w_post"] = (d * hat).sum(axis=0), (m * np.abs(hat)).sum(axis=0)
        t, mt = d * w_post, m * np.abs(w_post)
        d = r * (t - hat * (t * hat).mean(axis=1, keepdims=True))
        m = r * (mt + np.abs(hat) * (mt * np.abs(hat)).mean(axis=1, keepdims=True))
    g["d_block"], mag["d_block"] = d, m
    return g, mag


def w4_pack(codes):
    """Packed bytes [N, 64 * ceil(K / 128)] of codes [K, N], one code at a time."""
    K, N = codes.shape
    blocks = -(-K // 128)
    words = np.zeros((N, blocks, 16), np.uint32)
    for k in range(K):
        blk, r = divmod(k, 128)
        j, r = divmod(r, 32)
        q, o = divmod(r, 8)
        p = o // 2 + (4 if o % 2 else 0)
        words[:, blk, 4 * q + j] |= (codes[k].astype(np.uint32) & 15) << np.uint32(4 * p)
    return words.reshape(N, -1).astype("<u4").view(np.uint8).reshape(N, -1)


def w4_matrix(codes, scales, zeros, group):
    """W [K, N] in float64."""
    g = np.arange(codes.shape[0]) // group
    z = zeros[g].astype(np.float64) if zeros is not None else 8.0
    return (codes.astype(np.float64) - z) * scales[g]
