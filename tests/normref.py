"""The norms around a block in 64 bits, from their definitions, with bounds of what fp32 arithmetic
(u = 2^-24) may be off: every function returns values and bounds of the same shapes."""
import numpy as np

U32 = 2.0 ** -24
# A thread adds up to 16 squares in turn, then 6 steps of lanes, then up to 16 waves: 38 roundings of
# terms of one sign (54 are allowed for). The mean's product, the sum with eps, the root and the division: 4 more.
SUM = 58


def rstd(v, eps):
    """1 / sqrt(mean v^2 + eps) of the rows; its relative error is half the sum's, and the last steps'."""
    return 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps), (SUM / 2 + 4) * U32


def forward(x, y, pre, post, gate, alpha, beta, eps):
    """(r, h) with their bounds; None where absent. gate: [N] or [T, 1]."""
    r, r_tol = x, 0 * x
    if y is not None:
        term, rel = beta * y, 4 * U32
        if post is not None:
            ry, e = rstd(y, eps)
            term, rel = term * ry * post, rel + e
        if gate is not None:
            term = term * gate
        r = alpha * x + term
        r_tol = 2 * U32 * np.abs(alpha * x) + rel * np.abs(term) + U32 * np.abs(r)
    if pre is None:
        return (r, r_tol), None
    rx, e = rstd(r, eps)
    e = e + np.linalg.norm(r_tol, axis=-1, keepdims=True) / np.maximum(np.linalg.norm(r, axis=-1, keepdims=True), 1e-300)
    h = r * rx * pre
    return (r, r_tol), (h, np.abs(rx * pre) * r_tol + np.abs(h) * (e + 2 * U32))


def backward(r, dh, dr, y, pre, post, gate, alpha, beta, eps):
    """dict of (value, bound): dx, dy, dgate, dpre, dpost, as far as they exist. Without y the stream r is x itself, as
    in forward, and alpha has no part in it."""
    if y is None:
        alpha = 1.0
    T, N = r.shape
    out = {}
    dR = np.zeros((T, N)) if dr is None else dr
    tol = 0 * dR
    rows = (T + 40) * U32        # a sum over rows, one after another
    if pre is not None:
        rx, e = rstd(r, eps)
        rh, z = r * rx, dh * pre
        m = (z * rh).mean(-1, keepdims=True)
        size = np.abs(z * rh).mean(-1, keepdims=True)
        n = rx * (z - rh * m)
        dR = dR + n
        # the mean of terms of both signs: SUM roundings of their absolute sum, and rx twice
        tol = rx * (np.abs(z) * (e + 4 * U32) + np.abs(rh) * size * (3 * e + (SUM + 8) * U32)) + U32 * np.abs(dR)
        out["dpre"] = (dh * rh).sum(0), (np.abs(dh * rh)).sum(0) * (rows + e + 2 * U32)
    out["dx"] = alpha * dR, abs(alpha) * tol + 2 * U32 * np.abs(alpha * dR)
    if y is None:
        return out
    ry, e = rstd(y, eps) if post is not None else (np.ones((T, 1)), 0.0)
    yh, w = y * ry, np.ones(N) if post is None else post
    g = np.ones((1, 1)) if gate is None else gate
    S, S_size = (g * dR * yh), np.abs(g * dR * yh)
    S_tol = (np.abs(g * yh) * tol).sum(0) + S_size.sum(0) * (rows + e + 4 * U32)
    if gate is not None and gate.ndim == 1:
        S, S_tol = (dR * yh), (np.abs(yh) * tol).sum(0) + np.abs(dR * yh).sum(0) * (rows + e + 4 * U32)
        out["dgate"] = beta * w * S.sum(0), np.abs(beta * w) * S_tol + 3 * U32 * np.abs(beta * w * S.sum(0))
        S, S_tol = S * gate, S_tol * np.abs(gate)
    elif gate is not None:
        t, size = beta * (dR * yh * w), np.abs(beta * dR * yh * w).sum(-1, keepdims=True)
        t_tol = np.abs(beta * yh * w * tol).sum(-1, keepdims=True)
        out["dgate"] = t.sum(-1, keepdims=True), t_tol + size * (e + (SUM + 6) * U32)
    if post is not None:
        out["dpost"] = beta * S.sum(0), abs(beta) * S_tol + 3 * U32 * np.abs(beta * S.sum(0))
    v, v_tol = beta * g * w * dR, np.abs(beta * g * w) * tol + 5 * U32 * np.abs(beta * g * w * dR)
    if post is None:
        out["dy"] = v, v_tol + U32 * np.abs(v)
        return out
    m, size = (v * yh).mean(-1, keepdims=True), np.abs(v * yh).mean(-1, keepdims=True)
    m_tol = size * (e + (SUM + 8) * U32) + np.abs(yh * v_tol).mean(-1, keepdims=True)
    dy = ry * (v - yh * m)
    out["dy"] = dy, ry * (v_tol + np.abs(yh) * m_tol + (np.abs(v) + np.abs(yh * m)) * (2 * e + 4 * U32))
    return out
