"""Plain 64-bit references of the row operators (routing, sorting, combining,
adapters) in numpy, written from their definitions with loops over tokens where
that is the clearest form. Quantisation itself is the oracle's."""
import numpy as np


def route(l, k, score, bias=None, renorm=False, scale=1.0):
    """(ids, w, s) of logits l [T, E]; ids from the 64-bit ranks, ties to the lower index."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    ok = l > -np.inf
    s = np.zeros((T, E))
    for t in range(T):
        if not ok[t].any():
            continue
        if score == "softmax":
            e = np.where(ok[t], np.exp(np.where(ok[t], l[t], 0) - l[t][ok[t]].max()), 0.0)
            s[t] = e / e.sum()
        else:
            s[t] = np.where(ok[t], 1 / (1 + np.exp(-np.where(ok[t], l[t], 0))), 0.0)
    rank = np.where(ok, l if bias is None else s + np.asarray(bias, np.float64), -np.inf)
    rank = np.where(rank > -np.inf, rank, -np.inf)
    order = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    there = np.take_along_axis(rank, order, 1) > -np.inf
    ids = np.where(there, order, -1)
    return ids, weights(s, ids, renorm, scale), s


def weights(s, ids, renorm, scale):
    c = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        total = c.sum(1, keepdims=True)
        c = np.divide(c, total, out=np.zeros_like(c), where=total > 0)
    return scale * c


def route_grad(s, ids, dw, score, renorm, scale):
    """dlogits by the chain rule: w -> chosen scores -> logits, one token at a time."""
    T, E = s.shape
    out = np.zeros((T, E))
    for t in range(T):
        j = ids[t][ids[t] >= 0]
        g = scale * np.asarray(dw[t], np.float64)[ids[t] >= 0]
        c = s[t, j]
        if renorm:
            total = c.sum()
            g = (g - (g * c).sum() / total) / total if total > 0 else np.zeros_like(g)
        ds = np.zeros(E)
        ds[j] = g
        if score == "softmax":
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        else:
            out[t] = ds * s[t] * (1 - s[t])
    return out


def plan_contiguous(ids, G, align, cap):
    """(rows, slots, m_indices, offsets) by walking the slots once."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    counts = np.array([(flat == g).sum() for g in range(G)])
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    rows, slots, m = np.full(flat.size, -1), np.full(cap, -1), np.full(cap, -1)
    at = offsets[:-1].copy()
    for s, g in enumerate(flat):
        if 0 <= g < G:
            rows[s], slots[at[g]], m[at[g]] = at[g], s, g
            at[g] += 1
    return rows.reshape(ids.shape), slots, m, offsets


def plan_masked(ids, G, M_max):
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    rows, slots, n = np.full(flat.size, -1), np.full(G * M_max, -1), np.zeros(G, np.int64)
    for s, g in enumerate(flat):
        if 0 <= g < G and n[g] < M_max:
            rows[s] = g * M_max + n[g]
            slots[rows[s]] = s
            n[g] += 1
    return rows.reshape(ids.shape), slots, n


def combine(y, rows, w=None, base=None):
    """(out, sum of the terms' absolute values) in 64 bits."""
    T, k = rows.shape
    y = y.reshape(-1, y.shape[-1])
    out = np.zeros((T, y.shape[1])) if base is None else np.array(base, np.float64)
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                term = (1.0 if w is None else float(w[t, j])) * y[rows[t, j]].astype(np.float64)
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def adapters(D, x, A, B, scales, ids):
    """(out, h bound, delta bound): the bounds are the same sums with absolute values."""
    out = np.array(D, np.float64)
    h_size = np.zeros((D.shape[0], A.shape[1]))
    d_size = np.zeros(out.shape)
    for t, a in enumerate(ids):
        if 0 <= a < A.shape[0]:
            h = A[a].astype(np.float64) @ x[t].astype(np.float64)
            h_size[t] = np.abs(A[a]).astype(np.float64) @ np.abs(x[t]).astype(np.float64)
            out[t] += float(scales[a]) * (B[a].astype(np.float64) @ h)
            d_size[t] = abs(float(scales[a])) * (np.abs(B[a]).astype(np.float64) @ h_size[t])
    return out, d_size
