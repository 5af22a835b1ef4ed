"""The bf16 training operators in float64 -- test infrastructure, see
``oracle/__init__``: the norms around a block with its gate and residual scale,
the grouped products, the gated activation, and the gradient norm with
clipping, each with its backward pass written out from the forward formula.

Every function returns float64 arrays, unrounded, and where it says so the
magnitudes that an error bound of a float32 evaluation is built from."""
import numpy as np


def _as2(gate, T, H):
    """The gate broadcast to [T, H]."""
    if gate is None:
        return np.ones((T, H))
    g = np.asarray(gate, np.float64)
    return np.broadcast_to(g if g.ndim == 2 else g[None, :], (T, H))


def inv_rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def block_norm(x, b, w_pre, w_post, gate, alpha, beta, eps):
    """Returns (r, h or None, |terms of r|)."""
    if b is None:
        r, mag = x, np.abs(x)
    else:
        n = b if w_post is None else b * inv_rms(b, eps) * w_post
        t = beta * _as2(gate, *b.shape) * n
        r, mag = alpha * x + t, np.abs(alpha * x) + np.abs(t)
    h = None if w_pre is None else r * inv_rms(r, eps) * w_pre
    return r, h, mag


def block_norm_backward(r, dr, dh, b, w_pre, w_post, gate, alpha, beta, eps):
    """Gradients of block_norm, with r taken as stored.  Returns a dict of the
    gradients and, under "mag", the sums of the magnitudes of their terms."""
    T, H = r.shape
    out, mag = {}, {}
    d, dmag = np.zeros((T, H)), np.zeros((T, H))
    if dr is not None:
        d, dmag = d + dr, dmag + np.abs(dr)
    if dh is not None:
        ir = inv_rms(r, eps)
        rh = r * ir
        v = dh * w_pre
        d = d + ir * (v - rh * (v * rh).mean(1, keepdims=True))
        dmag = dmag + ir * (np.abs(v) + np.abs(rh) * np.abs(v * rh).mean(1, keepdims=True))
        out["dw_pre"], mag["dw_pre"] = (dh * rh).sum(0), np.abs(dh * rh).sum(0)
    if b is None:
        out["dx"], mag["dx"] = d, dmag
        return out | {"mag": mag}
    out["dx"], mag["dx"] = alpha * d, abs(alpha) * dmag
    g = _as2(gate, T, H)
    ib = inv_rms(b, eps) if w_post is not None else np.ones((T, 1))
    bh = b * ib
    w = w_post if w_post is not None else np.ones(H)
    dn, nmag = beta * g * d, abs(beta) * np.abs(g) * dmag
    if w_post is not None:
        u, umag = dn * w, nmag * np.abs(w)
        out["dw_post"], mag["dw_post"] = (dn * bh).sum(0), np.abs(nmag * bh).sum(0)
        out["db"] = ib * (u - bh * (u * bh).mean(1, keepdims=True))
        mag["db"] = ib * (umag + np.abs(bh) * np.abs(umag * bh).mean(1, keepdims=True))
    else:
        out["db"], mag["db"] = dn, nmag
    if gate is not None:
        e, emag = beta * d * bh * w, abs(beta) * dmag * np.abs(bh * w)
        axis = 0 if np.ndim(gate) == 1 else (1 if np.shape(gate)[1] == 1 else None)
        if axis is None:
            out["dgate"], mag["dgate"] = e, emag
        else:
            keep = axis == 1
            out["dgate"] = e.sum(axis, keepdims=keep)
            mag["dgate"] = emag.sum(axis, keepdims=keep)
    return out | {"mag": mag}


def _rows_of(m, index, lo, hi):
    return m[lo:hi] if index is None else m[index[lo:hi]]


def grouped_gemm(a, b, offsets, index=None, row_scale=None, kn=False):
    """Returns (out, sum of |products|)."""
    R = int(offsets[-1])
    n = b.shape[2] if kn else b.shape[1]
    out, mag = np.zeros((R, n)), np.zeros((R, n))
    for g in range(len(offsets) - 1):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if hi > lo:
            w = b[g] if kn else b[g].T
            rows = _rows_of(a, index, lo, hi)
            out[lo:hi], mag[lo:hi] = rows @ w, np.abs(rows) @ np.abs(w)
    if row_scale is not None:
        out, mag = out * row_scale[:, None], mag * np.abs(row_scale)[:, None]
    return out, mag


def grouped_wgrad(a, b, offsets, a_index=None, b_index=None):
    """Returns (out [G, n, k], sum of |products|)."""
    G = len(offsets) - 1
    out = np.zeros((G, a.shape[1], b.shape[1]))
    mag = np.zeros_like(out)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        x, y = _rows_of(a, a_index, lo, hi), _rows_of(b, b_index, lo, hi)
        out[g], mag[g] = x.T @ y, np.abs(x).T @ np.abs(y)
    return out, mag


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu(a):
    I = a.shape[1] // 2
    g, u = a[:, :I], a[:, I:]
    return g * sigmoid(g) * u


def swiglu_backward(a, dh, row_gate=None):
    """Gradients of row_gate * swiglu(a).  Returns (da, dgate, hg, sum of
    |terms of dgate|)."""
    I = a.shape[1] // 2
    g, u = a[:, :I], a[:, I:]
    s = sigmoid(g)
    silu = g * s
    w = np.ones((a.shape[0], 1)) if row_gate is None else np.asarray(row_gate)[:, None]
    h = silu * u
    da = np.concatenate([w * dh * u * (s + silu * (1 - s)), w * dh * silu], 1)
    return da, (h * dh).sum(1), w * h, np.abs(h * dh).sum(1)


def clip(grads, max_norm):
    """Returns (norm, coef)."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    if not np.isfinite(norm):
        return norm, 1.0
    return norm, min(1.0, max_norm / (norm + 1e-6))
