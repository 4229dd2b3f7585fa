"""fp64 CPU oracle of the loss, the embedding and the residual norm, with their
gradients (test infrastructure only).  Plain NumPy from the definitions in
include/dllm_loss.h, dllm_embed.h and dllm_norm.h, on fp64 copies of the bf16
inputs; nothing in between is rounded.  Each gradient comes with the scale of
the rounding errors in its terms where a test needs it."""
from __future__ import annotations

import numpy as np


def counted(mask, targets, V):
    """Positions that count, ascending."""
    t = np.asarray(targets).astype(np.int64)
    return np.nonzero((np.asarray(mask) != 0) & (t >= 0) & (t < V))[0]


def loss(W, H, mask, targets, weights=None, grad=1.0):
    """A dict of fp64 arrays: loss, losses [L], lse [L], d_hidden [L, d], d_W
    [V, d], the rows' dz [M, V], p [M, V] and idx [M]."""
    V, L = W.shape[0], H.shape[0]
    idx = counted(mask, targets, V)
    t = np.asarray(targets)[idx].astype(np.int64)
    w = np.ones(L) if weights is None else np.asarray(weights, dtype=np.float64)
    z = H[idx] @ W.T
    top = z.max(axis=1, keepdims=True) if len(idx) else z[:, :1]
    lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
    p = np.exp(z - lse[:, None])
    hot = np.zeros_like(p)
    hot[np.arange(len(idx)), t] = 1.0
    dz = (grad * w[idx])[:, None] * (p - hot)
    losses, full = np.zeros(L), np.zeros(L)
    losses[idx] = lse - z[np.arange(len(idx)), t]
    full[idx] = lse
    dH = np.zeros(H.shape)
    dH[idx] = dz @ W
    return dict(loss=float((w * losses).sum()), losses=losses, lse=full, d_hidden=dH, d_W=dz.T @ H[idx], dz=dz, p=p, idx=idx)


def lookup(table, tokens, scale=1.0):
    V = table.shape[0]
    tok = np.asarray(tokens).astype(np.int64)
    ok = (tok >= 0) & (tok < V)
    return np.where(ok[:, None], scale * table[np.where(ok, tok, 0)], 0.0)


def lookup_grad(tokens, d_out, V, scale=1.0):
    """(gradient [V, d], the sums of its terms' absolute values)."""
    g, size = np.zeros((V, d_out.shape[1])), np.zeros((V, d_out.shape[1]))
    for t, tok in enumerate(np.asarray(tokens).astype(np.int64)):
        if 0 <= tok < V:
            g[tok] += scale * d_out[t]
            size[tok] += np.abs(scale * d_out[t])
    return g, size


def rms(v, eps):
    """sqrt(mean(v^2) + eps) by row."""
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate_rows(gate, T):
    return np.ones((T, 1)) if gate is None else np.repeat(gate, T // gate.shape[0], axis=0)


def residual_norm(x, y, pre, post, gate, eps, scale):
    """(x', n, the size of the terms of x'); y, pre, post and gate may be None."""
    size = np.abs(x)
    if y is not None:
        u = y if post is None else post * y / rms(y, eps)
        step = scale * _gate_rows(gate, len(x)) * u
        x, size = x + step, size + np.abs(step)
    return x, None if pre is None else pre * x / rms(x, eps), size


def residual_norm_grad(x, y, pre, post, gate, eps, scale, d_n, d_x):
    """Gradients at the stream x behind the update.  A dict of (gradient, size
    of its terms) for x, y, pre, post and gate; None for what is not there."""
    T, d = x.shape
    out = dict(x=None, y=None, pre=None, post=None, gate=None)
    dx, size = (np.zeros_like(x), np.zeros_like(x)) if d_x is None else (d_x, np.abs(d_x))
    if d_n is not None:
        r = 1.0 / rms(x, eps)
        D = d_n * pre
        dx = dx + r * (D - x * r * r * (D * x).mean(axis=1, keepdims=True))
        size = size + r * (np.abs(D) + np.abs(x) * r * r * np.abs(D * x).mean(axis=1, keepdims=True))
        out["pre"] = (d_n * x * r).sum(axis=0), np.abs(d_n * x * r).sum(axis=0)
    out["x"] = dx, size
    if y is not None:
        q = np.ones((T, 1)) if post is None else 1.0 / rms(y, eps)
        yq = y * q
        u = yq if post is None else yq * post
        g = _gate_rows(gate, T)
        if gate is not None:
            by_run = lambda v: v.reshape(gate.shape[0], -1, d).sum(axis=1)  # noqa: E731
            out["gate"] = by_run(scale * dx * u), by_run(abs(scale) * size * np.abs(u))
        du, ds = scale * g * dx, abs(scale) * np.abs(g) * size
        if post is not None:
            out["post"] = (du * yq).sum(axis=0), (ds * np.abs(yq)).sum(axis=0)
            E, Es = du * post, ds * np.abs(post)
            du = q * (E - y * q * q * (E * y).mean(axis=1, keepdims=True))
            ds = q * (Es + np.abs(y) * q * q * (Es * np.abs(y)).mean(axis=1, keepdims=True))
        out["y"] = du, ds
    return out
