"""The selective state space scan, the short causal convolution and the
root-mean-square norm in fp64, token after token, with their gradients.

    dt = softplus(delta + bias),  h_n = exp(dt A_n) h_n + dt u B_n
    y = (sum_n C_n h_n + skip u) silu(z)

    c_t = bias + sum_j w_j x_{t-K+1+j},  y = silu(c)

    t = x + r,  y = t / sqrt(mean(t^2) + eps) w

Arrays are NumPy, [B,T,D] and [B,T,G,N].  ``magnitudes`` of a call is the same
computation on the sizes of all terms (nothing cancels), which rounding errors are
measured against.
"""

from __future__ import annotations

import numpy as np


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def _spread(x, D):
    """[B,G,N] to the channels."""
    return np.repeat(x, D // x.shape[1], axis=1)


def _per_group(x, G):
    """Sums over the channels of each group: [B,D,N] -> [B,G,N]."""
    return x.reshape(x.shape[0], G, -1, x.shape[2]).sum(2)


def selective(u, delta, A, B, C, skip=None, z=None, bias=None, softplus_on=True, h0=None, lengths=None, dy=None, dh_last=None,
              magnitudes=False):
    """y, h_last and, with ``dy``, a dict of gradients."""
    size = np.abs if magnitudes else (lambda v: v)
    nb, T, D = u.shape
    G, N = B.shape[2:]
    n = np.full(nb, T) if lengths is None else np.clip(lengths, 0, T)
    seen = np.arange(T)[None] < n[:, None]
    u, delta, B, C = (np.where(seen.reshape(nb, T, *[1] * (v.ndim - 2)), v, 0.0) for v in (u, delta, B, C))
    x = delta + (0.0 if bias is None else bias)
    dt = softplus(x) if softplus_on else x
    ddt_dx = sigmoid(x) if softplus_on else np.ones_like(x)
    u, B, C = size(u), size(B), size(C)
    skip = np.zeros(D) if skip is None else size(skip)
    h = np.zeros((nb, D, N)) if h0 is None else size(h0).copy()
    states = [h]
    s = np.zeros((nb, T, D))
    for t in range(T):
        a = np.exp(dt[:, t, :, None] * A)
        new = a * h + size(dt[:, t] * u[:, t])[..., None] * _spread(B[:, t], D)
        h = np.where(seen[:, t, None, None], new, h)
        states.append(h)
        s[:, t] = (h * _spread(C[:, t], D)).sum(2) + skip * u[:, t]
    zz = None if z is None else np.where(seen[..., None], z, 0.0)
    gate = np.ones_like(u) if z is None else size(zz * sigmoid(zz))
    y = s * gate * seen[..., None]
    if dy is None:
        return y, h
    dy = size(np.where(seen[..., None], dy, 0.0))
    ds = dy * gate
    g = np.zeros_like(h) if dh_last is None else size(dh_last).copy()
    out = {"du": skip * ds, "ddelta": np.zeros_like(u), "dB": np.zeros_like(B), "dC": np.zeros_like(C), "dA": np.zeros((D, N)),
           "dskip": (ds * u).sum((0, 1))}
    for t in reversed(range(T)):
        on = seen[:, t, None, None]
        a = np.exp(dt[:, t, :, None] * A)
        full = g + ds[:, t, :, None] * _spread(C[:, t], D)
        out["dC"][:, t] = _per_group(ds[:, t, :, None] * states[t + 1], G)
        out["dB"][:, t] = _per_group(on * full * size(dt[:, t] * u[:, t])[..., None], G)
        through = (on * full * _spread(B[:, t], D)).sum(2)
        q = on * full * a * states[t]
        out["du"][:, t] += size(dt[:, t]) * through
        out["ddelta"][:, t] = (u[:, t] * through + (q * size(A)).sum(2)) * ddt_dx[:, t]
        out["dA"] += (q * size(dt[:, t])[..., None]).sum(0)
        g = np.where(on, full * a, g)
    out["dbias"] = out["ddelta"].sum((0, 1))
    out["dh0"] = g
    if z is not None:
        p = sigmoid(zz)
        # silu' = p + p z (1 - p) has a zero at z = -1.278, where its two terms cancel
        out["dz"] = dy * s * (p + p * size(zz) * (1 - p))
    return y, h, out


def conv(x, w, bias=None, silu=True, state=None, lengths=None, dy=None, dlast=None, magnitudes=False):
    """y, the state behind the sequences and, with ``dy``, a dict of gradients."""
    size = np.abs if magnitudes else (lambda v: v)
    nb, T, D = x.shape
    K = w.shape[1]
    n = np.full(nb, T) if lengths is None else np.clip(lengths, 0, T)
    seen = (np.arange(T)[None] < n[:, None])[..., None]
    x = np.where(seen, x, 0.0)
    front = np.zeros((nb, K - 1, D)) if state is None else state
    line = np.concatenate([front, x], 1)
    c = np.zeros((nb, T, D)) + (0.0 if bias is None else bias)
    sizes = np.abs(c)   # of the terms of c, which an error of c goes by
    for j in range(K):
        c = c + line[:, j:j + T] * w[:, j]
        sizes = sizes + np.abs(line[:, j:j + T] * w[:, j])
    p = sigmoid(c)
    y = (c * p if silu else c) * seen
    last = np.stack([line[b, n[b]:n[b] + K - 1] for b in range(nb)]) if nb else np.zeros((0, K - 1, D))
    if magnitudes:
        y = sizes * seen
    if dy is None:
        return y, last
    slope = p * (1 + c * (1 - p)) if silu else np.ones_like(c)
    if magnitudes:
        slope = 1.2 + sizes   # |silu'| stays below 1.1, |silu''| below 1
    dc = size(np.where(seen, dy, 0.0)) * slope
    dline = np.zeros((nb, T + K - 1, D))
    if dlast is not None:
        for b in range(nb):
            dline[b, n[b]:n[b] + K - 1] += size(dlast[b])
    dw = np.zeros((D, K))
    for j in range(K):
        dline[:, j:j + T] += dc * size(w[:, j])
        dw[:, j] = (dc * size(line[:, j:j + T])).sum((0, 1))
    return y, last, {"dx": dline[:, K - 1:], "dw": dw, "dbias": dc.sum((0, 1)), "dstate": dline[:, :K - 1]}


def norm(t, w, eps, dy=None, dtotal=None, magnitudes=False):
    """y of the rows of t and, with ``dy``, (dx, dw)."""
    size = np.abs if magnitudes else (lambda v: v)
    rms = np.sqrt((t * t).mean(1, keepdims=True) + eps)
    n = size(t) / rms
    if dy is None:
        return n * size(w)
    g = size(dy) * size(w)
    back = n * (g * n).mean(1, keepdims=True)
    dx = (g + back if magnitudes else g - back) / rms + (0.0 if dtotal is None else size(dtotal))
    return n * size(w), dx, (size(dy) * n).sum(0)
