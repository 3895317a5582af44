"""fp64 reference of the gated linear recurrence and the layer norm (numpy).

Plain loops over the definitions, vectorised over channels only; see the
entry points' comments in ``include/ssmscan.h`` for the formulas.
"""
import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def gate_terms(r, i, A):
    """s, g, u, a, m of the recurrence for r, i [..., Dm] and A [Dm]."""
    s, g = sigmoid(_f64(r)), sigmoid(_f64(i))
    u = _f64(A) * s
    return s, g, u, np.exp(u), np.sqrt(-np.expm1(2.0 * u))


def gated_row(x, r, i, A, h0):
    """States [L, Dm] of one sequence started from h0 [Dm]."""
    _, g, _, a, m = gate_terms(r, i, A)
    b = m * g * _f64(x)
    h = np.empty_like(b)
    c = _f64(h0).copy()
    for t in range(b.shape[0]):
        c = a[t] * c + b[t]
        h[t] = c
    return h


def gated_row_bwd(x, r, i, A, h0, dy, dhf):
    """dx, dr, di [L, Dm], dA [Dm] and dh_init [Dm] of one sequence."""
    x, dy, A = _f64(x), _f64(dy), _f64(A)
    s, g, _, a, m = gate_terms(r, i, A)
    h = gated_row(x, r, i, A, h0)
    before = np.concatenate([_f64(h0)[None], h[:-1]]) if len(h) else h
    lam = np.empty_like(x)
    e = _f64(dhf).copy()
    for t in range(x.shape[0] - 1, -1, -1):
        lam[t] = dy[t] + e
        e = a[t] * lam[t]
    q = np.divide(g * x * a * a, m, out=np.zeros_like(m), where=m > 0)
    du = lam * (a * before - q)
    return {"dx": lam * m * g, "dr": du * A * s * (1 - s), "di": lam * m * x * g * (1 - g), "dA": (du * s).sum(0),
            "dh_init": e}


def gated(x, r, i, A, h0=None, cu=None):
    """(y, h_final) of a dense batch [B, L, Dm], or of packed rows [L, Dm]."""
    parts, rows = _parts(x, cu)
    h0 = np.zeros((rows, np.shape(A)[0])) if h0 is None else _f64(h0)
    y = np.empty(np.shape(x))
    hf = h0.copy()
    for k, at in enumerate(parts):
        h = gated_row(x[at], r[at], i[at], A, h0[k])
        y[at] = h
        if len(h):
            hf[k] = h[-1]
    return y, hf


def gated_bwd(x, r, i, A, dy, h0=None, dhf=None, cu=None):
    parts, rows = _parts(x, cu)
    z = np.zeros((rows, np.shape(A)[0]))
    h0 = z if h0 is None else _f64(h0)
    dhf = z if dhf is None else _f64(dhf)
    out = {k: np.empty(np.shape(x)) for k in ("dx", "dr", "di")}
    out["dA"], out["dh_init"] = np.zeros(np.shape(A)[0]), dhf.copy()
    for k, at in enumerate(parts):
        if x[at].shape[0] == 0:
            continue
        g = gated_row_bwd(x[at], r[at], i[at], A, h0[k], dy[at], dhf[k])
        for name in ("dx", "dr", "di"):
            out[name][at] = g[name]
        out["dA"] += g["dA"]
        out["dh_init"][k] = g["dh_init"]
    return out


def _parts(x, cu):
    if cu is None:
        return [(k,) for k in range(len(x))], len(x)
    return [(slice(int(cu[k]), int(cu[k + 1])),) for k in range(len(cu) - 1)], len(cu) - 1


def layer_norm(s, weight=None, bias=None, group=None, eps=1e-5):
    """(y, mean, rstd) of rows s [rows, Dm] normalised by groups."""
    s = _f64(s)
    rows, Dm = s.shape
    P = group or Dm
    v = s.reshape(rows, Dm // P, P)
    mean = v.mean(axis=2)
    rstd = 1.0 / np.sqrt(((v - mean[..., None]) ** 2).mean(axis=2) + eps)
    y = ((v - mean[..., None]) * rstd[..., None]).reshape(rows, Dm)
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def layer_norm_bwd(s, weight, mean, rstd, dy, dsum=None, group=None):
    """dx, dweight, dbias for given statistics [rows, Dm / group]."""
    s, dy, mean, rstd = _f64(s), _f64(dy), _f64(mean), _f64(rstd)
    rows, Dm = s.shape
    P = group or Dm
    v = s.reshape(rows, Dm // P, P)
    z = (v - mean[..., None]) * rstd[..., None]
    q = (dy if weight is None else dy * _f64(weight)).reshape(v.shape)
    dx = rstd[..., None] * (q - q.mean(2, keepdims=True) - z * (q * z).mean(2, keepdims=True))
    dx = dx.reshape(rows, Dm)
    if dsum is not None:
        dx = dx + _f64(dsum)
    return {"dx": dx, "dweight": (dy * z.reshape(rows, Dm)).sum(0), "dbias": dy.sum(0)}
