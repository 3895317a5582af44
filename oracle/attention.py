"""fp64 reference of linear attention with a decay per head, and of the norm and
rotation of queries and keys (numpy).

Plain loops over the definitions, vectorised over heads and values only; see
the entry points' comments in ``include/ssmscan.h`` for the formulas.
"""
import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def spread(t, H):
    """[..., Hkv, D] with every head repeated for the heads of q that share it."""
    return np.repeat(_f64(t), H // t.shape[-2], axis=-2)


def gather(t, Hkv):
    """The sum over the heads of q that share a head: [..., H, D] -> [..., Hkv, D]."""
    return t.reshape(*t.shape[:-2], Hkv, t.shape[-2] // Hkv, t.shape[-1]).sum(-2)


def parts(L, cu, Bsz):
    """(index of the sequence's steps, its state row) of every sequence."""
    if cu is None:
        return [((b, slice(0, L)), b) for b in range(Bsz)]
    return [((slice(int(cu[k]), int(cu[k + 1])),), k) for k in range(len(cu) - 1)]


def linear_row(q, k, v, lam, h0, scale):
    """One sequence: q [L, H, Dk], k [L, H, Dk], v [L, H, Dv], h0 [H, Dv, Dk]."""
    h = _f64(h0).copy()
    y = np.empty((len(q), *v.shape[1:]))
    for t in range(len(q)):
        h = lam[:, None, None] * h + v[t][:, :, None] * k[t][:, None, :]
        y[t] = scale * np.einsum("hvk,hk->hv", h, q[t])
    return y, h


def linear_row_bwd(q, k, v, lam, h0, scale, dy, dhf):
    """dq, dk, dv (per head of q) and dh_init of one sequence."""
    L = len(q)
    h, before = _f64(h0).copy(), []
    for t in range(L):
        h = lam[:, None, None] * h + v[t][:, :, None] * k[t][:, None, :]
        before.append(h)
    g = _f64(dhf).copy()
    dq, dk, dv = np.empty_like(q), np.empty_like(k), np.empty_like(v)
    for t in range(L - 1, -1, -1):
        g = g + scale * dy[t][:, :, None] * q[t][:, None, :]
        dq[t] = scale * np.einsum("hvk,hv->hk", before[t], dy[t])
        dk[t] = np.einsum("hvk,hv->hk", g, v[t])
        dv[t] = np.einsum("hvk,hk->hv", g, k[t])
        g = lam[:, None, None] * g
    return dq, dk, dv, g


def linear_attn(q, k, v, log_decay, scale, h0=None, cu=None, dy=None, dhf=None):
    """{"y", "h_final"} and, with dy, {"dq", "dk", "dv", "dh_init"}: dense
    [B, L, H, D] or packed [L, H, D] tensors."""
    q = _f64(q)
    H, Hkv = q.shape[-2], k.shape[-2]
    kk, vv, lam = spread(k, H), spread(v, H), np.exp(_f64(log_decay))
    rows = q.shape[0] if cu is None else len(cu) - 1
    at = parts(q.shape[-3], cu, rows)
    zero = np.zeros((rows, H, v.shape[-1], q.shape[-1]))
    h0 = zero if h0 is None else _f64(h0)
    out = {"y": np.zeros((*q.shape[:-1], v.shape[-1])), "h_final": h0.copy()}
    if dy is not None:
        dy = _f64(dy)
        dhf = zero if dhf is None else _f64(dhf)
        out.update(dq=np.zeros_like(q), dk=np.zeros_like(kk), dv=np.zeros_like(vv), dh_init=dhf.copy())
    for span, r in at:
        out["y"][span], out["h_final"][r] = linear_row(q[span], kk[span], vv[span], lam, h0[r], scale)
        if dy is not None:
            out["dq"][span], out["dk"][span], out["dv"][span], out["dh_init"][r] = linear_row_bwd(
                q[span], kk[span], vv[span], lam, h0[r], scale, dy[span], dhf[r])
    if dy is not None:
        out["dk"], out["dv"] = gather(out["dk"], Hkv), gather(out["dv"], Hkv)
    return out


def _pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def turn(x, positions, freqs, interleaved, back=False):
    """The pairs of the first 2 * len(freqs) values of x [rows, H, D] turned by
    positions * freqs."""
    R = 2 * len(freqs)
    a, b = _pairs(R, interleaved)
    # extended precision: its 64-bit significand holds most products exactly
    ang = np.asarray(positions).astype(np.longdouble)[:, None] * np.asarray(freqs).astype(np.longdouble)
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    if back:
        s = -s
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def norm_rope(x, positions, freqs, weight, eps, interleaved):
    x = _f64(x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r if weight is None else x * r * _f64(weight)
    return turn(n, positions, freqs, interleaved)


def norm_rope_bwd(x, dy, positions, freqs, weight, eps, interleaved):
    """dx and dweight for x, dy [rows, H, D]."""
    x = _f64(x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = x * r
    u = turn(_f64(dy), positions, freqs, interleaved, back=True)
    g = u if weight is None else u * _f64(weight)
    return r * (g - z * (g * z).mean(-1, keepdims=True)), (u * z).sum((0, 1))
