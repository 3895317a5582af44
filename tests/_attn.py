"""Inputs and derived error bounds of linear attention and of the norm and
rotation of queries and keys.

Bounds are first-order running error analyses in units of e = 2^-24 (half a
unit in the last place of fp32), with M the recurrence run on absolute values.

Linear attention, state H_t = l H_{t-1} + v k^T with l = exp(a):
  a power l^n is exp2 of a product of rounded factors: relative error
      (3 |n a| + 3) e.  Terms fade as they age, so with D_t = l (D_{t-1} +
      |a| M_{t-1}), the sum of |n a| l^n |v k| over ages n, the powers cost
      3 e D + 3 e M (and 3 e M again for the chunks' own decays)
  the states add one product per step and round once each (the adds of a
      chunk and its decay, at most 2 a step): E_t = l E_{t-1} + 2 e M_t
  the weighted v is a sum of bf16 terms whose rest is below 2^-24: 1 e M
  y = scale H q: the state's error, the sum over Dk products and over the chunk
      (Dk + 64 roundings), the weights, and for bf16 the two terms of the state
      or of the weighted scores, whose rest is below 2^-18 of the operand
  a value stored in T is off by its relative half step more.
The gradients are the same operation with other arguments.
"""
import numpy as np
import torch

from oracle import attention as A
from _layers import DT, E32, HALF, check, f64, stored  # noqa: F401


def _op(q, k, v, a, h0, undecayed, y_scale, k_scale, dtype):
    """One sequence's (y, bound, state, bound) for per-head tensors; undecayed:
    the entering state counts fully at the first step, the leaving one is
    decayed once more."""
    lam = np.exp(a)[:, None, None]
    aa = np.minimum(np.abs(a), 1e6)[:, None, None]
    h, M, D, E = h0.copy(), np.abs(h0), np.zeros_like(h0), np.zeros_like(h0)
    split = 2.0 ** -18 if dtype == "bf16" else 0.0
    L, Dk = len(q), q.shape[-1]
    y, Ey = (np.empty((L, *v.shape[1:])) for _ in range(2))

    def fade():
        nonlocal h, M, D, E
        h, D, M, E = lam * h, lam * (D + aa * M), lam * M, lam * E

    for t in range(L):
        if not (undecayed and t == 0):
            fade()
        kv = k_scale * v[t][:, :, None] * k[t][:, None, :]
        h = h + kv
        M = M + np.abs(kv)
        E = E + 2 * E32 * M
        y[t] = y_scale * np.einsum("hvk,hk->hv", h, q[t])
        aq = np.abs(q[t])
        my = np.einsum("hvk,hk->hv", M, aq)
        Ey[t] = abs(y_scale) * (np.einsum("hvk,hk->hv", E + 3 * E32 * D, aq) +
                                ((Dk + 64 + 12) * E32 + split) * my)
    if undecayed:
        fade()
    return y, Ey, h, E + 3 * E32 * D + 8 * E32 * M


def linear_reference(o, scale, cu=None, dtype="bf16"):
    """{name: (reference, bound before storage)}."""
    n = {k: f64(t) for k, t in o.items()}
    H, Hkv = n["q"].shape[-2], n["k"].shape[-2]
    q, k, v, a = n["q"], A.spread(n["k"], H), A.spread(n["v"], H), n["log_decay"]
    a = np.maximum(a, -1e30)
    rows = q.shape[0] if cu is None else len(cu) - 1
    zero = np.zeros((rows, H, v.shape[-1], q.shape[-1]))
    h0 = zero if n.get("h_init") is None else n["h_init"]
    names = {"y": (H, v.shape[-1])}
    grads = n.get("dy") is not None
    if grads:
        dhf = zero if n.get("dh_final") is None else n["dh_final"]
        names.update(dq=(H, q.shape[-1]), dk=(H, q.shape[-1]), dv=(H, v.shape[-1]))
    ref = {m: np.zeros((*q.shape[:-2], *s)) for m, s in names.items()}
    err = {m: np.zeros_like(r) for m, r in ref.items()}
    ref["h_final"], err["h_final"] = h0.copy(), np.zeros_like(h0)
    if grads:
        ref["dh_init"], err["dh_init"] = dhf.copy(), np.zeros_like(dhf)
    T = lambda t: np.swapaxes(t, -1, -2)
    for at, r in A.parts(q.shape[-3], cu, rows):
        qs, ks, vs = q[at], k[at], v[at]
        if len(qs) == 0:
            continue
        ref["y"][at], err["y"][at], ref["h_final"][r], err["h_final"][r] = _op(
            qs, ks, vs, a, h0[r], False, scale, 1.0, dtype)
        if not grads:
            continue
        dy = n["dy"][at]
        ref["dq"][at], err["dq"][at], _, _ = _op(dy, vs, ks, a, T(h0[r]), False, scale, 1.0, dtype)
        back = lambda t: t[::-1]
        dk, Ek, _, _ = _op(back(vs), back(dy), back(qs), a, T(dhf[r]), True, 1.0, scale, dtype)
        dv, Ev, ref["dh_init"][r], err["dh_init"][r] = _op(back(ks), back(qs), back(dy), a, dhf[r], True, 1.0, scale,
                                                           dtype)
        for m, x, e in (("dk", dk, Ek), ("dv", dv, Ev)):
            ref[m][at], err[m][at] = back(x), back(e)
    if grads and H != Hkv:
        for m in ("dk", "dv"):
            mag = A.gather(np.abs(ref[m]) + err[m], Hkv)
            ref[m], err[m] = A.gather(ref[m], Hkv), A.gather(err[m], Hkv) + (H // Hkv) * E32 * mag
    return ref, err


def check_linear(got, o, scale, dtype, what, cu=None):
    ref, err = linear_reference({**o, "dy": o.get("dy") if "dq" in got else None}, scale, cu, dtype)
    for m, t in got.items():
        if m in ("h_final", "dh_init"):
            check(t, ref[m], err[m] + E32 * np.abs(ref[m]) + 1e-37, f"{what}: {m}")
        else:
            check(t, ref[m], stored(ref[m], err[m], dtype), f"{what}: {m}")
    return ref


def make(shape, seed, dtype, dev, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype] if isinstance(dtype, str) else dtype).to(dev)


def slopes(H, dev, strong=-1.0, weak=-10.0):
    """Log decays spread geometrically from -2^strong to -2^weak."""
    e = torch.linspace(strong, weak, H, dtype=torch.float64) if H > 1 else torch.tensor([-4.0])
    return (-(2.0 ** e)).to(torch.float32).to(dev)


def linear_inputs(lead, H, Hkv, Dk, Dv, seed, dtype, dev, rows=None, state=True, grads=True, decay=None):
    rows = lead[0] if rows is None else rows
    f32 = torch.float32
    o = {"q": make((*lead, H, Dk), seed, dtype, dev), "k": make((*lead, Hkv, Dk), seed + 1, dtype, dev),
         "v": make((*lead, Hkv, Dv), seed + 2, dtype, dev),
         "log_decay": slopes(H, dev) if decay is None else torch.full((H,), decay, device=dev)}
    o["h_init"] = make((rows, H, Dv, Dk), seed + 3, f32, dev, 3.0) if state else None
    if grads:
        o["dy"] = make((*lead, H, Dv), seed + 4, dtype, dev)
        o["dh_final"] = make((rows, H, Dv, Dk), seed + 5, f32, dev) if state else None
    return o


def rope_inputs(rows, Hq, Hk, D, R, seed, dtype, dev, offset=0, far=1 << 20):
    """q, k, gradients, weights, positions (some negative, some far) and
    frequencies; offset: elements past an aligned address."""
    g = torch.Generator().manual_seed(seed)

    def put(shape, dt):
        v = torch.randn(shape, generator=g)
        buf = torch.empty(v.numel() + offset, dtype=dt, device=dev)
        buf[offset:] = v.to(dt).reshape(-1).to(dev)
        return buf[offset:].view(shape)

    t = DT[dtype]
    o = {"q": put((rows, Hq, D), t), "k": put((rows, Hk, D), t), "dq": put((rows, Hq, D), t),
         "dk": put((rows, Hk, D), t), "q_weight": put((D,), torch.float32), "k_weight": put((D,), torch.float32)}
    pos = torch.randint(-far, far, (rows,), generator=g)
    pos[: min(3, rows)] = torch.tensor([0, 1, far])[: min(3, rows)]
    o["positions"] = pos.to(dev)
    o["freqs"] = (10000.0 ** (-torch.arange(R // 2, dtype=torch.float32) / max(1, R // 2))).to(dev)
    return o


def _rope_terms(x, eps):
    """|z|, rstd and the relative error of rstd: a chain of D / 8 + 12 sums of
    squares (each 2 e), halved by the root, then root and quotient 3 e."""
    D = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return np.abs(x) * r, r, E32 * ((D / 8 + 12 + 2) / 2 + 3)


def _pair_magnitude(n, R, interleaved):
    """|n_a| + |n_b| of a value's pair; the value itself where nothing turns.
    (sine and cosine within 4 e: 2 e of sincospi, 1 e of the fraction's
    rounding times 2 pi on an angle of at most pi; products and sum 2 e)"""
    a, b = A._pairs(R, interleaved)
    m = np.abs(n).copy()
    m[..., a] = m[..., b] = np.abs(n)[..., a] + np.abs(n)[..., b]
    return m


def check_rope(got, o, dtype, what, eps=1e-6, interleaved=False, affine=True):
    n = {k: f64(t) if t.is_floating_point() else t.cpu().numpy() for k, t in o.items()}
    R = 2 * len(n["freqs"])
    turned = 16 * E32
    for m in ("q", "k"):
        w = n[m + "_weight"] if affine else None
        x, aw = n[m], 1.0 if w is None else np.abs(w)
        ref = A.norm_rope(x, n["positions"], n["freqs"], w, eps, interleaved)
        z, r, er = _rope_terms(x, eps)
        mag = _pair_magnitude(z * aw, R, interleaved)
        check(got[m], ref, stored(ref, (er + 3 * E32 + turned) * mag, dtype), f"{what}: {m}")
        if "d" + m not in got:
            continue
        dy, D = n["d" + m], x.shape[-1]
        dx, dw = A.norm_rope_bwd(x, dy, n["positions"], n["freqs"], w, eps, interleaved)
        u = _pair_magnitude(dy, R, interleaved)  # off by `turned` of this
        g = u * aw
        mean = (g * z).mean(-1, keepdims=True)
        eu = turned + (D / 8 + 12) * E32
        bound = r * ((turned + 6 * E32) * g + z * mean * (eu + 2 * er + 8 * E32) + er * (g + z * mean))
        check(got["d" + m], dx, stored(dx, bound, dtype), f"{what}: d{m}")
        if "d" + m + "_weight" in got:
            # a lane's chain (256 heads and one block's teams), then blocks
            heads = x.shape[0] * x.shape[1]
            k = min(heads, 256 + 64 + heads / 256) + 8
            check(got["d" + m + "_weight"], dw, (k * E32 + turned + er) * (u * z).sum((0, 1)) + 1e-37,
                  f"{what}: d{m}_weight")
