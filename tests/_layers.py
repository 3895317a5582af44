"""Inputs, fp64 references and derived error bounds of the gated recurrence
and the layer norm.

Bounds are first-order running error analyses in units of e = 2^-24 (half a
unit in the last place of fp32, relative), with M the same recurrence run on
absolute values:

  sigmoid of a value v: the exponent's rounding gives (1.5 |v|) e, exp 2 e, the
      sum 1 e and the reciprocal 2 e: KS = 1.5 |v| + 5
  a = exp(u), u = A s: the argument is off by |u| (KS + 3) e, exp by 2 e:
      KA = |u| (KS + 3) + 3
  m = sqrt(1 - a^2): half the relative error of 1 - a^2 (near u = 0 the
      product -2 u a p, relative KS + 1 + KA + 4; elsewhere 1.2 KA + 1), then
      sqrt 2 e: KM = (KS + KA + 5) / 2 + 2
  b = m g x: KB = KM + KS + 2
  h_t = a h + b: E_t = a E_{t-1} + e (KA a M_{t-1} + KB |b| + 5 M_t); the 5
      covers the rounding of the sum itself, of the decay products of a
      time-split evaluation and of the carry's fold

and a value stored in T is off by its relative half step more (2^-8 of the
value for bf16, nothing more for fp32, whose rounding the 5 holds).
"""
import numpy as np
import torch

from oracle import layers as O

E32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return None if t is None else t.detach().to("cpu").to(torch.float64).numpy()


def check(got, ref, bound, what):
    got, ref, bound = f64(got), np.asarray(ref), np.asarray(bound)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.size == 0:
        return
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    over = np.abs(got - ref) - bound
    at = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[at] <= 0, f"{what}{at}: got {got[at]:.9g}, expected {ref[at]:.9g} within {bound[at]:.3g}"


def stored(ref, bound, dtype):
    """Bound of a value with error `bound` before its rounding to storage;
    1e-37 covers results in the range of subnormal numbers."""
    return bound + HALF[dtype] * (np.abs(ref) + bound) + 1e-37


def gated_inputs(shape, seed, dtype, dev, rows=None, A=None, offset=0, state=True, grads=True):
    """x, r, i, dy of `shape`, A, and per-row states; offset > 0 puts every
    tensor that many elements past an aligned address."""
    g = torch.Generator().manual_seed(seed)
    D = shape[-1]

    def make(sh, dt, scale=1.0):
        v = (torch.randn(sh, generator=g) * scale).to(dt)
        n = v.numel()
        buf = torch.empty(n + offset, dtype=dt, device=dev)
        buf[offset:] = v.reshape(-1).to(dev)
        return buf[offset:].view(sh)

    t = DT[dtype]
    o = {"x": make(shape, t), "r": make(shape, t, 1.5), "i": make(shape, t, 1.5)}
    if A is None:
        a = -8.0 * torch.rand(D, generator=g) ** 3  # decays from nearly 1 to e^-8
        o["A"] = make((D,), torch.float32)
        o["A"].copy_(a)
    else:
        o["A"] = make((D,), torch.float32)
        o["A"].fill_(A)
    rows = shape[0] if rows is None else rows
    o["h_init"] = make((rows, D), torch.float32) if state else None
    if grads:
        o["dy"] = make(shape, t)
        o["dh_final"] = make((rows, D), torch.float32) if state else None
    return o


def _row(x, r, i, A, h0, dy=None, dhf=None):
    """Reference values and error bounds of one sequence, unrounded."""
    s, g, u, a, m = O.gate_terms(r, i, A)
    vs = np.abs(np.asarray(r)), np.abs(np.asarray(i))
    KR, KG = 1.5 * vs[0] + 5, 1.5 * vs[1] + 5
    KA = np.abs(u) * (KR + 3) + 3
    KM = (KR + KA + 5) / 2 + 2
    KB = KM + KG + 2
    b = m * g * x
    h = O.gated_row(x, r, i, A, h0)
    E, M, Eb, Mb = (np.empty_like(h) for _ in range(4))
    e, c = np.zeros_like(h0), np.abs(h0)
    for t in range(len(h)):
        Eb[t], Mb[t] = e, c
        mag = a[t] * c + np.abs(b[t])
        e = a[t] * e + E32 * (KA[t] * a[t] * c + KB[t] * np.abs(b[t]) + 5 * mag)
        c = mag
        E[t], M[t] = e, c
    out = {"h": h, "Eh": E}
    if dy is None:
        return out
    grads = O.gated_row_bwd(x, r, i, A, h0, dy, dhf)
    before = np.concatenate([h0[None], h[:-1]])
    El, Ml, lam = (np.empty_like(h) for _ in range(3))
    e, c, f = np.zeros_like(h0), np.abs(dhf), np.array(dhf)
    for t in range(len(h) - 1, -1, -1):
        lam[t] = dy[t] + f
        Ml[t] = np.abs(dy[t]) + c
        El[t] = e + 5 * E32 * Ml[t]
        e = a[t] * El[t] + E32 * (KA[t] + 2) * a[t] * Ml[t]
        c = a[t] * Ml[t]
        f = a[t] * lam[t]
    out.update(grads)
    al = np.abs(lam)
    mg = m * g
    out["Edx"] = mg * (El + E32 * (KM + KG + 4) * al)
    # 1 - g: g = 1 / (1 + w), w = exp(-v), is off by g (1 - g) (1.5 |v| + 2) e
    # through w (dg = -g (1 - g) dw / w) and by 3 g e through the rounding of
    # the sum and of the reciprocal, which no factor 1 - g damps; then the
    # difference rounds once
    off = lambda w, v: E32 * (w * ((1 - w) * (1.5 * v + 2) + 3) + 1)
    out["Edi"] = np.abs(x) * mg * ((1 - g) * (El + E32 * (KM + KG + 7) * al) + al * off(g, vs[1]))
    q = np.divide(g * np.abs(x) * a * a, m, out=np.zeros_like(m), where=m > 0)
    mag = a * Mb + q
    Edu = El * mag + al * (a * Eb + E32 * ((KA + 3) * a * Mb + (KG + 2 * KA + KM + 7) * q + 2 * mag))
    k = np.abs(A) * s
    out["Edr"] = k * ((1 - s) * (Edu + E32 * (KR + 5) * al * mag) + al * mag * off(s, vs[0]))
    out["EdA"] = (s * (Edu + E32 * (KR + 3) * al * mag)).sum(0)
    out["MdA"] = (s * al * mag).sum(0)
    out["Edh_init"] = e
    return out


def gated_reference(o, cu=None, want_grads=True, terms=None):
    """{name: (reference, bound before storage rounding)}."""
    n = {k: f64(v) for k, v in o.items()}
    parts, rows = O._parts(n["x"], cu)
    D = n["A"].shape[0]
    z = np.zeros((rows, D))
    h0 = z if n["h_init"] is None else n["h_init"]
    grads = want_grads and "dy" in n
    names = ("y", "dx", "dr", "di") if grads else ("y",)
    ref = {k: np.empty(n["x"].shape) for k in names}
    err = {k: np.empty(n["x"].shape) for k in names}
    ref["h_final"], err["h_final"] = h0.copy(), np.zeros_like(z)
    if grads:
        dhf = z if n["dh_final"] is None else n["dh_final"]
        ref["dh_init"], err["dh_init"] = dhf.copy(), np.zeros_like(z)
        ref["dA"], err["dA"], mag = np.zeros(D), np.zeros(D), np.zeros(D)
    steps = 0
    for k, at in enumerate(parts):
        x = n["x"][at]
        if len(x) == 0:
            continue
        steps += len(x)
        w = _row(x, n["r"][at], n["i"][at], n["A"], h0[k], n["dy"][at] if grads else None, dhf[k] if grads else None)
        ref["y"][at], err["y"][at] = w["h"], w["Eh"]
        ref["h_final"][k], err["h_final"][k] = w["h"][-1], w["Eh"][-1]
        if grads:
            for name in ("dx", "dr", "di"):
                ref[name][at], err[name][at] = w[name], w["E" + name]
            ref["dh_init"][k], err["dh_init"][k] = w["dh_init"], w["Edh_init"]
            ref["dA"] += w["dA"]
            err["dA"] += w["EdA"]
            mag += w["MdA"]
    if grads:
        # the sum of dA: every addition of a chain of at most
        # min(steps, 64 + steps / 64) terms rounds once
        err["dA"] += min(steps, 64 + steps / 64) * E32 * mag + 1e-37
    return ref, err


def check_gated(got, o, dtype, what, cu=None, floor=1e-37):
    ref, err = gated_reference(o, cu, want_grads="dx" in got)
    for k, t in got.items():
        if k == "carry":
            continue
        if k in ("y", "dx", "dr", "di"):
            check(t, ref[k], stored(ref[k], err[k], dtype) + floor, f"{what}: {k}")
        else:
            check(t, ref[k], err[k] + E32 * np.abs(ref[k]) + floor, f"{what}: {k}")


def norm_bounds(s, mean, rstd, weight, bias, group, eps):
    """Bounds of (y before storage, mean, rstd): sums over a group of P round
    at most d = P / 64 + 12 times a chain (64 lanes, then a tree)."""
    rows, Dm = s.shape
    P = group or Dm
    d = P / 64 + 12
    v = s.reshape(rows, Dm // P, P)
    Em = E32 * (d * np.abs(v).mean(2) + 2 * np.abs(mean))
    c = v - mean[..., None]
    Ec = Em[..., None] + E32 * np.abs(c)
    var = (c * c).mean(2)
    Ev = (2 * np.abs(c) * Ec + Ec * Ec).mean(2) + E32 * (d + 3) * var
    Er = rstd * (Ev / (2 * (var + eps)) + 4 * E32) if eps > 0 or (var > 0).all() else rstd * np.inf
    w = np.abs(weight).reshape(1, Dm // P, P) if weight is not None else 1.0
    z = np.abs(c) * rstd[..., None]
    Ey = w * (Ec * rstd[..., None] + np.abs(c) * Er[..., None] + 3 * E32 * z)
    Ey = Ey.reshape(rows, Dm)
    if bias is not None:
        Ey = Ey + 2 * E32 * np.abs(bias)
    return Ey, Em, Er


def norm_bwd_bounds(s, mean, rstd, weight, dy, dsum, group):
    """Bounds of dx (before storage), dweight, dbias for exact statistics."""
    rows, Dm = s.shape
    P = group or Dm
    d = P / 64 + 12
    v = s.reshape(rows, Dm // P, P)
    r = rstd[..., None]
    z = np.abs(v - mean[..., None]) * r
    Ez = 3 * E32 * z
    q = np.abs(dy if weight is None else dy * weight).reshape(v.shape)
    m1, m2 = q.mean(2, keepdims=True), (q * z).mean(2, keepdims=True)
    E1 = E32 * (d + 2) * m1
    E2 = E32 * (d + 6) * m2
    Ex = r * (E32 * q + E1 + z * E2 + Ez * m2 + 5 * E32 * (q + m1 + z * m2))
    Ex = Ex.reshape(rows, Dm)
    if dsum is not None:
        Ex = Ex + 2 * E32 * np.abs(dsum)
    # sums over rows: at most min(rows, 64 + rows / 64) additions in a chain
    k = min(rows, 64 + rows / 64) + 6
    zz = z.reshape(rows, Dm)
    return Ex, E32 * k * (np.abs(dy) * zz).sum(0) + 1e-37, E32 * k * np.abs(dy).sum(0) + 1e-37
