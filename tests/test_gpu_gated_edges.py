"""The gated recurrence at its edges: gates that nearly close (1 - a^2 in the
range of fp32's subnormal numbers, whose root is an ordinary number) and values
that are not finite next to a border of packed sequences, very many empty
sequences in the same place."""
import numpy as np
import pytest
import torch

from oracle import layers as O
import _layers as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ss():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_18_amd import ssmscan
    ssmscan.lib()
    return ssmscan


def nearly_closed(gates):
    """(r [steps, channels], A [channels]): gates from -90 to -80 at decays of
    the usual size, or decays at the edge of fp32's range at ordinary gates."""
    if gates == "closed":
        A = [-0.0085, -0.1, -0.45, -1.0, -8.0, -0.008, -0.02]
        r = np.arange(-90.0, -79.9, 0.5)
    else:
        A = [-1e-38, -2e-38, -1e-37, -1e-36, -1e-34, -1e-30, -1.2e-38]
        r = np.arange(-3.0, 3.1, 0.25)
    r = np.random.default_rng(4).permuted(np.tile(r[:, None], (1, len(A))), axis=0)
    return r, np.array(A)


def bounds(x, r, i, A, dy):
    """{name: (reference, bound)} of one sequence [L, D] from a zero state with
    no gradient of the final one, for |u| < 1e-29 (so a = 1 and q = g x / m to
    far below a rounding), in the terms of _layers: the values' relative
    errors KM, KG there, and two of the subnormal range's own:

      u = A s and its forms in base-2 units round to multiples of 2^-149, each
          by at most half of one, three times at most, and 1 - a^2 once more:
          2^-148 / |u|, and A in base-2 units 2^-150 / |A|
      s below 2^-126 counts as 0: all of what the step adds

    rho is what that makes of m and of 1 / m (their own share is half of it).
    With e = 2^-24, every sum over steps rounds once a step, the decays (off
    by 3 e each, like every product with them) once more: 8 e a step."""
    s, g, u, _, m = O.gate_terms(r, i, A)
    e, L = T.E32, len(x)
    KR, KG = 1.5 * np.abs(r) + 5, 1.5 * np.abs(i) + 5
    KM = (KR + 3 + 5) / 2 + 2
    rho = np.minimum(2.0 ** -148 / np.abs(u) + 2.0 ** -150 / np.abs(A), 1.0)
    rho = np.where(s < 2.0 ** -126 * (1 + e * KR), 1.0, rho)
    eps = e * (KM + KG + 8) + rho
    b = m * g * x
    y = np.cumsum(b, 0)
    Ey = np.cumsum(np.abs(b) * (eps + 8 * e * L), 0)
    back = lambda v: np.cumsum(v[::-1], 0)[::-1]
    lam, mag = back(dy), back(np.abs(dy))
    El = 8 * e * L * mag
    before = np.concatenate([np.zeros_like(y[:1]), y[:-1]])
    Eh = np.concatenate([np.zeros_like(y[:1]), Ey[:-1]])
    w, v = El + np.abs(lam) * eps, m * g
    # 1 - g and 1 - s are off by 4 e beyond their factor's error
    di = lam * v * x * (1 - g)
    Edi = np.abs(v * x) * ((1 - g) * w + np.abs(lam) * e * (KG + 5))
    q = g * x / m
    aq, ah = np.abs(q), np.abs(before)
    du = lam * (before - q)
    Edu = El * (ah + aq) + np.abs(lam) * (Eh + aq * eps + e * (KR + 6) * (ah + aq))
    k = np.abs(A) * s
    return {"y": (y, Ey), "dx": (lam * v, v * w), "di": (di, Edi),
            "dr": (du * A * s * (1 - s), k * ((1 - s) * Edu + np.abs(du) * e * (KR + 8))),
            "dA": ((du * s).sum(0), (s * (Edu + e * (KR + 8 + L) * np.abs(lam) * (ah + aq))).sum(0)),
            "h_final": (y[-1], Ey[-1]), "dh_init": (lam[0], El[0] + 8 * e * mag[0])}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gates", ["closed", "open"])
@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
def test_gates_that_nearly_close(ss, gates, packed, dtype):
    print(f"case: gated nearly closed {gates} {packed} {dtype}", flush=True)
    r, A = nearly_closed(gates)
    L, D = r.shape
    g = torch.Generator().manual_seed(6)
    t = T.DT[dtype]
    x, i, dy = (torch.randn(L, D, generator=g).to(t).to(DEV) for _ in range(3))
    r, A = torch.tensor(r).to(t).to(DEV), torch.tensor(A, dtype=torch.float32, device=DEV)
    cu = [0, 9, 10, L] if packed else [0, L]
    c = torch.tensor(cu, device=DEV) if packed else None
    lead = (L, D) if packed else (1, L, D)
    f = ss.scan_gated_fwd(x.view(lead), r.view(lead), i.view(lead), A, cu_seqlens=c, want_carry=True)
    b = ss.scan_gated_bwd(x.view(lead), r.view(lead), i.view(lead), A, dy.view(lead), cu_seqlens=c, carry=f["carry"])
    got = {k: v.view(-1, D) if v.dim() > 1 else v for k, v in {**f, **b}.items()}
    n = [T.f64(v) for v in (x, r, i, A, dy)]
    dA, EdA = np.zeros(D), np.zeros(D)
    for k in range(len(cu) - 1):
        at = slice(cu[k], cu[k + 1])
        want = bounds(n[0][at], n[1][at], n[2][at], n[3], n[4][at])
        for name in ("y", "dx", "di", "dr"):
            ref, err = want[name]
            T.check(got[name][at], ref, T.stored(ref, err, dtype), f"sequence {k}: {name}")
        for name in ("h_final", "dh_init"):
            ref, err = want[name]
            T.check(got[name][k], ref, T.stored(ref, err, "fp32"), f"sequence {k}: {name}")
        dA, EdA = dA + want["dA"][0], EdA + want["dA"][1]
    # (terms of the subnormal range in s * du: 2^-149 |lam| (|h| + |q|) each)
    T.check(got["dA"], dA, EdA + T.E32 * np.abs(dA) + 1e-37, "dA")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gates", ["closed", "open"])
def test_step_whose_gates_nearly_close(ss, gates, dtype):
    print(f"case: gated step nearly closed {gates} {dtype}", flush=True)
    r, A = nearly_closed(gates)
    g = torch.Generator().manual_seed(7)
    t = T.DT[dtype]
    x, i = (torch.randn(r.shape, generator=g).to(t).to(DEV) for _ in range(2))
    r, A = torch.tensor(r).to(t).to(DEV), torch.tensor(A, dtype=torch.float32, device=DEV)
    h = torch.zeros(r.shape, device=DEV)
    y = ss.step_gated(x, r, i, A, h)
    n = [T.f64(v) for v in (x, r, i, A)]
    for row in range(len(r)):
        at = slice(row, row + 1)
        ref, err = bounds(n[0][at], n[1][at], n[2][at], n[3], np.zeros_like(n[0][at]))["y"]
        T.check(y[at], ref, T.stored(ref, err, dtype), f"row {row}: y")
        T.check(h[at], ref, T.stored(ref, err, "fp32"), f"row {row}: h")


def run(ss, o, cu):
    """Every output of a packed forward and backward."""
    c = torch.tensor(cu, dtype=torch.int64, device=DEV)
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], cu_seqlens=c, h_init=o["h_init"], want_carry=True)
    g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], cu_seqlens=c, h_init=o["h_init"],
                          dh_final=o["dh_final"], carry=f["carry"])
    torch.cuda.synchronize()
    return {**f, **g}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("name", ["r", "i", "x", "dy"])
def test_non_finite_values_next_to_a_border_stay_in_their_sequence(ss, name, bad, dtype):
    """A bad value up to 15 steps after a sequence's start or before its end,
    each in a channel of its own: every other sequence of that channel, and
    every other channel, keeps its bits.  (r = -Inf closes the gate: finite.)"""
    print(f"case: gated non-finite border {name} {bad} {dtype}", flush=True)
    L, cu = 700, [0, 100, 228, 257, 261, 262, 334, 403, 480, 700]
    nseq, D = len(cu) - 1, 130
    o = T.gated_inputs((L, D), 52, dtype, DEV, rows=nseq)
    clean = run(ss, o, cu)
    at, gen = {}, np.random.default_rng(8)
    for c in range(0, D, 2):
        k = int(gen.integers(nseq))
        d = int(gen.integers(min(16, cu[k + 1] - cu[k])))
        at[c] = (k, cu[k] + d if c % 4 else cu[k + 1] - 1 - d)
    p = dict(o, **{name: o[name].clone()})
    for c, (_, t) in at.items():
        p[name][t, c] = bad
    got = run(ss, p, cu)
    keep_t = torch.ones(L, D, dtype=torch.bool, device=DEV)
    keep_s = torch.ones(nseq, D, dtype=torch.bool, device=DEV)
    for c, (k, _) in at.items():
        keep_t[cu[k]:cu[k + 1], c] = False
        keep_s[k, c] = False
    for k in ("y", "dx", "dr", "di"):
        assert torch.equal(got[k][keep_t], clean[k][keep_t]), k
    for k in ("h_final", "dh_init"):
        assert torch.equal(got[k][keep_s], clean[k][keep_s]), k
    assert torch.equal(got["dA"][1::2], clean["dA"][1::2])


@pytest.mark.parametrize("where", ["behind", "between"])
def test_time_does_not_follow_the_empty_sequences(ss, where):
    """131072 empty sequences at one step.  Passing them one load after another
    takes 0.2 us each at the least, 26 ms; a search takes 17 loads, and the
    empty sequences' states are 4 MB in and out."""
    print(f"case: gated empty sequences' time {where}", flush=True)
    L, D, n = 700, 8, 1 << 17
    o = T.gated_inputs((L, D), 78, "bf16", DEV, rows=n + 2)
    cu = torch.full((n + 3,), 331 if where == "between" else L, dtype=torch.int64)
    cu[0], cu[1], cu[-1] = 0, 331, L
    few = torch.tensor([0, n + 1 if where == "between" else 1], device=DEV)
    c, times = cu.to(DEV), []
    for _ in range(4):
        torch.cuda.synchronize()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], cu_seqlens=c, h_init=o["h_init"], want_carry=True)
        g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], cu_seqlens=c, h_init=o["h_init"],
                              dh_final=o["dh_final"], carry=f["carry"])
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    got = {**f, **g}
    w = dict(o, h_init=o["h_init"][few].contiguous(), dh_final=o["dh_final"][few].contiguous())
    want = run(ss, w, [0, 331, L])
    for k, t in want.items():
        assert torch.equal(got[k][few] if k in ("h_final", "dh_init") else got[k], t), k
    assert min(times) < 10.0, times


@pytest.mark.parametrize("L, D", [(450, 3101), (300, 6011)])
def test_odd_rows_of_24_to_47_column_pairs(ss, L, D):
    """bf16 rows of an odd length that the backward takes one channel a lane, in
    chain groups of 8 links (25 and 47 columns of two channels)."""
    print(f"case: gated odd rows {L} {D}", flush=True)
    cu = [0, 1, 64, 130, L - 70, L - 70, L]
    o = T.gated_inputs((L, D), 79, "bf16", DEV, rows=len(cu) - 1)
    T.check_gated(run(ss, o, cu), o, "bf16", "packed", cu)
    d = {k: t[None] if t.shape[0] == L else t[:1] if t.dim() > 1 else t for k, t in o.items()}
    f = ss.scan_gated_fwd(d["x"], d["r"], d["i"], d["A"], h_init=d["h_init"], want_carry=True)
    g = ss.scan_gated_bwd(d["x"], d["r"], d["i"], d["A"], d["dy"], h_init=d["h_init"], dh_final=d["dh_final"],
                          carry=f["carry"])
    T.check_gated({**f, **g}, d, "bf16", "dense")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_input_gates_that_nearly_close(ss, dtype):
    """Input gates from -100 to -60, where g below 2^-114 counts as 0: each of
    82 steps then lacks at most 2^-114 times what the gate multiplies (below
    100 here, 1 / m included), so every sum at most 82 * 100 * 2^-114 < 1e-30."""
    print(f"case: gated input gates {dtype}", flush=True)
    o = T.gated_inputs((1, 82, 130), 80, dtype, DEV, A=-2.0)
    o["i"].copy_(torch.arange(-100.0, -59.0, 0.5)[None, :, None].expand(1, 82, 130))
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=o["h_init"], want_carry=True)
    g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], h_init=o["h_init"], dh_final=o["dh_final"],
                          carry=f["carry"])
    T.check_gated({**f, **g}, o, dtype, "input gates", floor=1e-30)
    o["h_init"].zero_()  # nothing but the gated inputs
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=o["h_init"])
    T.check_gated(f, o, dtype, "input gates alone", floor=1e-30)
    assert f["y"][0, 80:].abs().max() > 1e-28  # and those above are there
