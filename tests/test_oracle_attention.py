"""Pins of the fp64 definitions of linear attention and of the norm and rotation
of queries and keys (CPU): the quadratic form, closed forms, differences."""
import numpy as np
import pytest

from oracle import attention as A


def inputs(L=7, H=4, Hkv=2, Dk=5, Dv=3, rows=1, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((L, H, Dk)), k=r.standard_normal((L, Hkv, Dk)), v=r.standard_normal((L, Hkv, Dv)),
                log_decay=-r.uniform(0.01, 1.0, H), h0=r.standard_normal((rows, H, Dv, Dk)),
                dy=r.standard_normal((L, H, Dv)), dhf=r.standard_normal((rows, H, Dv, Dk)))


def attn(o, cu=None, **k):
    if cu is None:  # one sequence, as a dense batch of one row
        d = {n: t[None] for n, t in o.items() if n in ("q", "k", "v", "dy")}
        out = A.linear_attn(d["q"], d["k"], d["v"], o["log_decay"], 0.5, o["h0"], None, d["dy"], o["dhf"], **k)
        return {n: t if n in ("h_final", "dh_init") else t[0] for n, t in out.items()}
    return A.linear_attn(o["q"], o["k"], o["v"], o["log_decay"], 0.5, o["h0"], cu, o["dy"], o["dhf"], **k)


def test_quadratic_form():
    o = inputs()
    L, H = o["q"].shape[:2]
    kk, vv, lam = np.repeat(o["k"], 2, 1), np.repeat(o["v"], 2, 1), np.exp(o["log_decay"])
    got = attn(o)
    for h in range(H):
        for t in range(L):
            y = lam[h] ** (t + 1) * o["h0"][0, h] @ o["q"][t, h]
            for s in range(t + 1):
                y = y + lam[h] ** (t - s) * (o["q"][t, h] @ kk[s, h]) * vv[s, h]
            np.testing.assert_allclose(got["y"][t, h], 0.5 * y, rtol=1e-12, atol=1e-12)


def test_geometric_sum():
    """Equal steps: the state is the sum of a geometric series."""
    L, lam = 50, 0.9
    q, k, v = (np.full((L, 1, 1), c) for c in (2.0, 3.0, 5.0))
    out = A.linear_attn(q[None], k[None], v[None], np.log([lam]), 1.0)
    n = np.arange(1, L + 1)
    np.testing.assert_allclose(out["y"][0, :, 0, 0], 2.0 * 15.0 * (1 - lam ** n) / (1 - lam), rtol=1e-12)


def test_no_memory():
    o = inputs()
    o["log_decay"][:] = -np.inf
    got = attn(o)
    kk, vv = np.repeat(o["k"], 2, 1), np.repeat(o["v"], 2, 1)
    np.testing.assert_allclose(got["y"], 0.5 * (o["q"] * kk).sum(-1, keepdims=True) * vv, rtol=1e-13)


def test_packed_is_each_sequence_alone():
    cu = [0, 3, 3, 7]
    o = inputs(rows=3)
    got = attn(o, cu)
    for s in range(3):
        one = {n: t[cu[s]:cu[s + 1]] if n in ("q", "k", "v", "dy") else t[s:s + 1] if n in ("h0", "dhf") else t
               for n, t in o.items()}
        want = attn(one)
        for n in want:
            a = got[n][s:s + 1] if n in ("h_final", "dh_init") else got[n][cu[s]:cu[s + 1]]
            np.testing.assert_array_equal(a, want[n])


@pytest.mark.parametrize("name,grad", [("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh_init")])
def test_gradients_against_differences(name, grad):
    o = inputs(L=5, seed=3)
    got = attn(o)[grad]
    loss = lambda: (attn(o)["y"] * o["dy"]).sum() + (attn(o)["h_final"] * o["dhf"]).sum()
    r = np.random.default_rng(4)
    for _ in range(8):
        at = tuple(r.integers(n) for n in o[name].shape)
        x, step = o[name][at], 1e-5
        o[name][at] = x + step
        up = loss()
        o[name][at] = x - step
        down = loss()
        o[name][at] = x
        # the loss is linear in h0 and bilinear in the others: differences are exact but for rounding
        assert abs(got[at] - (up - down) / (2 * step)) < 1e-7 * max(1.0, abs(got[at]))


def test_rotation_depends_on_the_distance_alone():
    """Scores of turned queries and keys go by the difference of positions."""
    r = np.random.default_rng(5)
    q, k = r.standard_normal((1, 1, 8)), r.standard_normal((1, 1, 8))
    freqs = 1.0 / 100.0 ** (np.arange(3) / 3)
    for inter in (False, True):
        score = lambda m, n: (A.turn(q, [m], freqs, inter) * A.turn(k, [n], freqs, inter)).sum()
        assert abs(score(5, 2) - score(1005, 1002)) < 1e-10
        assert abs(score(5, 2) - score(5, 3)) > 1e-3
        y = A.turn(q, [17], freqs, inter)
        np.testing.assert_allclose(A.turn(y, [17], freqs, inter, back=True), q, atol=1e-14)
        np.testing.assert_array_equal(y[..., 6:], q[..., 6:])
        np.testing.assert_allclose((y * y).sum(), (q * q).sum(), rtol=1e-14)


def test_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    quarter = np.array([np.pi / 2, np.pi / 2])
    np.testing.assert_allclose(A.turn(x, [1], quarter, False), [[[-3.0, -4.0, 1.0, 2.0]]], atol=1e-15)
    np.testing.assert_allclose(A.turn(x, [1], quarter, True), [[[-2.0, 1.0, -4.0, 3.0]]], atol=1e-15)


def test_norm_of_constant_values():
    y = A.norm_rope(np.full((2, 3, 8), -4.0), [0, 9], np.zeros(0), np.arange(8.0), 0.0, False)
    np.testing.assert_allclose(y, np.broadcast_to(-np.arange(8.0), y.shape))


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_gradients_against_differences(inter):
    r = np.random.default_rng(6)
    x, dy, w = r.standard_normal((3, 2, 8)), r.standard_normal((3, 2, 8)), r.standard_normal(8)
    pos, freqs = np.array([0, 7, 100]), np.array([0.3, 0.01])
    dx, dw = A.norm_rope_bwd(x, dy, pos, freqs, w, 1e-6, inter)
    loss = lambda: (A.norm_rope(x, pos, freqs, w, 1e-6, inter) * dy).sum()
    for t, g in ((x, dx), (w, dw)):
        for _ in range(6):
            at = tuple(r.integers(n) for n in t.shape)
            v, step = t[at], 1e-5
            t[at] = v + step
            up = loss()
            t[at] = v - step
            down = loss()
            t[at] = v
            # third derivatives of order 1 times step^2, and rounding / step
            assert abs(g[at] - (up - down) / (2 * step)) < 1e-7 * max(1.0, abs(g[at]))
