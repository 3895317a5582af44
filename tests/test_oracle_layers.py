"""Pins of the fp64 gated recurrence and layer norm: closed forms, limits and
finite differences."""
import numpy as np
import pytest

from oracle import layers as O


def _case(seed, L=9, D=5, A=None):
    g = np.random.default_rng(seed)
    return dict(x=g.normal(size=(L, D)), r=g.normal(size=(L, D)), i=g.normal(size=(L, D)),
                A=-np.exp(g.normal(size=D)) if A is None else np.full(D, A), h0=g.normal(size=D),
                dy=g.normal(size=(L, D)), dhf=g.normal(size=D))


def test_constant_gates_give_a_geometric_series():
    # r = i = 0: s = g = 1/2, a = exp(A/2) every step; x = 1 from h = 0:
    # h_t = m/2 (1 - a^(t+1)) / (1 - a)
    L, D = 12, 3
    A = np.array([-0.1, -1.0, -4.0])
    z = np.zeros((L, D))
    h = O.gated_row(np.ones((L, D)), z, z, A, np.zeros(D))
    a = np.exp(A / 2)
    t = np.arange(1, L + 1)[:, None]
    np.testing.assert_allclose(h, np.sqrt(1 - a * a) / 2 * (1 - a ** t) / (1 - a), rtol=1e-12)


def test_closed_and_open_gates():
    c = _case(1)
    shut = np.full_like(c["r"], -800.0)  # a = 1, m = 0: the state is kept
    h = O.gated_row(c["x"], shut, c["i"], c["A"], c["h0"])
    np.testing.assert_array_equal(h, np.broadcast_to(c["h0"], h.shape))
    c["A"] = np.full(5, -800.0)  # an open gate forgets: h = g x
    wide = np.full_like(c["r"], 800.0)
    h = O.gated_row(c["x"], wide, c["i"], c["A"], c["h0"])
    np.testing.assert_allclose(h, O.sigmoid(c["i"]) * c["x"], rtol=1e-13)


def test_split_sequences_and_packing_agree():
    c = _case(2, L=20)
    whole = O.gated_row(c["x"], c["r"], c["i"], c["A"], c["h0"])
    first = O.gated_row(c["x"][:7], c["r"][:7], c["i"][:7], c["A"], c["h0"])
    rest = O.gated_row(c["x"][7:], c["r"][7:], c["i"][7:], c["A"], first[-1])
    np.testing.assert_allclose(np.concatenate([first, rest]), whole, rtol=1e-13)
    cu = np.array([0, 7, 7, 20])
    h0 = np.stack([c["h0"], c["dhf"], c["h0"] * 2])
    y, hf = O.gated(c["x"], c["r"], c["i"], c["A"], h0, cu)
    np.testing.assert_array_equal(y[:7], first)
    np.testing.assert_array_equal(hf[1], c["dhf"])
    np.testing.assert_array_equal(y[7:], O.gated_row(c["x"][7:], c["r"][7:], c["i"][7:], c["A"], h0[2]))


@pytest.mark.parametrize("name,arg", [("dx", "x"), ("dr", "r"), ("di", "i"), ("dA", "A"), ("dh_init", "h0")])
def test_gated_gradients_against_differences(name, arg):
    c = _case(3)

    def loss(v):
        k = dict(c, **{arg: v})
        h = O.gated_row(k["x"], k["r"], k["i"], k["A"], k["h0"])
        return (h * c["dy"]).sum() + (h[-1] * c["dhf"]).sum()

    got = O.gated_row_bwd(c["x"], c["r"], c["i"], c["A"], c["h0"], c["dy"], c["dhf"])[name]
    ref = _differences(loss, c[arg])
    # central differences of step 1e-5: error about 1e-10 of the third
    # derivative plus 1e-16/1e-5 of the loss
    np.testing.assert_allclose(got, ref, rtol=1e-6, atol=1e-8)


def _differences(loss, v, h=1e-5):
    out = np.empty_like(v)
    for at in np.ndindex(v.shape):
        up, down = v.copy(), v.copy()
        up[at] += h
        down[at] -= h
        out[at] = (loss(up) - loss(down)) / (2 * h)
    return out


def test_gated_gradient_where_the_input_scale_vanishes():
    c = _case(4, A=0.0)
    g = O.gated_row_bwd(c["x"], c["r"], c["i"], c["A"], c["h0"], c["dy"], c["dhf"])
    assert all(np.isfinite(v).all() for v in g.values())
    assert not g["dr"].any() and not g["dx"].any()


def test_layer_norm_closed_forms():
    g = np.random.default_rng(5)
    s = g.normal(size=(4, 12)) * 3 + 7
    y, mean, rstd = O.layer_norm(s, group=4, eps=0.0)
    v = y.reshape(4, 3, 4)
    np.testing.assert_allclose(v.mean(2), 0, atol=1e-12)
    np.testing.assert_allclose((v * v).mean(2), 1, rtol=1e-12)
    # unchanged by a shift and a scale of a group
    np.testing.assert_allclose(O.layer_norm(5 * s - 2, group=4, eps=0.0)[0], y, rtol=1e-9)
    assert mean.shape == rstd.shape == (4, 3)


@pytest.mark.parametrize("group", [None, 4])
@pytest.mark.parametrize("name", ["dx", "dweight", "dbias"])
def test_layer_norm_gradients_against_differences(group, name):
    g = np.random.default_rng(6)
    c = dict(s=g.normal(size=(3, 8)), weight=g.normal(size=8), bias=g.normal(size=8))
    dy, dsum = g.normal(size=(3, 8)), g.normal(size=(3, 8))
    _, mean, rstd = O.layer_norm(c["s"], c["weight"], c["bias"], group)
    arg = {"dx": "s", "dweight": "weight", "dbias": "bias"}[name]

    def loss(v):
        k = dict(c, **{arg: v})
        y = O.layer_norm(k["s"], k["weight"], k["bias"], group)[0]
        return (y * dy).sum() + (k["s"] * dsum).sum()

    got = O.layer_norm_bwd(c["s"], c["weight"], mean, rstd, dy, dsum, group)[name]
    np.testing.assert_allclose(got, _differences(loss, c[arg]), rtol=1e-6, atol=1e-8)
