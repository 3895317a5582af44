"""Refusals of the gated recurrence and the layer norm at the C ABI, on the
CPU: bad arguments end in a status before any device call."""
import ctypes

import pytest

P = [0x1000000 * (k + 1) for k in range(16)]  # never dereferenced
F32, BF16 = 0, 1
v = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from selective_state_space_18_amd import ssmscan
    return ssmscan.lib()


def fwd(L, x=P[0], r=P[1], i=P[2], A=P[3], cu=None, nseq=0, hi=None, y=P[4], hf=P[5], carry=P[6], B=2, T=100, D=8,
        dtype=BF16):
    return L.ssm_scan_gated_fwd(v(x), v(r), v(i), v(A), v(cu), nseq, v(hi), v(y), v(hf), v(carry), B, T, D, dtype, None)


def bwd(L, x=P[0], r=P[1], i=P[2], A=P[3], cu=None, nseq=0, hi=None, carry=P[6], dy=P[7], dhf=None, dx=P[8], dr=P[9],
        di=P[10], dA=P[11], dhi=P[12], B=2, T=100, D=8, dtype=BF16):
    return L.ssm_scan_gated_bwd(v(x), v(r), v(i), v(A), v(cu), nseq, v(hi), v(carry), v(dy), v(dhf), v(dx), v(dr),
                                v(di), v(dA), v(dhi), B, T, D, dtype, None)


def step(L, x=P[0], r=P[1], i=P[2], A=P[3], h=P[4], ho=P[5], y=P[6], B=2, D=8, dtype=BF16):
    return L.ssm_step_gated(v(x), v(r), v(i), v(A), v(h), v(ho), v(y), B, D, dtype, None)


def norm(L, x=P[0], res=P[1], w=P[2], b=P[3], s=P[4], y=P[5], mean=P[6], rstd=P[7], rows=4, D=8, group=8, eps=1e-5,
         dtype=BF16):
    return L.ssm_layer_norm_fwd(v(x), v(res), v(w), v(b), v(s), v(y), v(mean), v(rstd), rows, D, group, eps, dtype, None)


def normb(L, s=P[0], w=P[1], mean=P[2], rstd=P[3], dy=P[4], dsum=P[5], dx=P[6], dw=P[7], db=P[8], rows=4, D=8,
          group=8, dtype=BF16):
    return L.ssm_layer_norm_bwd(v(s), v(w), v(mean), v(rstd), v(dy), v(dsum), v(dx), v(dw), v(db), rows, D, group,
                                dtype, None)


@pytest.mark.parametrize("f", [fwd, bwd, step, norm, normb])
def test_common_refusals(L, f):
    assert f(L, dtype=2) == 3 and f(L, dtype=-1) == 3
    assert f(L, D=-1) == 2
    first = {"s": P[0]} if f is normb else {"x": P[0]}
    key = next(iter(first))
    assert f(L, **{key: 0}) == 1 and b"NULL" in L.ssm_last_error()
    assert f(L, **{key: P[0] + 1}) == 5
    assert f(L, dtype=F32, **{key: P[0] + 2}) == 5


def test_gated_forward_refusals(L):
    assert fwd(L, B=-1) == 2 and fwd(L, T=-1) == 2
    assert fwd(L, B=1 << 31, T=0) == 2 and fwd(L, T=1 << 62, D=1 << 10) == 2
    assert fwd(L, B=1, D=(1 << 22) + 1) == 2 and b"1 GiB" in L.ssm_last_error()
    assert fwd(L, B=1, T=(1 << 28) + 1, D=1) == 2 and b"2^28" in L.ssm_last_error()
    far = [k << 44 for k in range(1, 15)]  # room for outputs of such sizes
    big = dict(x=far[0], r=far[1], i=far[2], A=far[3], y=far[4], hf=far[5], carry=far[6])
    assert fwd(L, B=8192, T=1 << 18, D=1, **big) == 2 and b"2^22" in L.ssm_last_error()
    more = dict(dy=far[7], dx=far[8], dr=far[9], di=far[10], dA=far[11], dhi=far[12])
    del big["y"], big["hf"]
    assert bwd(L, B=8192, T=1 << 16, D=1, **big, **more) == 2 and b"2^22" in L.ssm_last_error()
    assert bwd(L, B=1, T=(1 << 28) + 1, D=1) == 2
    for k in ("r", "i", "A", "y"):
        assert fwd(L, **{k: 0}) == 1
    assert fwd(L, A=P[3] + 2) == 5 and fwd(L, carry=P[6] + 2) == 5
    assert fwd(L, y=P[0]) == 6 and fwd(L, y=P[1] + 2) == 6 and fwd(L, hf=P[4]) == 6 and fwd(L, carry=P[5]) == 6
    assert fwd(L, hi=P[5] + 4) == 6 and fwd(L, hi=P[4]) == 6 and fwd(L, hi=P[6]) == 6
    assert fwd(L, carry=P[2]) == 6
    # packed sequences
    assert fwd(L, cu=P[13], nseq=3, B=2) == 2
    assert fwd(L, cu=P[13], nseq=-1, B=1) == 2 and fwd(L, cu=P[13], nseq=0, B=1) == 2
    assert fwd(L, cu=P[13] + 4, nseq=3, B=1) == 5
    assert fwd(L, cu=P[13], nseq=1 << 60, B=1) == 2
    assert fwd(L, cu=P[13], nseq=3, B=1, hi=P[5]) == 6
    assert fwd(L, cu=P[13], nseq=3, B=1, y=P[13]) == 6
    # nothing to do
    assert fwd(L, B=0, x=0, r=0, i=0, y=0, hf=0, carry=0) == 0
    assert fwd(L, D=0, x=0, r=0, i=0, A=0, y=0, hf=0, carry=0) == 0
    assert fwd(L, T=0, x=0, r=0, i=0, y=0, hf=None, carry=0) == 0
    assert fwd(L, T=0, x=0, r=0, i=0, y=0, hi=P[5], hf=P[5], carry=0) == 0
    assert L.ssm_last_error() == b""


def test_gated_backward_refusals(L):
    assert bwd(L, B=-1) == 2 and bwd(L, T=-1) == 2 and bwd(L, B=1, D=(1 << 22) + 1) == 2
    for k in ("r", "i", "A", "dy", "dx", "dr", "di", "dA"):
        assert bwd(L, **{k: 0}) == 1, k
    for k in ("dx", "dr", "di", "dA", "dhi"):
        assert bwd(L, **{k: P[0]}) == 6 and bwd(L, **{k: P[7]}) == 6 and bwd(L, **{k: P[6]}) == 6, k
    assert bwd(L, dr=P[8]) == 6 and bwd(L, dA=P[12]) == 6
    assert bwd(L, hi=P[12], dhi=P[12]) == 6 and bwd(L, dhf=P[12], dhi=P[12]) == 6
    assert bwd(L, cu=P[13], nseq=3, B=2) == 2 and bwd(L, cu=P[13], nseq=0, B=1) == 2
    assert bwd(L, carry=P[6] + 2) == 5
    assert bwd(L, D=0, x=0, r=0, i=0, A=0, dy=0, dx=0, dr=0, di=0, dA=0, dhi=0, carry=0) == 0
    assert L.ssm_gated_carry_steps() > 0


def test_gated_step_refusals(L):
    assert step(L, B=-1) == 2 and step(L, B=1 << 20, D=1 << 20) == 2
    for k in ("r", "i", "A", "h", "ho", "y"):
        assert step(L, **{k: 0}) == 1, k
    assert step(L, ho=P[4] + 4) == 6 and step(L, y=P[4]) == 6 and step(L, y=P[5]) == 6 and step(L, ho=P[3]) == 6
    assert step(L, h=P[4] + 2) == 5
    assert step(L, B=0, x=0, r=0, i=0, A=0, h=0, ho=0, y=0) == 0
    assert step(L, D=0, x=0, r=0, i=0, A=0, h=0, ho=0, y=0) == 0


def test_norm_refusals(L):
    assert norm(L, rows=-1) == 2 and norm(L, group=0) == 2 and norm(L, group=3) == 2 and norm(L, group=-8) == 2
    assert norm(L, D=(1 << 20) + 1, group=(1 << 20) + 1) == 2
    assert norm(L, rows=1 << 28, D=64, group=1) == 2
    assert norm(L, eps=-1.0) == 9 and norm(L, eps=float("nan")) == 9
    assert norm(L, res=0) == 1 and b"residual" in L.ssm_last_error()
    assert norm(L, y=0) == 1
    assert norm(L, w=P[2] + 2) == 5 and norm(L, mean=P[6] + 1) == 5
    assert norm(L, y=P[0]) == 6 and norm(L, s=P[5]) == 6 and norm(L, y=P[1]) == 6 and norm(L, s=P[0]) == 6
    assert norm(L, s=P[1] + 2) == 6 and norm(L, rstd=P[6]) == 6 and norm(L, mean=P[2]) == 6
    assert norm(L, rows=0, x=0, res=0, y=0, s=0, mean=0, rstd=0) == 0


def test_norm_backward_refusals(L):
    assert normb(L, rows=-1) == 2 and normb(L, group=0) == 2 and normb(L, group=5) == 2
    for k in ("mean", "rstd", "dy", "dx"):
        assert normb(L, **{k: 0}) == 1, k
    for k in ("dx", "dw", "db"):
        assert normb(L, **{k: P[0]}) == 6 and normb(L, **{k: P[5]}) == 6 and normb(L, **{k: P[3]}) == 6
    assert normb(L, dw=P[8]) == 6 and normb(L, dx=P[7]) == 6
    assert normb(L, dw=P[7] + 2) == 5
    assert normb(L, rows=0, D=0, group=1, s=0, w=0, mean=0, rstd=0, dy=0, dsum=0, dx=0, dw=0, db=0) == 0


def test_binding_refuses_host_tensors_and_bad_groups():
    import torch

    from selective_state_space_18_amd import ssmscan as ss
    t = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):
        ss.scan_gated_fwd(t, t, t, torch.zeros(4))
    with pytest.raises(ValueError):
        ss.scan_gated_bwd(t, t, t, torch.zeros(4), t)
    with pytest.raises(ValueError):
        ss.step_gated(t[0], t[0], t[0], torch.zeros(4), torch.zeros(3, 4))
    with pytest.raises(ValueError):
        ss.layer_norm_fwd(t)
    with pytest.raises(ValueError):
        ss.layer_norm_bwd(t, None, t, t, t)
