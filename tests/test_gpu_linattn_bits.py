"""Linear attention's bits on the GPU: inputs for which every product and sum is
exact in 32 bits, so that a result is the one rounding of an exactly known value
to its storage type, and an operand cut to fewer bits is seen.

The values lie next to the middle between two neighbours of bf16 (8 significant
bits): what decides the rounding is a distance of 2^-23 to 2^-18 from it, which
two bf16 terms of the operand (16 bits) lose.
"""
import pytest
import torch

import _attn as T
from test_gpu_linattn import DEV, parts_of, ss  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (128, 128), (64, 128), (128, 64), (96, 96), (40, 72)]


def near_middles(*shape):
    """fp32 values (1 + odd 2^-8 + d) 2^j, d of either sign and down to 2^-23 (one unit)."""
    n = torch.arange(torch.Size(shape).numel(), dtype=torch.float64)
    d = torch.tensor([2.0 ** -23, -(2.0 ** -23), 2.0 ** -20, -(2.0 ** -20), 2.0 ** -18, -(2.0 ** -18), 3 * 2.0 ** -21])
    x = (1 + (2 * (n % 64) + 1) * 2.0 ** -8 + d.double()[(n % 7).long()]) * 2.0 ** (n % 5 - 2) * (1 - 2 * (n % 3 == 1).double())
    f = x.float()
    assert torch.equal(f.double(), x)  # 24 bits hold them
    return f.view(shape).to(DEV)


def one_hot(L, D, H, dtype):
    """[1, L, H, D]: step t has a one at t modulo D."""
    t = torch.zeros(L, D)
    t[torch.arange(L), torch.arange(L) % D] = 1.0
    return t.to(T.DT[dtype])[None, :, None].expand(1, L, H, D).contiguous().to(DEV)


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dims", DIMS, ids=str)
def test_states_enter_products_with_all_their_bits(ss, parts_of, dims, dtype, part):
    """y and dq of a state that stays as it is (no decay, no k), dk and dv of an
    adjoint state that does (no dy): one value of the state each."""
    print(f"case: linear attention bits of a state {dims} {dtype} {part}", flush=True)
    parts_of(part)
    (Dk, Dv), H, L, t = dims, 2, 200, T.DT[dtype]
    a = torch.zeros(H, device=DEV)
    state = near_middles(1, H, Dv, Dk)
    by_k, by_v = state[0].permute(2, 0, 1), state[0].transpose(1, 2).permute(2, 0, 1)  # [Dk, H, Dv], [Dv, H, Dk]
    at = torch.arange(L, device=DEV)
    ek, ev = one_hot(L, Dk, H, dtype), one_hot(L, Dv, H, dtype)
    zk, zv = torch.zeros_like(ek), torch.zeros_like(ev)
    f = ss.linear_attn_fwd(ek, zk, zv, a, h_init=state, scale=1.0)
    assert torch.equal(f["y"][0], by_k[at % Dk].to(t)) and torch.equal(f["h_final"], state)
    g = ss.linear_attn_bwd(ek, zk, zv, a, ev, h_init=state, scale=1.0)
    assert torch.equal(g["dq"][0], by_v[at % Dv].to(t))
    g = ss.linear_attn_bwd(zk, ek, ev, a, zv, dh_final=state, scale=1.0)
    assert torch.equal(g["dv"][0], by_k[at % Dk].to(t)) and torch.equal(g["dk"][0], by_v[at % Dv].to(t))
    assert torch.equal(g["dh_init"], state)
    # a shared head of k and v: the second head's adjoint state is zero
    state[:, 1] = 0
    g = ss.linear_attn_bwd(zk, ek[:, :, :1].contiguous(), ev[:, :, :1].contiguous(), a, zv, dh_final=state, scale=1.0)
    assert torch.equal(g["dv"][0], by_k[at % Dk].to(t)[:, :1]) and torch.equal(g["dk"][0], by_v[at % Dv].to(t)[:, :1])


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dims", DIMS, ids=str)
def test_weights_enter_products_with_all_their_bits(ss, parts_of, dims, dtype, part):
    """The scale is the weight of every score, and in the backward of every step
    in a state."""
    print(f"case: linear attention bits of a weight {dims} {dtype} {part}", flush=True)
    parts_of(part)
    (Dk, Dv), H = dims, 2
    a = torch.zeros(H, device=DEV)
    low = min(Dk, Dv)
    L = 3 * low
    # steps repeat after `low` of them; of q and dy the last `low` steps are there, of k and v all
    ek, ev = one_hot(L, low, H, dtype), one_hot(L, low, H, dtype)
    ek, ev = (torch.nn.functional.pad(e, (0, D - low)) for e, D in ((ek, Dk), (ev, Dv)))
    last = (torch.arange(L, device=DEV) >= L - low).view(1, L, 1, 1)
    for scale in near_middles(24).tolist():
        want = torch.tensor(scale).to(T.DT[dtype]).to(DEV)
        # scores of the last steps alone: y_t = scale v_t
        f = ss.linear_attn_fwd(ek, ek * last, ev * last, a, scale=scale)
        assert torch.equal(f["y"], ev * last * want), scale
        # every dk_t and dv_t has one term, from inside its chunk or through the adjoint state
        g = ss.linear_attn_bwd(ek * last, ek, ev, a, ev * last, scale=scale)
        assert torch.equal(g["dv"], ev * want) and torch.equal(g["dk"], ek * want), scale
        # dq_t: v_s and k_s of the first steps, through the state
        g = ss.linear_attn_bwd(ek * last, ek * ~last, ev * ~last, a, ev * last, scale=scale)
        assert torch.equal(g["dq"], ek * last * (2 * torch.tensor(scale)).to(want.dtype).to(DEV)), scale


def test_a_part_adds_steps_with_all_their_bits(ss, parts_of):
    """States of steps that are weighted one by one in the first of three parts:
    each value has one term.  Its weight is off by (3 |n a| + 3) e (e = 2^-24), the
    product by 1 e, its sum of terms by 2^-27 of it, the two states' fading by 2 e
    each (a factor and a product): 3 |n a| + 9 in units of e, where two bf16
    terms lose up to 64."""
    print("case: linear attention bits of a part's sum", flush=True)
    parts_of(64)
    for dims in DIMS:
        (Dk, Dv), H, L = dims, 3, 192
        a = torch.tensor([-0.001, -0.005, -0.02], device=DEV)
        k = one_hot(L, Dk, H, "bf16")
        k[:, min(64, Dk):] = 0
        v = T.make((1, L, H, Dv), 5, "bf16", DEV)
        f = ss.linear_attn_fwd(k, k, v, a, scale=1.0)
        n = min(64, Dk)
        back = (L - 1 - torch.arange(n, dtype=torch.float64))[:, None] * a.double().cpu()
        want = (torch.exp(back)[:, :, None] * v[0, :n].double().cpu()).permute(1, 2, 0)  # [H, Dv, n]
        bound = want.abs() * (3 * 64 * a.abs().double().cpu()[:, None, None] + 9) * T.E32
        got = f["h_final"][0].double().cpu()
        assert (got[:, :, n:] == 0).all()
        assert ((got[:, :, :n] - want).abs() <= bound).all(), (dims, ((got[:, :, :n] - want).abs() / bound).max())
