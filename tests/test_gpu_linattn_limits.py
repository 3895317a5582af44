"""Linear attention's calls at the sizes that the interface still takes."""
import pytest
import torch

from test_gpu_linattn import DEV, ss  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.slow
@pytest.mark.parametrize("states", [2 ** 23, 2 ** 24 - 8], ids=["2^23", "2^24-8"])
def test_decode_step_of_many_states(ss, states):
    """More than 2^32 threads' worth of states.  Whole numbers, no decay: every result is exact."""
    H, Dk, Dv = 8, 8, 128
    B = states // H
    need = states * Dk * Dv * 4 * 1.3
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need / 2 ** 30:.0f} GiB")
    print(f"case: linear attention step of {states} states", flush=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    q, k, v = whole(B, H, Dk), whole(B, H, Dk), whole(B, H, Dv)
    h = torch.ones(B, H, Dv, Dk, device=DEV)
    y = ss.step_linear_attn(q, k, v, torch.zeros(H, device=DEV), h, scale=1.0)
    torch.cuda.synchronize()
    for at in range(0, B, 2 ** 17):
        n = slice(at, at + 2 ** 17)
        want = 1 + v[n, :, :, None].float() * k[n, :, None, :].float()
        assert torch.equal(h[n], want), at
        assert torch.equal(y[n].float(), (want * q[n, :, None, :].float()).sum(-1)), at
