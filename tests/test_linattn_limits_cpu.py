"""Linear attention's limits of sequences times heads at the C ABI, on the CPU."""
import pytest

from test_attn_abi_cpu import L, P, bwd, fwd  # noqa: F401 (fixture)


@pytest.mark.parametrize("f", [fwd, bwd])
def test_states_times_heads(L, f):
    """More than 2^30 are refused before anything else is looked at; at the limit
    the call goes on to its pointers (here too close together)."""
    for B, H in ((1 << 28, 5), (1 << 20, 1025), ((1 << 29) + 1, 2)):
        assert f(L, B=B, T=1, H=H, Hkv=H, Dk=8, Dv=8) == 2 and b"2^30" in L.ssm_last_error(), (B, H)
        assert f(L, cu=P[13], nseq=B, B=1, T=5, H=H, Hkv=H, Dk=8, Dv=8) == 2 and b"2^30" in L.ssm_last_error(), (B, H)
    for B, H in ((1 << 28, 4), (1 << 20, 1024), (1 << 20, 9), (1 << 29, 2)):
        assert f(L, B=B, T=1, H=H, Hkv=H, Dk=8, Dv=8) == 6, (B, H)
        assert f(L, cu=P[13], nseq=B, B=1, T=5, H=H, Hkv=H, Dk=8, Dv=8) == 6, (B, H)
    # without steps nothing is cut
    assert f(L, B=1 << 28, T=0, H=8, Hkv=8, Dk=8, Dv=8) != 2
