"""Linear attention's packed calls whose sequences leave steps of the row over, as a
padded batch does: those steps of every output stay as they were."""
import pytest
import torch

import _attn as T
from test_gpu_linattn import DEV, parts_of, ss  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(4, 4), (4, 2), (6, 1)], ids=str)
def test_steps_of_no_sequence_are_left_by_the_backward(ss, parts_of, heads, dtype, part):
    print(f"case: linear attention rest of the row, backward {heads} {dtype} {part}", flush=True)
    parts_of(part)
    (H, Hkv), Dk, Dv, L = heads, 64, 72, 300
    # what an earlier call left in the scratch is no number
    o = T.linear_inputs((2, 400), H, Hkv, Dk, Dv, 1, dtype, DEV, state=False)
    ss.linear_attn_bwd(o["q"], o["k"], o["v"], o["log_decay"], torch.full_like(o["dy"], float("nan")))
    for cu in ([0, 30, 30, 211], [0, 0, 0, 1], [17, 40, 150, 299]):
        o = T.linear_inputs((L,), H, Hkv, Dk, Dv, 2, dtype, DEV, rows=3)
        first, last = cu[0], cu[-1]
        out = {n: torch.full_like(o[n[1:]], 7.0) for n in ("dq", "dk", "dv")}
        ss.linear_attn_bwd(o["q"], o["k"], o["v"], o["log_decay"], o["dy"], dh_final=o["dh_final"], h_init=o["h_init"],
                           cu_seqlens=torch.tensor(cu, device=DEV), scale=0.125, out=out)
        for n, t in out.items():
            assert (t[:first] == 7).all() and (t[last:] == 7).all(), (cu, n)
        used = {n: o[n][first:last].contiguous() for n in ("q", "k", "v", "dy")}
        used.update({n: o[n] for n in ("log_decay", "h_init", "dh_final")})
        ref, err = T.linear_reference(used, 0.125, [c - first for c in cu], dtype)
        for n, t in out.items():
            T.check(t[first:last], ref[n], T.stored(ref[n], err[n], dtype), n)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padded_rows_of_a_captured_backward(ss, dtype):
    """The borders are read when the graph replays: other sequences, other steps left."""
    print(f"case: linear attention rest of the row, captured {dtype}", flush=True)
    H, Hkv, D, L = 4, 2, 64, 260
    o = T.linear_inputs((L,), H, Hkv, D, D, 3, dtype, DEV, rows=2, state=False)
    cu = torch.tensor([0, 100, 260], device=DEV)
    out = {n: torch.zeros_like(o[n[1:]]) for n in ("dq", "dk", "dv")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: ss.linear_attn_bwd(o["q"], o["k"], o["v"], o["log_decay"], o["dy"], cu_seqlens=cu, scale=0.125,
                                      want_dh_init=False, out=out)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for end in (260, 201, 100, 259):
        cu.copy_(torch.tensor([0, 100, end], device=DEV))
        for t in out.values():
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        used = {n: o[n][:end].contiguous() for n in ("q", "k", "v", "dy")}
        ref, err = T.linear_reference({**used, "log_decay": o["log_decay"]}, 0.125, [0, 100, end], dtype)
        for n, t in out.items():
            assert (t[end:] == 7).all(), (end, n)
            T.check(t[:end], ref[n], T.stored(ref[n], err[n], dtype), n)
