"""Linear attention's parts of the time axis on the GPU: few (summed by the output
pass) and many (carried), both in one packed call, and calls that a graph records
before they ever ran."""
import pytest
import torch

import _attn as T
from test_gpu_linattn import DEV, parts_of, run, ss  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dims", [(128, 128), (96, 128), (96, 64), (64, 64), (24, 104)], ids=str)
def test_few_and_many_parts(ss, parts_of, dims, dtype):
    print(f"case: linear attention few and many parts {dims} {dtype}", flush=True)
    o = T.linear_inputs((2, 600), 2, 1, *dims, 21, dtype, DEV)
    for part in (64, 128):  # 10 parts a row, 5 parts
        parts_of(part)
        T.check_linear(run(ss, o), o, dims[0] ** -0.5, dtype, f"parts of {part}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_and_many_parts_in_one_call(ss, parts_of, dtype):
    """Sequences of 8, 9, 1, no and 10 parts next to each other."""
    print(f"case: linear attention mixed parts {dtype}", flush=True)
    parts_of(64)
    cu = [0, 512, 1025, 1060, 1060, 1660]
    o = T.linear_inputs((cu[-1],), 2, 1, 64, 96, 31, dtype, DEV, rows=5)
    T.check_linear(run(ss, o, cu), o, 0.125, dtype, "mixed", cu)


@pytest.mark.parametrize("L", [500, 700])  # 8 parts and 11
def test_initial_state_may_be_replaced_with_many_parts(ss, parts_of, L):
    print(f"case: linear attention h_final = h_init, {L} steps", flush=True)
    parts_of(64)
    o = T.linear_inputs((2, L), 2, 2, 128, 64, 41, "bf16", DEV, grads=False)
    want = run(ss, o, grads=False)
    h = o["h_init"].clone()
    got = ss.linear_attn_fwd(o["q"], o["k"], o["v"], o["log_decay"], h_init=h, out={"h_final": h})
    assert torch.equal(got["y"], want["y"]) and torch.equal(h, want["h_final"])


def test_strong_decay_over_many_parts(ss, parts_of):
    """A decay whose power over a part is 0, next to ones that hardly fade."""
    print("case: linear attention strong and weak decays over parts", flush=True)
    parts_of(64)
    o = T.linear_inputs((1, 640), 4, 2, 64, 64, 51, "bf16", DEV)
    o["log_decay"] = torch.tensor([-1e5, -3.0, -1e-7, 0.0], device=DEV)
    T.check_linear(run(ss, o), o, 0.125, "bf16", "decays over parts")


def test_a_graph_may_record_the_first_call(ss):
    """Nothing but the stream's scratch has to be there: no kernel of these sizes ran before."""
    print("case: linear attention recorded first", flush=True)
    s = torch.cuda.Stream()
    big = T.linear_inputs((1, 4096), 4, 4, 128, 128, 61, "fp32", DEV)
    with torch.cuda.stream(s):
        ss.linear_attn_bwd(big["q"], big["k"], big["v"], big["log_decay"], big["dy"])
    s.synchronize()
    o = T.linear_inputs((2, 300), 2, 2, 88, 112, 62, "bf16", DEV)
    out = {"y": torch.zeros(2, 300, 2, 112, dtype=torch.bfloat16, device=DEV),
           "h_final": torch.zeros(2, 2, 112, 88, device=DEV)}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ss.linear_attn_fwd(o["q"], o["k"], o["v"], o["log_decay"], h_init=o["h_init"], out=out)
    want = run(ss, o, grads=False)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in out)
    T.check_linear(want, o, 88 ** -0.5, "bf16", "recorded first")
