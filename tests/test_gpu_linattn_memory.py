"""Linear attention on the GPU over a million steps of weak decay, and a call that a
graph records before the process ran any other of its kernels."""
import os
import subprocess
import sys

import pytest
import torch

import _attn as T
import _attn_memory as M
from test_gpu_linattn import DEV, parts_of, ss  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dims", [(8, 8), (16, 4 * 24)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_memory_fades_without_bias(ss, parts_of, dtype, dims):
    """States without new steps, 2^20 of them in one part: the factors of 16384 or 32768
    chunks, forward and backward, to the bounds of _attn_memory."""
    print(f"case: linear attention long fading {dtype} {dims}", flush=True)
    parts_of(M.STEPS)
    (Dk, Dv), H = dims, M.HEADS
    chunk = 64 if dtype == "bf16" else 32
    a = M.decays(chunk)
    value, mean = M.bounds(chunk)  # (a mean over M.DK * M.DV values or more)
    assert Dk * Dv >= M.DK * M.DV
    t = T.DT[dtype]
    zk, zv = (torch.zeros(1, M.STEPS, 1, D, dtype=t, device=DEV) for D in dims)
    q, dy = (torch.zeros(1, M.STEPS, H, D, dtype=t, device=DEV) for D in dims)
    h = T.make((1, H, Dv, Dk), 5, "fp32", DEV)
    decay = torch.from_numpy(a).to(DEV)
    want = h[0].double().cpu().flatten(1) * torch.exp(torch.from_numpy(a).double() * M.STEPS)[:, None]
    f = ss.linear_attn_fwd(q, zk, zv, decay, h_init=h)
    g = ss.linear_attn_bwd(q, zk, zv, decay, dy, dh_final=h)
    for name, got in (("h_final", f["h_final"]), ("dh_init", g["dh_init"])):
        off = M.worst((got[0].double().cpu().flatten(1) / want).numpy())
        assert off[0] <= value and off[1] <= mean, (name, off, value, mean)


CHILD = """
import torch
import _attn as T
from selective_state_space_18_amd import ssmscan as ss
s = torch.cuda.Stream()
big = T.linear_inputs((1, 4096), 4, 4, 64, 64, 61, "fp32", "cuda:0")
with torch.cuda.stream(s):  # sizes the stream's scratch, with kernels of the other storage type
    ss.linear_attn_bwd(big["q"], big["k"], big["v"], big["log_decay"], big["dy"])
s.synchronize()
o = T.linear_inputs((2, 300), 4, 2, 128, 96, 62, "bf16", "cuda:0")
args = (o["q"], o["k"], o["v"], o["log_decay"])
out = {"y": torch.zeros_like(o["dy"]), "h_final": torch.zeros_like(o["h_init"])}
grads = {"dq": torch.zeros_like(o["q"]), "dk": torch.zeros_like(o["k"]), "dv": torch.zeros_like(o["v"]),
         "dh_init": torch.zeros_like(o["h_init"])}
def both(a, b):
    a = ss.linear_attn_fwd(*args, h_init=o["h_init"], out=a)
    return {**a, **ss.linear_attn_bwd(*args, o["dy"], h_init=o["h_init"], dh_final=o["dh_final"], out=b)}
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    both(out, grads)
want = both(None, None)
for _ in range(3):
    for t in (*out.values(), *grads.values()):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for n, t in {**out, **grads}.items():
        assert torch.equal(t, want[n]), n
T.check_linear(want, o, 128 ** -0.5, "bf16", "recorded first")
print("recorded first: ok", flush=True)
"""


def test_a_graph_may_record_the_first_call_of_a_process(ss):
    print("case: linear attention recorded first, in a process of its own", flush=True)
    env = {**os.environ, "PYTHONPATH": os.pathsep.join((ROOT, os.path.join(ROOT, "tests")))}
    r = subprocess.run([sys.executable, "-u", "-c", CHILD], cwd=ROOT, env=env, timeout=100, capture_output=True, text=True)
    assert r.returncode == 0 and "recorded first: ok" in r.stdout, (r.stdout, r.stderr)
