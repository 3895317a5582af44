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


def whole(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device=DEV, dtype=torch.int8).to(dtype)


@pytest.mark.slow
@pytest.mark.parametrize("Dv", [8, 72])
def test_many_sequences_of_many_heads(ss, Dv):
    """2^18 sequences of 64 heads, one step each but for some empty ones and one of
    1000: more blocks than one launch takes.  Whole numbers, so results are exact."""
    print(f"case: linear attention 2^24 blocks, Dv {Dv}", flush=True)
    n, H, Dk = 2 ** 18 + 3, 64, 8
    lens = torch.ones(n, dtype=torch.int64)
    lens[::1000] = 0
    lens[7] = 1000
    cu = torch.zeros(n + 1, dtype=torch.int64)
    cu[1:] = lens.cumsum(0)
    L, cu = int(cu[-1]), cu.to(DEV)
    q, k, v, dy = whole((L, H, Dk), 1), whole((L, H, Dk), 2), whole((L, H, Dv), 3), whole((L, H, Dv), 4)
    a = torch.full((H,), float("-inf"), device=DEV)  # no memory: every step by itself
    f = ss.linear_attn_fwd(q, k, v, a, cu_seqlens=cu, scale=1.0)
    b = ss.linear_attn_bwd(q, k, v, a, dy, cu_seqlens=cu, scale=1.0, want_dh_init=False)
    torch.cuda.synchronize()
    dot = lambda x, y: (x.float() * y.float()).sum(-1, keepdim=True)
    assert torch.equal(f["y"].float(), dot(q, k) * v)
    last = (cu[1:] - 1)[lens.to(DEV) > 0]
    at = torch.nonzero(lens.to(DEV) > 0).squeeze(1)
    for i in range(0, len(at), 2 ** 15):
        j = last[i:i + 2 ** 15]
        assert torch.equal(f["h_final"][at[i:i + 2 ** 15]], v[j, :, :, None].float() * k[j, :, None, :].float()), i
    assert (f["h_final"][::1000] == 0).all()
    assert torch.equal(b["dq"].float(), dot(dy, v) * k) and torch.equal(b["dk"].float(), dot(dy, v) * q)
    assert torch.equal(b["dv"].float(), dot(q, k) * dy)


@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_a_capture_with_too_little_scratch_records_nothing(ss, direction):
    print(f"case: linear attention capture without scratch {direction}", flush=True)
    H, D = 2, 64
    q = whole((40, H, D), 2)
    cu = torch.tensor([0, 0, 40, 40], device=DEV)
    a, y, state = torch.zeros(H, device=DEV), torch.full_like(q, 7.0), torch.full((3, H, D, D), 7.0, device=DEV)
    out = [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    ss.release_workspaces()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    mark = torch.zeros(4, device=DEV)
    with torch.cuda.graph(g, stream=s):
        with pytest.raises(ss.SSMError) as e:
            if direction == "forward":
                ss.linear_attn_fwd(q, q, q, a, cu_seqlens=cu, out={"y": y, "h_final": state})
            else:
                ss.linear_attn_bwd(q, q, q, a, q, cu_seqlens=cu,
                                   out={"dq": y, "dk": out[0], "dv": out[1], "dh_init": state})
        mark.add_(1.0)  # (the graph is not empty)
    assert e.value.code == 10
    g.replay()
    torch.cuda.synchronize()
    assert (mark == 1).all() and (y == 7).all() and (state == 7).all()


@pytest.mark.slow
def test_short_forced_parts_of_many_heads(ss):
    """Parts of 64 steps would be 2^23 + 1024 blocks: they are made longer.  Whole
    numbers without decay: sums stay below 2^24, so every cut gives the same bits."""
    print("case: linear attention parts of many heads", flush=True)
    H, D, L = 1024, 8, 2 ** 19 + 64
    q, k, v = whole((1, L, H, D), 3), whole((1, L, 1, D), 4), whole((1, L, 1, D), 5)
    a = torch.zeros(H, device=DEV)
    cu = torch.tensor([0, 5, L // 3, L], device=DEV)
    for args in ((q, k, v), (q[0], k[0], v[0])):
        kw = dict(scale=1.0, cu_seqlens=None if args[0].dim() == 4 else cu)
        want = ss.linear_attn_fwd(*args, a, **kw)
        ss.set_option(ss.SSM_OPT_SEGMENT_LEN, 64)
        try:
            got = ss.linear_attn_fwd(*args, a, **kw)
        finally:
            ss.set_option(ss.SSM_OPT_SEGMENT_LEN, 0)
        assert torch.equal(got["y"], want["y"]) and torch.equal(got["h_final"], want["h_final"])
        assert want["h_final"].abs().max() > 100
        del want, got


def test_scratch_of_many_short_sequences(ss):
    """4096 documents, nearly all of one part: states are kept for parts with a
    predecessor (257 MB at most here), not for every document (4.5 GB)."""
    print("case: linear attention scratch of short documents", flush=True)
    n, H, D = 4096, 16, 128
    lens = torch.full((n,), 12)
    lens[5], lens[77], lens[-1] = 3000, 2049, 257
    lens[100:100 + n // 8] = 0
    cu = torch.zeros(n + 1, dtype=torch.int64)
    cu[1:] = lens.cumsum(0)
    L = int(cu[-1])
    q, k, v, dy = (whole((L, H, D), i) for i in range(4))
    a = torch.zeros(H, device=DEV)
    cu = cu.to(DEV)
    y, grads = torch.empty_like(q), [torch.empty_like(q) for _ in range(3)]

    def both(part):
        ss.set_option(ss.SSM_OPT_SEGMENT_LEN, part)
        try:
            ss.linear_attn_fwd(q, k, v, a, cu_seqlens=cu, scale=1.0, want_state=False, out={"y": y})
            ss.linear_attn_bwd(q, k, v, a, dy, cu_seqlens=cu, scale=1.0, want_dh_init=False,
                               out=dict(zip(("dq", "dk", "dv"), grads)))
        finally:
            ss.set_option(ss.SSM_OPT_SEGMENT_LEN, 0)
        torch.cuda.synchronize()
        return [t.clone() for t in (y, *grads)]
    want = both(8192)  # one part a document
    ss.release_workspaces()
    free = torch.cuda.mem_get_info()[0]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = both(256)
    used = free - torch.cuda.mem_get_info()[0]
    # (whole numbers without decay: every cut gives the same bits)
    assert all(torch.equal(x, w) for x, w in zip(got, want))
    assert used < 1 << 30, used
