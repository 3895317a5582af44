"""Linear attention on the GPU against its fp64 definition, within derived
bounds: dense and packed, forward, backward, decode step."""
import pytest
import torch

import _attn as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ss():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_18_amd import ssmscan
    ssmscan.lib()
    return ssmscan


@pytest.fixture
def parts_of(ss):
    """Sets the parts' length for a test."""
    yield lambda n: ss.set_option(ss.SSM_OPT_SEGMENT_LEN, n)
    ss.set_option(ss.SSM_OPT_SEGMENT_LEN, 0)


def run(ss, o, cu=None, scale=None, grads=True):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)
    got = ss.linear_attn_fwd(o["q"], o["k"], o["v"], o["log_decay"], cu_seqlens=c, h_init=o["h_init"], scale=scale)
    if grads:
        got.update(ss.linear_attn_bwd(o["q"], o["k"], o["v"], o["log_decay"], o["dy"], cu_seqlens=c,
                                      h_init=o["h_init"], dh_final=o["dh_final"], scale=scale))
    torch.cuda.synchronize()
    return got


SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 2, 1, 16, 24), (1, 31, 3, 3, 64, 64), (1, 32, 2, 2, 128, 128),
          (2, 33, 4, 2, 128, 64), (1, 63, 2, 2, 64, 128), (3, 64, 6, 2, 128, 128), (1, 65, 1, 1, 128, 128),
          (2, 100, 5, 5, 96, 96), (1, 127, 4, 1, 72, 40), (1, 129, 2, 2, 40, 72), (2, 200, 3, 1, 128, 120),
          (1, 257, 2, 2, 64, 64), (1, 320, 2, 2, 128, 128), (1, 300, 8, 2, 32, 128), (1, 190, 1, 1, 128, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dense(ss, shape, dtype):
    B, L, H, Hkv, Dk, Dv = shape
    print(f"case: linear attention {shape} {dtype}", flush=True)
    o = T.linear_inputs((B, L), H, Hkv, Dk, Dv, 7 * L + Dk, dtype, DEV)
    T.check_linear(run(ss, o), o, Dk ** -0.5, dtype, "states")
    o["h_init"] = o["dh_final"] = None
    T.check_linear(run(ss, o, scale=1.5), o, 1.5, dtype, "no states")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dims", [(128, 128), (64, 128), (128, 64), (64, 64), (96, 80)], ids=str)
@pytest.mark.parametrize("part", [64, 128, 192])
def test_parts_of_the_time_axis(ss, parts_of, part, dims, dtype):
    """Parts joined by their states give the whole, forward and backward."""
    print(f"case: linear attention parts {part} {dims} {dtype}", flush=True)
    parts_of(part)
    o = T.linear_inputs((2, 333), 4, 2, *dims, part, dtype, DEV)
    T.check_linear(run(ss, o), o, dims[0] ** -0.5, dtype, "parts")
    cu = [0, 0, 64, 65, 200, 200, 328, 333]
    o = T.linear_inputs((333,), 4, 2, *dims, part + 1, dtype, DEV, rows=7)
    T.check_linear(run(ss, o, cu), o, dims[0] ** -0.5, dtype, "packed parts", cu)


BORDERS = [[0, 1], [0, 0, 1, 1], [0, 64, 128], [0, 5, 5, 69, 70, 200], [0, 0, 0, 130], [0, 130, 130, 130],
           [0, 1, 2, 3, 4, 5, 40, 41], [0, 63, 127, 192, 256, 257]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", BORDERS, ids=str)
def test_packed(ss, cu, dtype):
    print(f"case: linear attention packed {cu} {dtype}", flush=True)
    n, L = len(cu) - 1, cu[-1]
    o = T.linear_inputs((L,), 4, 2, 64, 96, L + n, dtype, DEV, rows=n)
    T.check_linear(run(ss, o, cu), o, 0.125, dtype, "packed", cu)
    o["h_init"] = o["dh_final"] = None
    T.check_linear(run(ss, o, cu), o, 0.125, dtype, "packed, no states", cu)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("decay", [0.0, -1e-6, -1e-3, -0.7, -5.0, -40.0, -1e5, float("-inf")])
def test_decays(ss, parts_of, decay, dtype):
    """From a sum over everything to no memory at all."""
    print(f"case: linear attention decay {decay} {dtype}", flush=True)
    parts_of(128)
    o = T.linear_inputs((1, 300), 2, 2, 64, 128, 11, dtype, DEV, decay=decay)
    T.check_linear(run(ss, o), o, 0.125, dtype, "decay")


def test_initial_state_may_be_replaced(ss, parts_of):
    print("case: linear attention h_final = h_init", flush=True)
    for part in (0, 64):
        parts_of(part)
        o = T.linear_inputs((2, 260), 3, 3, 128, 128, 5, "bf16", DEV, grads=False)
        want = run(ss, o, grads=False)
        h = o["h_init"].clone()
        got = ss.linear_attn_fwd(o["q"], o["k"], o["v"], o["log_decay"], h_init=h, out={"h_final": h})
        assert torch.equal(got["y"], want["y"]) and torch.equal(h, want["h_final"])


def test_no_steps(ss):
    print("case: linear attention without steps", flush=True)
    o = T.linear_inputs((2, 0), 3, 3, 64, 64, 5, "bf16", DEV)
    got = run(ss, o)
    assert torch.equal(got["h_final"], o["h_init"]) and torch.equal(got["dh_init"], o["dh_final"])
    o["h_init"] = o["dh_final"] = None
    got = run(ss, o)
    assert (got["h_final"] == 0).all() and (got["dh_init"] == 0).all()
    o = T.linear_inputs((0,), 3, 3, 64, 64, 6, "bf16", DEV, rows=4)
    got = run(ss, o, [0] * 5)
    assert torch.equal(got["h_final"], o["h_init"]) and torch.equal(got["dh_init"], o["dh_final"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 8, 8), (3, 4, 2, 128, 128), (2, 6, 1, 40, 72), (5, 2, 2, 96, 120),
                                   (2, 3, 3, 64, 8), (65, 8, 8, 128, 64)], ids=str)
def test_decode_step(ss, shape, dtype):
    B, H, Hkv, Dk, Dv = shape
    print(f"case: linear attention step {shape} {dtype}", flush=True)
    o = T.linear_inputs((B, 1), H, Hkv, Dk, Dv, B + Dk, dtype, DEV, grads=False)
    q, k, v = (o[n][:, 0].contiguous() for n in ("q", "k", "v"))
    h = o["h_init"].clone()
    ho = torch.empty_like(h)
    y = ss.step_linear_attn(q, k, v, o["log_decay"], h, h_out=ho)
    torch.cuda.synchronize()
    assert torch.equal(h, o["h_init"])
    T.check_linear({"y": y[:, None], "h_final": ho}, o, Dk ** -0.5, dtype, "step")
    y2 = ss.step_linear_attn(q, k, v, o["log_decay"], h)
    assert torch.equal(y2, y) and torch.equal(h, ho)


def test_steps_follow_the_prompt(ss):
    """A prompt, then single steps from its state, against the whole."""
    print("case: linear attention prompt and steps", flush=True)
    o = T.linear_inputs((2, 90), 4, 2, 128, 64, 21, "bf16", DEV, grads=False)
    head = {n: o[n][:, :70].contiguous() for n in ("q", "k", "v")}
    f = ss.linear_attn_fwd(head["q"], head["k"], head["v"], o["log_decay"], h_init=o["h_init"])
    h, ys = f["h_final"], [f["y"]]
    for t in range(70, 90):
        ys.append(ss.step_linear_attn(*(o[n][:, t].contiguous() for n in ("q", "k", "v")), o["log_decay"], h)[:, None])
    T.check_linear({"y": torch.cat(ys, 1), "h_final": h}, o, 128 ** -0.5, "bf16", "steps")


def test_gradients_against_differences(ss):
    """fp32: directional derivatives of a weighted sum of y and h_final.  The
    sum is linear in each of q, k, v, h_init, so a central difference has no
    truncation error; what is left is the rounding of both sides."""
    print("case: linear attention differences", flush=True)
    o = T.linear_inputs((1, 150), 4, 2, 64, 40, 31, "fp32", DEV)
    got = run(ss, o)

    def loss(**change):
        a = {**o, **change}
        f = ss.linear_attn_fwd(a["q"], a["k"], a["v"], o["log_decay"], h_init=a["h_init"])
        return float((f["y"].double() * o["dy"]).sum() + (f["h_final"].double() * o["dh_final"]).sum()), \
            float((f["y"].double() * o["dy"]).abs().sum() + (f["h_final"].double() * o["dh_final"]).abs().sum())
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h_init", "dh_init")):
        d = T.make(o[name].shape, 77, "fp32", DEV)
        up, m1 = loss(**{name: o[name] + d})
        down, m2 = loss(**{name: o[name] - d})
        want = float((got[grad].double() * d).sum())
        # rounding of o +- d (1 e of each value) and of the two sums' terms
        tol = 2.0 ** -24 * (64 + 64 + 150) * (m1 + m2) + 2.0 ** -24 * 300 * float((got[grad].double() * d).abs().sum())
        assert abs((up - down) / 2 - want) <= tol, (name, up, down, want, tol)


def test_equal_calls_give_equal_bits(ss, parts_of):
    print("case: linear attention equal bits", flush=True)
    parts_of(64)
    cu = [0, 100, 100, 513, 700]
    o = T.linear_inputs((700,), 8, 2, 128, 128, 41, "bf16", DEV, rows=4)
    first = run(ss, o, cu)
    for _ in range(3):
        again = run(ss, o, cu)
        assert all(torch.equal(again[n], first[n]) for n in first)


def test_sequences_keep_to_themselves(ss):
    """A sequence of NaN and infinities leaves its neighbours' bits alone."""
    print("case: linear attention NaN neighbours", flush=True)
    cu = [0, 70, 140, 220]
    o = T.linear_inputs((220,), 2, 2, 64, 64, 51, "bf16", DEV, rows=3)
    clean = run(ss, o, cu)
    for bad in (float("nan"), float("inf")):
        p = {n: t.clone() for n, t in o.items()}
        for n in ("q", "k", "v", "dy"):
            p[n][70:140] = bad
        p["h_init"][1] = bad
        got = run(ss, p, cu)
        for n in ("y", "dq", "dk", "dv"):
            assert torch.equal(got[n][:70], clean[n][:70]) and torch.equal(got[n][140:], clean[n][140:]), n
        for n in ("h_final", "dh_init"):
            assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][2], clean[n][2]), n


def test_steps_of_no_sequence_are_left(ss):
    print("case: linear attention rest of the row", flush=True)
    o = T.linear_inputs((200,), 2, 2, 64, 64, 61, "bf16", DEV, rows=2)
    cu = torch.tensor([0, 30, 130], device=DEV)
    out = {"y": torch.full((200, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)}
    ss.linear_attn_fwd(o["q"], o["k"], o["v"], o["log_decay"], cu_seqlens=cu, h_init=o["h_init"], out=out)
    assert (out["y"][130:] == 7).all()
    used = {**{n: o[n][:130].contiguous() for n in ("q", "k", "v")}, "log_decay": o["log_decay"], "h_init": o["h_init"]}
    T.check_linear({"y": out["y"][:130]}, used, 0.125, "bf16", "rest", [0, 30, 130])


def test_bad_sequence_borders_stay_in_bounds(ss, parts_of):
    """cu_seqlens that break the rules: unspecified values, but nothing is
    written outside the outputs."""
    print("case: linear attention bad borders", flush=True)
    parts_of(64)
    L, H, D = 500, 2, 64
    o = T.linear_inputs((L,), H, H, D, D, 71, "bf16", DEV, rows=4)
    for cu in ([0, 300, 200, 400, 500], [5, 10, 20, 30, 499], [-7, 100, 900, 901, 10 ** 12], [0, 0, 0, 0, 0],
               [-5, -4, -3, -2, -1], [600, 600, 600, 600, 600], [0, 500, 0, 500, 0]):
        guard = {k: torch.full((L + 64, H, D), 7.0, dtype=torch.bfloat16, device=DEV) for k in ("y", "dq", "dk", "dv")}
        st = {k: torch.full((4 + 8, H, D, D), 7.0, device=DEV) for k in ("h_final", "dh_init")}
        c = torch.tensor(cu, dtype=torch.int64, device=DEV)
        ss.linear_attn_fwd(o["q"], o["k"], o["v"], o["log_decay"], cu_seqlens=c, h_init=o["h_init"],
                           out={"y": guard["y"][32:32 + L], "h_final": st["h_final"][4:8]})
        ss.linear_attn_bwd(o["q"], o["k"], o["v"], o["log_decay"], o["dy"], cu_seqlens=c, h_init=o["h_init"],
                           dh_final=o["dh_final"], out={**{k: guard[k][32:32 + L] for k in ("dq", "dk", "dv")},
                                                        "dh_init": st["dh_init"][4:8]})
        torch.cuda.synchronize()
        for k, t in guard.items():
            assert (t[:32] == 7).all() and (t[32 + L:] == 7).all(), k
        for k, t in st.items():
            assert (t[:4] == 7).all() and (t[8:] == 7).all(), k


def test_long_memory(ss):
    """A weak decay over many chunks: the states keep their accuracy."""
    print("case: linear attention long memory", flush=True)
    o = T.linear_inputs((1, 6000), 1, 1, 8, 8, 81, "fp32", DEV, decay=-1e-5)
    T.check_linear(run(ss, o), o, 8 ** -0.5, "fp32", "long")


def test_many_short_sequences(ss):
    print("case: linear attention many sequences", flush=True)
    n = 3000
    cu = [0]
    for i in range(n):
        cu.append(cu[-1] + i % 4)
    o = T.linear_inputs((cu[-1],), 2, 1, 16, 8, 91, "bf16", DEV, rows=n)
    T.check_linear(run(ss, o, cu), o, 0.25, "bf16", "many", cu)


def test_graph_replays_match_eager(ss, parts_of):
    print("case: linear attention graph", flush=True)
    parts_of(64)
    cu = torch.tensor([0, 100, 100, 250, 400], device=DEV)
    o = T.linear_inputs((400,), 4, 2, 64, 64, 101, "bf16", DEV, rows=4)
    args = (o["q"], o["k"], o["v"], o["log_decay"])

    def both(out):
        f = ss.linear_attn_fwd(*args, cu_seqlens=cu, h_init=o["h_init"], out={n: out[n] for n in ("y", "h_final")})
        ss.linear_attn_bwd(*args, o["dy"], cu_seqlens=cu, h_init=o["h_init"], dh_final=o["dh_final"],
                           out={n: out[n] for n in ("dq", "dk", "dv", "dh_init")})
        return f
    want = run(ss, o, [0, 100, 100, 250, 400])
    out = {n: torch.zeros_like(t) for n, t in want.items()}
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        both(out)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both(out)
    for _ in range(4):
        for t in out.values():
            t.zero_()
        eager = run(ss, o, [0, 100, 100, 250, 400])
        g.replay()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], want[n]) and torch.equal(eager[n], want[n]), n


def test_two_streams(ss, parts_of):
    print("case: linear attention streams", flush=True)
    parts_of(64)
    cases = []
    for k, dims in enumerate(((128, 128), (64, 64))):
        o = T.linear_inputs((2, 600), 4, 4, *dims, 111 + k, "bf16", DEV)
        cases.append((o, run(ss, o), torch.cuda.Stream()))
    for _ in range(3):
        torch.cuda.synchronize()
        outs = []
        for o, _, s in cases:
            with torch.cuda.stream(s):
                outs.append([ss.linear_attn_bwd(o["q"], o["k"], o["v"], o["log_decay"], o["dy"], h_init=o["h_init"],
                                                dh_final=o["dh_final"]) for _ in range(3)])
        torch.cuda.synchronize()
        for (_, want, _), got in zip(cases, outs):
            for one in got:
                assert all(torch.equal(t, want[n]) for n, t in one.items())


@pytest.mark.slow
def test_offsets_past_32_bits(ss):
    """More than 2^31 values a tensor: the last steps and heads against a call
    of their own, resumed from a state."""
    print("case: linear attention 2^31 values", flush=True)
    B, L, H, D = 3, 100000, 60, 128
    assert B * L * H * D > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, dy = (torch.randn(B, L, H, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(4))
    a = T.slopes(H, DEV)
    f = ss.linear_attn_fwd(q, k, v, a)
    b = ss.linear_attn_bwd(q, k, v, a, dy)
    cut, heads = L - 300, [0, H - 1]
    pick = lambda t, s: t[B - 1:, s][:, :, heads].contiguous()
    tail = slice(cut, L)
    h0 = ss.linear_attn_fwd(*(pick(t, slice(0, cut)) for t in (q, k, v)), a[heads])["h_final"]
    o = {"q": pick(q, tail), "k": pick(k, tail), "v": pick(v, tail), "log_decay": a[heads], "h_init": h0,
         "dy": pick(dy, tail), "dh_final": None}
    got = {"y": pick(f["y"], tail), "h_final": f["h_final"][B - 1:][:, heads]}
    got.update({n: pick(b[n], tail) for n in ("dq", "dk", "dv")})
    ref, err = T.linear_reference(o, D ** -0.5, None, "bf16")
    for n, t in got.items():
        # h0 is itself off by the bound of a state that old
        slack = 1e-4 * abs(ref[n]).max()
        T.check(t, ref[n], (err[n] + T.E32 * abs(ref[n]) if n == "h_final" else T.stored(ref[n], err[n], "bf16")) + slack, n)
