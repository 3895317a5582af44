"""The gated linear recurrence on the GPU against its fp64 definition, within
derived bounds: forward, packed sequences, backward, decode step."""
import numpy as np
import pytest
import torch

from oracle import layers as O
import _layers as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ss():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_18_amd import ssmscan
    ssmscan.lib()
    return ssmscan


def run(ss, o, cu=None, carry=True, out=None):
    """Forward and backward; every output of both."""
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], cu_seqlens=c, h_init=o["h_init"], want_carry=carry)
    g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], cu_seqlens=c, h_init=o["h_init"],
                          dh_final=o["dh_final"], carry=f.get("carry"))
    torch.cuda.synchronize()
    return {**f, **g}


# Steps around one thread's run, one wave's, one tile and the groups of tiles;
# channels around one lane's vector, a wave and a tile.
SHAPES = [(1, 1, 1), (2, 2, 3), (1, 7, 64), (3, 8, 65), (1, 15, 2), (1, 16, 127), (2, 17, 128), (1, 63, 129),
          (2, 64, 66), (1, 65, 130), (1, 127, 254), (2, 128, 5), (1, 129, 256), (1, 255, 33), (2, 256, 62),
          (1, 300, 383), (1, 1023, 9), (2, 1025, 70), (1, 2049, 130), (1, 4500, 37), (2, 2304, 128),
          # columns enough for the link-by-link chain, and rows of whole 64-byte pieces
          (24, 450, 130), (50, 300, 63), (7, 260, 1024), (4, 2500, 160),
          # and for groups of 8 links
          (2, 1500, 1030)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(ss, shape, dtype):
    T_state = shape[1] % 2 == 1 or shape[0] > 1
    print(f"case: gated {shape} {dtype}", flush=True)
    o = T.gated_inputs(shape, 100 + sum(shape), dtype, DEV, state=T_state)
    T.check_gated(run(ss, o), o, dtype, f"{shape}")


@pytest.mark.parametrize("dtype,shape", [("bf16", (1, 40001, 66)), ("fp32", (2, 33000, 5))], ids=str)
def test_long_rows_of_few_channels(ss, shape, dtype):
    """One or two channel groups along many tiles: the chain's longer groups."""
    print(f"case: gated long {shape} {dtype}", flush=True)
    o = T.gated_inputs(shape, 17, dtype, DEV)
    T.check_gated(run(ss, o), o, dtype, f"{shape}")
    cu = [0, 1, 8192, 16385, 16385, 30000, shape[1]]
    p = {k: (t[0].contiguous() if t.dim() == 3 else t) for k, t in o.items()}
    g = torch.Generator().manual_seed(3)
    for k in ("h_init", "dh_final"):
        p[k] = torch.randn(len(cu) - 1, shape[2], generator=g).to(DEV)
    T.check_gated(run(ss, p, cu), p, dtype, "packed", cu)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 130, 66), (1, 257, 128)], ids=str)
def test_unaligned_tensors(ss, shape, dtype):
    print(f"case: gated unaligned {shape} {dtype}", flush=True)
    for offset in (1, 2, 3):
        o = T.gated_inputs(shape, 7 + offset, dtype, DEV, offset=offset)
        T.check_gated(run(ss, o), o, dtype, f"offset {offset}")


PACKED = {
    "one": (5, [0, 5]),
    "ones": (9, list(range(10))),
    "empty_ends": (130, [0, 0, 0, 64, 64, 129, 130, 130, 130]),
    "edges": (400, [0, 1, 8, 16, 17, 63, 64, 65, 127, 128, 129, 130, 256, 257, 400]),
    "long": (4700, [0, 3, 2048, 2049, 2049, 4096, 4700]),
    "whole": (2500, [0, 2500]),
    "second": (700, [0, 0, 700]),
    "many": (515, sorted([0, 515] + [(k * k * 7 + 3 * k) % 515 for k in range(200)])),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", list(PACKED))
@pytest.mark.parametrize("state", [True, False], ids=["state", "zero"])
def test_packed(ss, name, dtype, state):
    L, cu = PACKED[name]
    D = 130 if dtype == "bf16" else 67
    print(f"case: gated packed {name} {dtype} {state}", flush=True)
    o = T.gated_inputs((L, D), 11 + L, dtype, DEV, rows=len(cu) - 1, state=state)
    T.check_gated(run(ss, o, cu), o, dtype, name, cu)


# Packed rows wide enough for the link-by-link chain (the last in lone bf16
# channels), for groups of 8 links, and long ones of one or two columns.
@pytest.mark.parametrize("L, D, dtype", [(450, 6100, "bf16"), (450, 3100, "fp32"), (300, 3101, "bf16"),
                                         (1500, 2100, "bf16"), (1500, 1030, "fp32"), (1500, 2101, "bf16"),
                                         (33000, 66, "bf16"), (33000, 66, "fp32")])
def test_packed_wide_and_long(ss, L, D, dtype):
    print(f"case: gated packed {L} {D} {dtype}", flush=True)
    cu = [0, 0, 1, 7, 64, 130, 131, L - 120, L - 120, L - 64, L - 1, L, L]
    o = T.gated_inputs((L, D), 31 + L, dtype, DEV, rows=len(cu) - 1)
    T.check_gated(run(ss, o, cu), o, dtype, f"{L} {D}", cu)


def test_packed_with_very_many_empty_sequences(ss):
    """70000 sequences, all but a few without steps, against the same call
    without the empty ones."""
    print("case: gated many empty", flush=True)
    L, D, n = 300, 5, 70000
    o = T.gated_inputs((L, D), 77, "bf16", DEV, rows=n)
    ends = [(9, 5), (10, 6), (40000, 131), (65535, 132), (65536, 200), (69999, 300)]  # (sequence, its end)
    cu = torch.zeros(n + 1, dtype=torch.int64)
    for k, t in ends:
        cu[k + 1:] = t
    rows = torch.tensor([k for k, _ in ends], device=DEV)
    got = run(ss, o, cu.tolist())
    few = {**o, "h_init": o["h_init"][rows].contiguous(), "dh_final": o["dh_final"][rows].contiguous()}
    want = run(ss, few, [0] + [t for _, t in ends])
    for name, t in want.items():
        assert torch.equal(got[name][rows] if name in ("h_final", "dh_init") else got[name], t), name
    empty = torch.ones(n, dtype=torch.bool, device=DEV)
    empty[rows] = False
    assert torch.equal(got["h_final"][empty], o["h_init"][empty])
    assert torch.equal(got["dh_init"][empty], o["dh_final"][empty])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_and_dense_rows_agree(ss, dtype):
    """The same rows run densely and packed.  Where a sequence starts the
    packed form rounds a h_init + b once, the dense form carries h_init
    through the products of the decays: equal up to the derived bounds."""
    print(f"case: gated packed rows {dtype}", flush=True)
    o = T.gated_inputs((3, 256, 70), 5, dtype, DEV)
    ref, err = T.gated_reference(o)
    d = run(ss, o)
    p = {k: (t.reshape(768, 70) if t.dim() == 3 else t) for k, t in o.items()}
    q = run(ss, p, [0, 256, 512, 768])
    for k in ("y", "dx", "dr", "di"):
        b = T.stored(ref[k], err[k], dtype)
        T.check(d[k], ref[k], b, k)
        T.check(q[k].reshape(3, 256, 70), ref[k], b, k)
    for k in ("h_final", "dh_init", "dA"):
        T.check(q[k], ref[k], err[k] + T.E32 * np.abs(ref[k]), k)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_without_the_carry(ss, dtype):
    print(f"case: gated no carry {dtype}", flush=True)
    for shape, cu in (((2, 700, 66), None), ((700, 66), [0, 90, 90, 401, 700])):
        rows = None if cu is None else len(cu) - 1
        o = T.gated_inputs(shape, 21, dtype, DEV, rows=rows)
        a, b = run(ss, o, cu), run(ss, o, cu, carry=False)
        for k in ("dx", "dr", "di", "dA", "dh_init"):
            assert torch.equal(a[k], b[k]), k


def test_optional_outputs_and_buffers(ss):
    print("case: gated optional outputs", flush=True)
    o = T.gated_inputs((2, 333, 66), 22, "bf16", DEV)
    a = run(ss, o)
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=o["h_init"], want_state=False)
    assert set(f) == {"y"} and torch.equal(f["y"], a["y"])
    # the final state may replace the initial one
    h = o["h_init"].clone()
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=h, out={"h_final": h})
    assert torch.equal(h, a["h_final"]) and torch.equal(f["y"], a["y"])
    g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], h_init=o["h_init"], dh_final=o["dh_final"],
                          carry=a["carry"], want_dh_init=False)
    assert "dh_init" not in g and torch.equal(g["dA"], a["dA"])
    with pytest.raises(ValueError):
        ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], out={"z": h})
    with pytest.raises(ValueError):
        ss.scan_gated_fwd(o["x"].transpose(1, 2), o["r"], o["i"], o["A"])
    with pytest.raises(TypeError):
        ss.scan_gated_fwd(o["x"], o["r"].float(), o["i"], o["A"])
    with pytest.raises(TypeError):
        ss.scan_gated_fwd(o["x"].half(), o["r"].half(), o["i"].half(), o["A"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(64, 200, 130), (3, 1500, 66), (1, 40000, 40), (24, 700, 520)], ids=str)
def test_final_state_in_the_initial_states_place(ss, shape, dtype):
    """Every tile has read h_init before any tile writes h_final over it."""
    print(f"case: gated in place {shape} {dtype}", flush=True)
    o = T.gated_inputs(shape, 23, dtype, DEV, grads=False)
    want = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=o["h_init"])
    for _ in range(10):
        h = o["h_init"].clone()
        f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=h, out={"h_final": h})
        assert f["h_final"] is h and torch.equal(h, want["h_final"]) and torch.equal(f["y"], want["y"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zero_steps(ss, dtype):
    print(f"case: gated empty {dtype}", flush=True)
    o = T.gated_inputs((2, 0, 5), 1, dtype, DEV)
    a = run(ss, o)
    assert torch.equal(a["h_final"], o["h_init"]) and torch.equal(a["dh_init"], o["dh_final"])
    assert not a["dA"].any()
    o["h_init"] = o["dh_final"] = None
    a = run(ss, o)
    assert not a["h_final"].any() and not a["dh_init"].any()
    o = T.gated_inputs((0, 5), 1, dtype, DEV, rows=3)
    a = run(ss, o, [0, 0, 0, 0])
    assert torch.equal(a["h_final"], o["h_init"]) and torch.equal(a["dh_init"], o["dh_final"])
    assert not a["dA"].any()


def test_outputs_keep_to_their_rows(ss):
    """Memory on both sides of every output keeps its values, packed with
    empty sequences at the end, at channels and steps that end inside a tile."""
    print("case: gated canaries", flush=True)
    L, D, cu = 201, 67, [0, 50, 50, 201, 201]
    o = T.gated_inputs((L, D), 31, "bf16", DEV, rows=4)
    bufs = {}

    def guarded(name, shape, dt):
        n = int(np.prod(shape))
        b = torch.full((n + 512,), 7.0, dtype=dt, device=DEV)
        bufs[name] = (b, n)
        return b[256:256 + n].view(shape)

    c = torch.tensor(cu, device=DEV)
    tiles = -(-L // ss.gated_carry_steps())
    fo = {"y": guarded("y", (L, D), torch.bfloat16), "h_final": guarded("h_final", (4, D), torch.float32),
          "carry": guarded("carry", (1, tiles, D), torch.float32)}
    f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], cu_seqlens=c, h_init=o["h_init"], want_carry=True, out=fo)
    go = {k: guarded(k, (L, D), torch.bfloat16) for k in ("dx", "dr", "di")}
    go["dA"] = guarded("dA", (D,), torch.float32)
    go["dh_init"] = guarded("dh_init", (4, D), torch.float32)
    g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], cu_seqlens=c, h_init=o["h_init"],
                          dh_final=o["dh_final"], carry=f["carry"], out=go)
    torch.cuda.synchronize()
    for name, (b, n) in bufs.items():
        assert (b[:256] == 7).all() and (b[256 + n:] == 7).all(), name
    T.check_gated({**f, **g}, o, "bf16", "guarded", cu)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_degenerate_gates(ss, dtype):
    """A = 0 and gates at their limits: everything stays finite, the state is
    kept where a = 1, and dr, dx vanish there."""
    print(f"case: gated degenerate {dtype}", flush=True)
    o = T.gated_inputs((2, 200, 66), 41, dtype, DEV, A=0.0)
    a = run(ss, o)
    T.check_gated(a, o, dtype, "A = 0")
    assert torch.equal(a["h_final"], o["h_init"]) and not a["dr"].any() and not a["dx"].any()
    o = T.gated_inputs((2, 200, 66), 42, dtype, DEV)
    o["r"][:, 50:60] = -200.0  # closed
    o["r"][:, 60:70] = 200.0   # open
    o["i"][:, 90:95] = -200.0
    o["i"][:, 95:99] = 200.0
    o["r"][:, 120] = float("-inf")
    o["r"][:, 121] = float("inf")
    o["i"][:, 122] = float("-inf")
    o["i"][:, 123] = float("inf")
    a = run(ss, o)
    for k, t in a.items():
        assert torch.isfinite(t).all(), k
    # the bounds grow with |r|: compare against gates clamped to +-100, whose
    # sigmoid differs by less than 4e-44, so m by less than sqrt(2 |A| 4e-44)
    # = 8e-22 and a value it multiplies (below 1e3 here) by less than 1e-18
    n = dict(o, r=o["r"].clamp(-100, 100), i=o["i"].clamp(-100, 100))
    T.check_gated(a, n, dtype, "limits", floor=1e-18)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_stay_in_their_sequence(ss, bad):
    print(f"case: gated non-finite {bad}", flush=True)
    L, D, cu = 900, 66, [0, 100, 300, 301, 550, 900]
    o = T.gated_inputs((L, D), 51, "bf16", DEV, rows=5)
    clean = run(ss, o, cu)
    p = dict(o, x=o["x"].clone(), dy=o["dy"].clone())
    p["x"][250, 3] = bad    # sequence 1
    p["x"][600, 5] = bad    # sequence 4
    p["dy"][560, 7] = bad   # sequence 4
    p["dy"][120, 9] = bad   # sequence 1
    got = run(ss, p, cu)
    rows = torch.zeros(L, dtype=torch.bool, device=DEV)
    rows[0:100] = rows[300:550] = True  # sequences 0, 2, 3
    for k in ("y", "dx", "dr", "di"):
        assert torch.equal(got[k][rows], clean[k][rows]), k
    for k in ("h_final", "dh_init"):
        for s in (0, 2, 3):
            assert torch.equal(got[k][s], clean[k][s]), (k, s)
    assert not torch.isfinite(got["y"][299, 3]) and not torch.isfinite(got["y"][899, 5])
    assert torch.equal(got["y"][:250], clean["y"][:250])  # before it in time
    cols = [c for c in range(D) if c not in (3, 5, 7, 9)]
    for k in ("y", "dx", "dr", "di", "dA"):
        assert torch.equal(got[k][..., cols], clean[k][..., cols]), k


def test_gradients_against_differences_of_the_forward(ss):
    """fp32: directional derivatives of a loss of the library's own forward."""
    print("case: gated differences", flush=True)
    o = T.gated_inputs((2, 150, 34), 61, "fp32", DEV)
    # away from A = 0, where the input scale has no finite curvature
    o["A"].clamp_(max=-0.3)
    g = run(ss, o)

    def loss(k):
        f = ss.scan_gated_fwd(k["x"], k["r"], k["i"], k["A"], h_init=k["h_init"])
        return float((f["y"].double() * o["dy"].double()).sum() +
                     (f["h_final"].double() * o["dh_final"].double()).sum())

    gen = torch.Generator().manual_seed(5)
    # each y is off by a few e |y|: with n values of order 1 added at random
    # the loss by about 10 e sqrt(n), and a difference over a step of 2 h by
    # that / (2 h); the third-order term is h^2 times a sum of order sqrt(n)
    h, n = 3e-3, o["x"].numel()
    tol = 10 * T.E32 * n ** 0.5 / (2 * h) * 4 + 10 * h * h * n ** 0.5
    for name, arg in (("dx", "x"), ("dr", "r"), ("di", "i"), ("dA", "A"), ("dh_init", "h_init")):
        v = torch.randn(o[arg].shape, generator=gen).to(DEV)
        up, down = dict(o), dict(o)
        up[arg], down[arg] = o[arg] + h * v, o[arg] - h * v
        step = (up[arg].double() - down[arg].double())  # as rounded
        slope = (loss(up) - loss(down))
        want = float((g[name].double() * step).sum())
        assert abs(slope - want) <= 2 * h * tol, (name, slope / (2 * h), want / (2 * h), tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 3), (4, 64), (3, 65), (7, 777), (256, 130), (5, 2050)], ids=str)
def test_step(ss, shape, dtype):
    print(f"case: gated step {shape} {dtype}", flush=True)
    for offset in (0, 1):
        o = T.gated_inputs((1, *shape), 71 + offset, dtype, DEV, rows=shape[0], offset=offset, grads=False)
        t = {k: o[k].view(shape) for k in ("x", "r", "i")}
        n = {k: T.f64(t[k]).reshape(1, -1) for k in t}
        w = T._row(n["x"], n["r"], n["i"], np.tile(T.f64(o["A"]), shape[0]), T.f64(o["h_init"]).reshape(-1))
        ref, err = w["h"].reshape(shape), w["Eh"].reshape(shape)
        h = o["h_init"].clone()
        h_out = torch.empty_like(h)
        y = ss.step_gated(t["x"], t["r"], t["i"], o["A"], h, h_out=h_out)
        assert torch.equal(h, o["h_init"])
        T.check(h_out, ref, err + 1e-37, "h_out")
        T.check(y, ref, T.stored(ref, err, dtype), "y")
        y2 = ss.step_gated(t["x"], t["r"], t["i"], o["A"], h)
        assert torch.equal(h, h_out) and torch.equal(y, y2)
        # one step of the scan is a decode step
        f = ss.scan_gated_fwd(*(t[k].reshape(shape[0], 1, shape[1]) for k in ("x", "r", "i")), o["A"],
                              h_init=o["h_init"])
        T.check(f["h_final"], ref, err + 1e-37, "scan")


def test_decode_continues_a_prefill(ss):
    """Prefill 300 steps, then 40 decode steps: the scan over all 340."""
    print("case: gated prefill then decode", flush=True)
    o = T.gated_inputs((3, 340, 70), 81, "bf16", DEV, grads=False)
    ref, err = T.gated_reference(o)
    cut = {k: o[k][:, :300].contiguous() for k in ("x", "r", "i")}
    f = ss.scan_gated_fwd(cut["x"], cut["r"], cut["i"], o["A"], h_init=o["h_init"])
    h, ys = f["h_final"], [f["y"]]
    for t in range(300, 340):
        ys.append(ss.step_gated(*(o[k][:, t].contiguous() for k in ("x", "r", "i")), o["A"], h)[:, None])
    y = torch.cat(ys, 1)
    T.check(y, ref["y"], T.stored(ref["y"], err["y"], "bf16"), "y")
    T.check(h, ref["h_final"], err["h_final"] + 1e-37, "h")


def test_replays_match_eager(ss):
    print("case: gated graph replay", flush=True)
    o = T.gated_inputs((2, 3000, 130), 91, "bf16", DEV)
    e = run(ss, o)
    s = torch.cuda.Stream()
    bufs = {k: torch.empty_like(t) for k, t in e.items()}
    fo = {k: bufs[k] for k in ("y", "h_final", "carry")}
    go = {k: bufs[k] for k in ("dx", "dr", "di", "dA", "dh_init")}

    def both():
        ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=o["h_init"], want_carry=True, out=fo)
        ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], h_init=o["h_init"], dh_final=o["dh_final"],
                          carry=bufs["carry"], out=go)

    with torch.cuda.stream(s):
        both()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for k in range(4):
        for t in bufs.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, t in bufs.items():
            assert torch.equal(t, e[name]), (k, name)
        # other work of the same stream's scratch between replays
        with torch.cuda.stream(s):
            ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], h_init=o["h_init"], dh_final=o["dh_final"])
        s.synchronize()


def test_two_streams(ss):
    print("case: gated two streams", flush=True)
    a = T.gated_inputs((2, 3000, 200), 92, "bf16", DEV)
    b = T.gated_inputs((1, 5000, 130), 93, "fp32", DEV)
    ea, eb = run(ss, a), run(ss, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        outs = []
        for s, o in ((s1, a), (s2, b)):
            with torch.cuda.stream(s):
                f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], h_init=o["h_init"], want_carry=True)
                g = ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], h_init=o["h_init"],
                                      dh_final=o["dh_final"], carry=f["carry"])
                outs.append({**f, **g})
        torch.cuda.synchronize()
        for got, want in zip(outs, (ea, eb)):
            for k in want:
                assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
def test_tiles_shared_by_several_calls(ss, packed):
    """Calls with more tiles than the chip holds blocks, on three streams at
    once: blocks of each start late, when other blocks may have taken every
    tile of their call."""
    print("case: gated tiles shared", flush=True)
    cases = []
    for k, (B, L, D) in enumerate([(1, 700, 6400), (1, 4500, 6400), (1, 750, 6272)]):
        o = T.gated_inputs((L, D) if packed else (B, L, D), 95 + k, "bf16", DEV, rows=3 if packed else None)
        cu = [0, 3, L - 9, L] if packed else None
        e = run(ss, o, cu)
        cases.append((o, None if cu is None else torch.tensor(cu, device=DEV), e, torch.cuda.Stream()))
    for _ in range(3):
        torch.cuda.synchronize()
        outs = []
        for o, cu, e, s in cases:
            with torch.cuda.stream(s):
                outs.append([ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], cu_seqlens=cu,
                                               h_init=o["h_init"], dh_final=o["dh_final"], carry=e["carry"])
                             for _ in range(4)])
        torch.cuda.synchronize()
        for (_, _, e, _), got in zip(cases, outs):
            for one in got:
                for name, t in one.items():
                    assert torch.equal(t, e[name]), name


def test_bad_sequence_borders_stay_in_bounds(ss):
    """cu_seqlens that break the rules: unspecified values, but nothing is
    written outside the outputs and finite inputs are only read in bounds."""
    print("case: gated bad borders", flush=True)
    L, D = 500, 66
    o = T.gated_inputs((L, D), 94, "bf16", DEV, rows=4)
    for cu in ([0, 300, 200, 400, 500], [5, 10, 20, 30, 499], [-7, 100, 900, 901, 10 ** 12], [0, 0, 0, 0, 0],
               [-5, -4, -3, -2, -1], [600, 600, 600, 600, 600]):
        guard = {k: torch.full((L + 64, D), 7.0, dtype=torch.bfloat16, device=DEV) for k in ("y", "dx", "dr", "di")}
        st = {k: torch.full((4 + 8, D), 7.0, device=DEV) for k in ("h_final", "dh_init")}
        c = torch.tensor(cu, dtype=torch.int64, device=DEV)
        f = ss.scan_gated_fwd(o["x"], o["r"], o["i"], o["A"], cu_seqlens=c, h_init=o["h_init"], want_carry=True,
                              out={"y": guard["y"][32:32 + L], "h_final": st["h_final"][4:8]})
        ss.scan_gated_bwd(o["x"], o["r"], o["i"], o["A"], o["dy"], cu_seqlens=c, h_init=o["h_init"],
                          dh_final=o["dh_final"], carry=f["carry"],
                          out={**{k: guard[k][32:32 + L] for k in ("dx", "dr", "di")}, "dh_init": st["dh_init"][4:8]})
        torch.cuda.synchronize()
        for k, t in guard.items():
            assert (t[:32] == 7).all() and (t[32 + L:] == 7).all(), k
        for k, t in st.items():
            assert (t[:4] == 7).all() and (t[8:] == 7).all(), k


@pytest.mark.slow
def test_more_than_2_31_values(ss):
    """Offsets past 32 bits: the last batch rows against their own small call
    (forward and backward) and the fp64 definition on sampled channels."""
    print("case: gated 2^31 values", flush=True)
    B, L, D = 260, 2048, 4224
    assert B * L * D > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r, i, dy = (torch.randn(B, L, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(4))
    A = -torch.rand(D, generator=g, device=DEV)
    f = ss.scan_gated_fwd(x, r, i, A, want_carry=True)
    b = ss.scan_gated_bwd(x, r, i, A, dy, carry=f["carry"])
    cols = [0, 63, 64, 127, 128, 2111, D - 1]
    for row in (0, 255, B - 1):
        pick = lambda t: t[row:row + 1, :, cols].contiguous()
        o = {"x": pick(x), "r": pick(r), "i": pick(i), "A": A[cols], "h_init": None, "dy": pick(dy), "dh_final": None}
        got = {"y": pick(f["y"]), "h_final": f["h_final"][row:row + 1, cols]}
        got.update({k: pick(b[k]) for k in ("dx", "dr", "di")}, dh_init=b["dh_init"][row:row + 1, cols])
        T.check_gated(got, o, "bf16", f"row {row}")


def test_layer_of_norm_recurrence_and_head_norm(ss):
    """The operators as a layer runs them: residual norm, gated recurrence,
    norm per head; then their backward calls in the reverse order, against
    the fp64 chain on the same stored intermediate values."""
    print("case: gated layer", flush=True)
    B, L, D, P = 2, 260, 128, 64
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    x, res, r, i, dout, dres = (rnd(B, L, D) for _ in range(6))
    A = -torch.rand(D, generator=g).to(DEV)
    w1, b1, w2, b2 = (torch.randn(D, generator=g).to(DEV) for _ in range(4))
    n1 = ss.layer_norm_fwd(x, w1, b1, residual=res, want_stats=True)
    f = ss.scan_gated_fwd(n1["y"], r, i, A, want_carry=True)
    n2 = ss.layer_norm_fwd(f["y"], w2, b2, group=P, want_stats=True)
    g2 = ss.layer_norm_bwd(f["y"], w2, n2["mean"], n2["rstd"], dout, group=P)
    gs = ss.scan_gated_bwd(n1["y"], r, i, A, g2["dx"], carry=f["carry"])
    g1 = ss.layer_norm_bwd(n1["sum"], w1, n1["mean"], n1["rstd"], gs["dx"], dsum=dres)
    torch.cuda.synchronize()
    o = {"x": n1["y"], "r": r, "i": i, "A": A, "h_init": None, "dy": g2["dx"], "dh_final": None}
    T.check_gated({**f, **gs}, o, "bf16", "recurrence")
    flat = lambda t: T.f64(t).reshape(B * L, -1)
    for s, n, w, b, group, y in ((n1["sum"], n1, w1, b1, None, n1["y"]), (f["y"], n2, w2, b2, P, n2["y"])):
        ry, rm, rr = O.layer_norm(flat(s), T.f64(w), T.f64(b), group)
        ey, _, _ = T.norm_bounds(flat(s), rm, rr, T.f64(w), T.f64(b), group, 1e-5)
        T.check(y.reshape(B * L, D), ry, T.stored(ry, ey, "bf16"), "norm y")
    for s, n, w, group, dy, dsum, got in ((f["y"], n2, w2, P, dout, None, g2), (n1["sum"], n1, w1, None, gs["dx"], dres, g1)):
        a = (flat(s), flat(n["mean"]), flat(n["rstd"]), T.f64(w))
        ds = None if dsum is None else flat(dsum)
        ref = O.layer_norm_bwd(a[0], a[3], a[1], a[2], flat(dy), ds, group)
        ex, ew, eb = T.norm_bwd_bounds(a[0], a[1], a[2], a[3], flat(dy), ds, group)
        T.check(got["dx"].reshape(B * L, D), ref["dx"], T.stored(ref["dx"], ex, "bf16"), "norm dx")
        T.check(got["dweight"], ref["dweight"], ew, "dweight")
        T.check(got["dbias"], ref["dbias"], eb, "dbias")
