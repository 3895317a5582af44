"""Norm and rotation of queries and keys on the GPU against the fp64
definition, within derived bounds; and the layer of norm and rotation, linear
attention and norm per head that they make up."""
import pytest
import torch

from oracle import attention as A
from oracle import layers as O
import _attn as T
import _layers as TL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ss():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_18_amd import ssmscan
    ssmscan.lib()
    return ssmscan


def run(ss, o, eps=1e-6, interleaved=False, affine=True):
    kw = dict(interleaved=interleaved, eps=eps)
    if affine:
        kw.update(q_weight=o["q_weight"], k_weight=o["k_weight"])
    f = o["freqs"] if len(o["freqs"]) else None
    got = ss.qk_norm_rope_fwd(o["q"], o["k"], o["positions"], f, **kw)
    got.update(ss.qk_norm_rope_bwd(o["q"], o["k"], o["dq"], o["dk"], o["positions"], f, **kw))
    torch.cuda.synchronize()
    return got


# rows, Hq, Hk, D, R
SHAPES = [(1, 1, 1, 1, 0), (1, 1, 1, 2, 2), (3, 2, 1, 7, 4), (2, 3, 3, 16, 16), (5, 4, 2, 32, 32), (3, 2, 2, 64, 64),
          (4, 8, 8, 64, 32), (7, 3, 1, 80, 80), (2, 5, 5, 96, 72), (9, 40, 8, 128, 128), (6, 2, 1, 128, 64),
          (3, 4, 4, 112, 96), (2, 2, 2, 160, 160), (3, 7, 1, 192, 128), (2, 6, 2, 256, 256), (2, 3, 1, 250, 250),
          (1, 2, 2, 512, 512), (2, 1, 1, 520, 24), (1, 1, 2, 1024, 1024), (2, 1, 1, 1000, 998), (1, 1, 1, 1023, 512),
          (300, 4, 1, 64, 64), (1500, 1, 1, 128, 128), (5, 33, 3, 128, 0), (4, 2, 0, 64, 64), (4, 0, 2, 64, 64),
          (33, 2, 2, 129, 34), (17, 2, 2, 130, 18)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(ss, shape, dtype, interleaved):
    print(f"case: qk norm rope {shape} {dtype} {interleaved}", flush=True)
    o = T.rope_inputs(*shape, sum(shape), dtype, DEV)
    T.check_rope(run(ss, o, interleaved=interleaved), o, dtype, "rope", interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_weights_and_with_eps(ss, dtype):
    print(f"case: qk norm rope plain {dtype}", flush=True)
    o = T.rope_inputs(6, 4, 2, 64, 64, 3, dtype, DEV)
    T.check_rope(run(ss, o, eps=0.5, affine=False), o, dtype, "plain", eps=0.5, affine=False)
    o["q"].zero_()
    o["k"][2] = 0
    T.check_rope(run(ss, o), o, dtype, "zeros")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [1, 2, 3, 4, 6])
def test_unaligned_tensors(ss, offset, dtype):
    print(f"case: qk norm rope offset {offset} {dtype}", flush=True)
    for inter in (False, True):
        o = T.rope_inputs(5, 4, 2, 128, 128, offset, dtype, DEV, offset=offset)
        T.check_rope(run(ss, o, interleaved=inter), o, dtype, "unaligned", interleaved=inter)


def test_far_positions(ss):
    """Positions of 2^40: the angle still has 64 bits."""
    print("case: qk norm rope far positions", flush=True)
    o = T.rope_inputs(9, 2, 2, 64, 64, 5, "fp32", DEV, far=1 << 40)
    # 2^40 positions of frequency 1 are 2^37.3 turns: a product of 53 bits is
    # off by 2^-16 turns, 10^-4 radians
    kw = dict(q_weight=o["q_weight"], k_weight=o["k_weight"])
    got = ss.qk_norm_rope_fwd(o["q"], o["k"], o["positions"], o["freqs"], **kw)
    for m in ("q", "k"):
        x, w = T.f64(o[m]), T.f64(o[m + "_weight"])
        ref = A.norm_rope(x, o["positions"].cpu().numpy(), T.f64(o["freqs"]), w, 1e-6, False)
        z, _, er = T._rope_terms(x, 1e-6)
        mag = T._pair_magnitude(z * abs(w), 64, False)
        T.check(got[m], ref, T.stored(ref, (er + 20 * T.E32 + 3 * 2.0 ** -53 * 2.0 ** 40) * mag, "fp32"), m)


def test_outputs_may_replace_inputs(ss):
    print("case: qk norm rope in place", flush=True)
    for dims in ((128, 128), (192, 64), (250, 250), (1023, 512)):
        for inter in (False, True):
            o = T.rope_inputs(37, 4, 2, *dims, 7, "bf16", DEV)
            kw = dict(q_weight=o["q_weight"], k_weight=o["k_weight"], interleaved=inter)
            want = ss.qk_norm_rope_fwd(o["q"], o["k"], o["positions"], o["freqs"], **kw)
            q, k = o["q"].clone(), o["k"].clone()
            ss.qk_norm_rope_fwd(q, k, o["positions"], o["freqs"], out={"q": q, "k": k}, **kw)
            assert torch.equal(q, want["q"]) and torch.equal(k, want["k"])


def test_heads_keep_to_themselves(ss):
    print("case: qk norm rope NaN neighbours", flush=True)
    o = T.rope_inputs(6, 4, 2, 64, 64, 9, "bf16", DEV)
    clean = run(ss, o)
    o["q"][2, 1, 5] = float("nan")
    o["dq"][4, 3, 7] = float("inf")
    got = run(ss, o)
    touched = torch.zeros(6, 4, dtype=torch.bool, device=DEV)
    touched[2, 1] = True
    assert torch.equal(got["q"][~touched], clean["q"][~touched]) and torch.equal(got["k"], clean["k"])
    touched[4, 3] = True
    assert torch.equal(got["dq"][~touched], clean["dq"][~touched]) and torch.equal(got["dk"], clean["dk"])
    assert torch.equal(got["dk_weight"], clean["dk_weight"])


def test_no_rows_and_no_weight_gradients(ss):
    print("case: qk norm rope empty", flush=True)
    o = T.rope_inputs(0, 4, 2, 64, 64, 9, "bf16", DEV)
    got = run(ss, o)
    assert got["q"].shape == (0, 4, 64) and (got["dq_weight"] == 0).all() and (got["dk_weight"] == 0).all()
    o = T.rope_inputs(5, 4, 2, 64, 64, 9, "bf16", DEV)
    want = run(ss, o, affine=False)
    got = ss.qk_norm_rope_bwd(o["q"], o["k"], o["dq"], o["dk"], o["positions"], o["freqs"], want_params=False)
    assert set(got) == {"dq", "dk"} and all(torch.equal(got[n], want[n]) for n in got)


def test_gradients_against_differences(ss):
    """fp32, central differences along random directions.  With f the weighted
    sum and a step of s, the truncation is s^2 / 6 times the third derivative;
    at s = 2^-6 two steps' difference bounds it, and the rounding of the sums
    is 2^-24 of the sum of their terms' magnitudes over the step."""
    print("case: qk norm rope differences", flush=True)
    o = T.rope_inputs(40, 3, 2, 96, 72, 13, "fp32", DEV)
    got = run(ss, o)

    def loss(name, d, s):
        a = {**o, name: o[name] + s * d}
        f = ss.qk_norm_rope_fwd(a["q"], a["k"], o["positions"], o["freqs"], q_weight=a["q_weight"],
                                k_weight=a["k_weight"])
        t = torch.cat([(f["q"].double() * o["dq"]).flatten(), (f["k"].double() * o["dk"]).flatten()])
        return float(t.sum()), float(t.abs().sum())
    for name in ("q", "k", "q_weight", "k_weight"):
        d = T.make(o[name].shape, 17, "fp32", DEV)
        slope, noise = [], 0.0
        for s in (2.0 ** -6, 2.0 ** -7):
            (up, mu), (dn, md) = loss(name, d, s), loss(name, d, -s)
            slope.append((up - dn) / (2 * s))
            noise = max(noise, 32 * T.E32 * (mu + md) / (2 * s))
        want = float((got["d" + name].double() * d).sum())
        best = (4 * slope[1] - slope[0]) / 3  # without the s^2 term
        assert abs(best - want) <= 2 * noise + abs(slope[1] - slope[0]) / 3, (name, slope, want, noise)


def test_equal_calls_give_equal_bits_and_graph_replays(ss):
    print("case: qk norm rope graph", flush=True)
    o = T.rope_inputs(700, 8, 2, 128, 128, 15, "bf16", DEV)
    want = run(ss, o)
    kw = dict(q_weight=o["q_weight"], k_weight=o["k_weight"])
    out = {n: torch.zeros_like(t) for n, t in want.items()}

    def both():
        ss.qk_norm_rope_fwd(o["q"], o["k"], o["positions"], o["freqs"], out={n: out[n] for n in ("q", "k")}, **kw)
        ss.qk_norm_rope_bwd(o["q"], o["k"], o["dq"], o["dk"], o["positions"], o["freqs"],
                            out={n: out[n] for n in ("dq", "dk", "dq_weight", "dk_weight")}, **kw)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both()
    for _ in range(4):
        for t in out.values():
            t.zero_()
        eager = run(ss, o)
        g.replay()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], want[n]) and torch.equal(eager[n], want[n]), n


def test_layer_of_rotation_attention_and_head_norm(ss):
    """The operators as a layer runs them: norm and rotation of q and k, linear
    attention, norm per head; then their backward calls in reverse order, against
    the fp64 chain on the same stored intermediate values; and the prompt's last
    steps once more as single tokens."""
    print("case: retention layer", flush=True)
    B, L, H, Hkv, D = 2, 150, 4, 2, 64
    o = T.rope_inputs(B * L, H, Hkv, D, D, 19, "bf16", DEV)
    q, k = o["q"].view(B, L, H, D), o["k"].view(B, L, Hkv, D)
    v, dout = T.make((B, L, Hkv, D), 21, "bf16", DEV), T.make((B, L, H, D), 22, "bf16", DEV)
    pos = torch.arange(L, device=DEV).expand(B, L).contiguous()
    a = T.slopes(H, DEV)
    w, b = torch.randn(H * D, device=DEV), torch.randn(H * D, device=DEV)
    kw = dict(q_weight=o["q_weight"], k_weight=o["k_weight"])
    r = ss.qk_norm_rope_fwd(q, k, pos, o["freqs"], **kw)
    f = ss.linear_attn_fwd(r["q"], r["k"], v, a)
    y2 = f["y"].view(B, L, H * D)
    n = ss.layer_norm_fwd(y2, w, b, group=D, want_stats=True)
    gn = ss.layer_norm_bwd(y2, w, n["mean"], n["rstd"], dout.view(B, L, H * D), group=D)
    dy = gn["dx"].view(B, L, H, D)
    ga = ss.linear_attn_bwd(r["q"], r["k"], v, a, dy)
    gr = ss.qk_norm_rope_bwd(q, k, ga["dq"], ga["dk"], pos, o["freqs"], **kw)
    torch.cuda.synchronize()
    flat = lambda t: t.reshape(B * L, *t.shape[2:])
    ro = {**o, "positions": flat(pos), "dq": flat(ga["dq"]), "dk": flat(ga["dk"])}
    T.check_rope({"q": flat(r["q"]), "k": flat(r["k"]), "dq": flat(gr["dq"]), "dk": flat(gr["dk"]),
                  "dq_weight": gr["dq_weight"], "dk_weight": gr["dk_weight"]}, ro, "bf16", "layer")
    lo = {"q": r["q"], "k": r["k"], "v": v, "log_decay": a, "h_init": None, "dy": dy, "dh_final": None}
    T.check_linear({**f, **ga}, lo, D ** -0.5, "bf16", "layer")
    s = TL.f64(y2).reshape(B * L, -1)
    ry, rm, rr = O.layer_norm(s, TL.f64(w), TL.f64(b), D)
    ey, _, _ = TL.norm_bounds(s, rm, rr, TL.f64(w), TL.f64(b), D, 1e-5)
    TL.check(n["y"].reshape(B * L, -1), ry, TL.stored(ry, ey, "bf16"), "norm y")
    # the last ten steps one by one from the state before them
    cut = L - 10
    part = lambda t: t[:, :cut].contiguous()
    h = ss.linear_attn_fwd(part(r["q"]), part(r["k"]), part(v), a)["h_final"]
    ys = []
    for t in range(cut, L):
        rt = ss.qk_norm_rope_fwd(q[:, t].contiguous(), k[:, t].contiguous(), pos[:, t].contiguous(), o["freqs"], **kw)
        assert torch.equal(rt["q"], r["q"][:, t]) and torch.equal(rt["k"], r["k"][:, t])
        ys.append(ss.step_linear_attn(rt["q"], rt["k"], v[:, t].contiguous(), a, h))
    ref, err = T.linear_reference({**lo, "dy": None}, D ** -0.5)
    tail = torch.stack(ys, 1)
    T.check(tail, ref["y"][:, cut:], T.stored(ref["y"], err["y"], "bf16")[:, cut:], "steps y")
    T.check(h, ref["h_final"], err["h_final"] + T.E32 * abs(ref["h_final"]) + 1e-37, "steps h")
