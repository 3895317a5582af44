"""Rounding of the norm and rotation on the GPU, with inputs for which all but the
step under test is exact."""
import numpy as np
import pytest
import torch

import _attn as T
from test_gpu_qkrope import DEV, ss  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
E = T.E32


@pytest.mark.parametrize("rows", [2048, 4096, 65536])
@pytest.mark.parametrize("D", [128, 512, 1024])
def test_sums_of_weight_gradients(ss, rows, D):
    """Rows of ones have a norm of 1 exactly, so that dweight is the sum of dy down
    the rows.  Blocks sum a few rows each, and their sums are joined pair by pair:
    adds whose partial sums make up 1, 1/2 + 1/2, 1/4 + ... of the whole are off by
    up to e = 2^-24 of theirs, evenly spread, so the whole is off by
    sqrt(1/3 (1 + 1/2 + 1/4 + ...)) e = 0.82 e, rms.  (What blocks add averages out
    over more than a thousand of them.)  One after another, 128 would be off by
    sqrt(128 / 9) e = 3.8 e at worst and 2.9 e with values of one size."""
    print(f"case: qk norm rope sums {rows} {D}", flush=True)
    x = torch.ones(rows, 1, D, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(rows + D)
    dq, dk = (2.0 * torch.randint(2 ** 18, 2 ** 19, (rows, 1, D), generator=g, device=DEV) + 1 for _ in range(2))
    got = ss.qk_norm_rope_bwd(x, x, dq, dk, eps=0.0)
    for n, d in (("dq_weight", dq), ("dk_weight", dk)):
        want = d.double().sum((0, 1))
        off = ((got[n].double() - want) / want).cpu().numpy() / E
        rms = np.sqrt((off ** 2).mean())
        # (128 columns: their rms is within a fifth of the expected one)
        assert rms <= 1.0 and abs(off).max() <= 7, (n, rms, abs(off).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("freq", [1.0, 0.73, 1e-2, 3.7e-5])
def test_cosines_and_sines_are_rounded_once(ss, freq, interleaved):
    """A head of (2, 0, 0, 0) has a norm of 1 and is turned into (2 cos, 2 sin, 0, 0).
    Position times frequency is exact in 64 bits (21 + 24 bits), its part of a turn off
    by 2^-53 of at most 2^18 turns, 2^-32 of an angle; the rest is one rounding."""
    print(f"case: qk norm rope cosines {freq} {interleaved}", flush=True)
    rows = 65536
    x = torch.zeros(rows, 1, 4, device=DEV)
    x[:, 0, 0] = 2
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(-(2 ** 20), 2 ** 20, (rows,), generator=g)
    f = torch.tensor([freq])
    got = ss.qk_norm_rope_fwd(x, x, pos.to(DEV), f.to(DEV), interleaved=interleaved, eps=0.0)
    angle = pos.numpy().astype(np.longdouble) * f.numpy().astype(np.longdouble)[0]
    for n in ("q", "k"):
        y = got[n][:, 0].cpu().numpy()
        assert (y[:, 2:] == 0).all()
        for i, want in enumerate((np.cos(angle), np.sin(angle))):
            half = np.spacing(abs(2 * want).astype(np.float32)) / 2.0
            off = abs(y[:, i].astype(np.longdouble) - 2 * want) - 2.0 ** -31
            worst = (off / half).max()
            # (a value just below a power of two may be rounded up to it: half a step of the upper side)
            assert worst <= 1 + 2.0 ** -4, (n, i, worst)
