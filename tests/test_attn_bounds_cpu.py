"""The bounds of linear attention's precision tests tell the arithmetic they are for
from coarser ones (CPU)."""
import numpy as np
import pytest
import torch

import _attn_memory as M


@pytest.mark.parametrize("chunk", [64, 32])
def test_long_memory_needs_factors_that_make_up(chunk):
    a = M.decays(chunk)
    value, mean = M.bounds(chunk)
    got = M.worst(M.faded(a, chunk, True))
    assert got[0] <= value and got[1] <= mean, (got, value, mean)
    got = M.worst(M.faded(a, chunk, False))
    assert got[0] > 5 * value and got[1] > 5 * mean, (got, value, mean)


def test_a_factor_off_by_little_is_seen():
    """2^-22 at every chunk."""
    value, mean = M.bounds(64)
    ratio = M.faded(M.decays(64), 64, True) * (1 + 2.0 ** -22) ** (M.STEPS // 64)
    assert M.worst(ratio)[1] > 5 * mean


def test_two_terms_of_a_weighted_step_are_seen():
    """Bound of a part's sum of single steps (3 |n a| + 9 units of 2^-24): three bf16 terms of
    the weighted value are inside, two are not, cut off or rounded."""
    v = np.random.default_rng(2).standard_normal((64, 64)).astype(np.float32)
    v = torch.from_numpy(v).to(torch.bfloat16).double().numpy()
    for a in (-0.001, -0.005, -0.02):
        back = np.arange(63, -1, -1) * float(np.float32(a))
        w = (np.exp(back)[:, None] * v).astype(np.float32)
        bound = (3 * 64 * abs(a) + 9) * M.E
        for cut in (True, False):
            rest, total, off = w.copy(), np.zeros(w.shape), []
            for _ in range(3):
                if cut:
                    term = (rest.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
                else:
                    term = torch.from_numpy(rest).to(torch.bfloat16).float().numpy()
                total, rest = total + term, rest - term
                off.append(abs(total / (np.exp(back)[:, None] * v) - 1).max())
            assert off[2] <= bound / 4 and off[1] > 1.5 * bound, (a, cut, off, bound)
