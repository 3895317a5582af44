"""A state of linear attention that only fades, chunk after chunk, for very long:
decays, the two ways of rounding the factors, and bounds.

Without k (or dy) every chunk multiplies the state by exp(C a), C steps to a
chunk, in fp32: h <- fl(h f).  A factor f that is always rounded the same way is
off by the same part d of e = 2^-24 every time, n d e after n chunks.  Factors
that make up for what the ones before them were off by leave the products'
roundings: n independent ones of at most e each, so that (Hoeffding) a value is
off by more than 6 sqrt(n) e with a chance of 2 exp(-18), 3e-8, and the mean over
m values by more than 6 sqrt(n / m) e with the same; 2 e covers the last factor."""
import numpy as np

E = 2.0 ** -24
STEPS = 1 << 20
HEADS, DK, DV = 8, 8, 8


def decays(chunk):
    """Log decays (fp32) of about exp(-1) over STEPS whose factor over a chunk is
    nearly half a unit from what fp32 holds, to either side."""
    a = -(0.5 + np.arange(4000) / 4000).astype(np.float32) / np.float32(STEPS)
    exact = np.exp(a.astype(np.float64) * chunk)
    off = (exact.astype(np.float32).astype(np.float64) / exact - 1) / E
    order = np.argsort(off)
    pick = np.concatenate([order[:HEADS // 2], order[-(HEADS // 2):]])
    assert (abs(off[pick]) > 0.4).all()
    return a[pick]


def bounds(chunk):
    """(of a value, of a head's mean), relative"""
    n = STEPS // chunk
    return (6 * np.sqrt(n) + 2) * E, (6 * np.sqrt(n / (DK * DV)) + 2) * E


def faded(a, chunk, compensated):
    """The state [HEADS, DV * DK] after STEPS, relative to the exact one."""
    h0 = np.random.default_rng(1).standard_normal((len(a), DV * DK)).astype(np.float32)
    exact = np.exp(a.astype(np.float64) * chunk)
    h, error = h0.copy(), np.zeros(len(a))
    for _ in range(STEPS // chunk):
        now = exact * (1 + error) if compensated else exact
        f = now.astype(np.float32)
        error = (now - f) / exact
        h *= f[:, None]
    return h / (h0 * np.exp(a.astype(np.float64) * STEPS)[:, None])


def worst(ratio):
    """(largest error of a value, largest mean error of a head), ratio [HEADS, values]."""
    off = np.asarray(ratio, dtype=np.float64) - 1
    return abs(off).max(), abs(off.mean(1)).max()
