"""Grids that are sized by what a compute unit holds at once, against the
registers that the compiler gives those kernels.  (A CU has 4 SIMDs; the
compiler reports the waves that each of them holds.)"""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from selective_state_space_18_amd import build

SOURCES = ("norm_f32.hip", "norm_bf16.hip", "gated_f32.hip", "gated_bf16.hip")


def waves_per_cu(source):
    """{mangled kernel name: waves a CU holds by registers and LDS}"""
    r = subprocess.run([build.hipcc(), *build.COMMON, "-x", "hip", "--cuda-device-only", "-c",
                        os.path.join(build.CSRC, source), "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    held, name = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"remark:\s+(Function Name|Occupancy \[waves/SIMD\]): (\S+)", line)
        if m and m[1] == "Function Name":
            name = m[2]
        elif m:
            held[name] = 4 * int(m[2])
    return held


@pytest.fixture(scope="module")
def held():
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    with ThreadPoolExecutor(4) as ex:
        return {k: v for d in ex.map(waves_per_cu, SOURCES) for k, v in d.items()}


def header(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return f.read()


def test_norm_grids_fit_the_chip(held):
    """kNormFwdHeld and kNormBwdHeld, per vector of a lane, are no more waves
    than a CU holds of any kernel they are used for."""
    text = header("norm_kernels.h")
    fwd = int(re.search(r"kNormFwdHeld = (\d+);", text)[1])
    m = re.search(r"kNormBwdHeld = sizeof\(T\) == 4 \? (\d+) : (\d+);", text)
    most = {("fwd", "f"): fwd, ("fwd", "DF16b"): fwd, ("bwd", "f"): int(m[1]), ("bwd", "DF16b"): int(m[2])}
    seen = 0
    for kernel, waves in held.items():
        k = re.search(r"norm_(fwd|bwd)_kernelI(f|DF16b)Li\d+ELi\d+ELi(\d+)ELb[01]E", kernel)
        if k:
            seen += 1
            assert waves >= most[k[1], k[2]] // int(k[3]), (kernel, waves)
    assert seen == 2 * 2 * 6 * 2


def test_gated_backward_blocks_that_stay_fit_the_chip(held):
    """Where blocks take tile after tile, two of 8 waves are launched per CU."""
    text = header("gated_kernels.h")
    assert "held = 2 * (int64_t)q.f.cus" in text and "constexpr int kGatedWaves = 8;" in text
    seen = 0
    for kernel, waves in held.items():
        if re.search(r"gated_bwd_kernelI(f|DF16b)Li\dELb[01]ELi0ELi\dE", kernel):
            seen += 1
            assert waves // 8 == 2, (kernel, waves)
    assert seen == 2 * (1 + 3)
