"""The functions behind SiLU and GELU, evaluated in fp32 on the host from the
source's own coefficients, against their 64-bit forms, with the reciprocal and
the exponential off by one ulp each, either way: the bounds that the source
states."""
import os
import re

import numpy as np
import pytest
from scipy.special import ndtr

from combine_fp32_router_amd import build

f32 = np.float32


def source(name):
    with open(os.path.join(build.CSRC, "expert_rows.hpp")) as f:
        s = f.read()
    s = s[s.index("float " + name):]
    return s[:s.index("\n}\n")]


def fma(a, b, c):
    """Rounded once (but for double rounding, 2^-29 of a step)."""
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(f32)


def off_by(v, ulp):
    return v if ulp == 0 else np.nextafter(v, f32(ulp * np.inf))


@pytest.mark.parametrize("rcp", [-1, 0, 1])
@pytest.mark.parametrize("exp", [-1, 0, 1])
def test_sigmoid(rcp, exp):
    z = np.concatenate([np.linspace(-80, 80, 400001), np.linspace(-1, 1, 200001)]).astype(f32)
    log2e = f32(re.search(r"exp2f\(z \* (-[\d.]+)f\)", source("sigmoid"))[1])
    e = off_by(np.exp2(np.float64(z * log2e)).astype(f32), exp)
    s = off_by((1.0 / np.float64(f32(1) + e)).astype(f32), rcp)
    want = 1 / (1 + np.exp(-np.float64(z)))
    assert (np.abs(s - want) <= (1.25 * np.abs(z) + 5) * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("rcp", [-1, 0, 1])
@pytest.mark.parametrize("exp", [-1, 0, 1])
def test_normal_below(rcp, exp):
    text = source("normal_below")
    coeffs = re.findall(r"p = (?:fmaf\(p, t, )?(-?[\d.]+)f\)?;", text)
    assert len(coeffs) == 10
    third, gauss = re.search(r"fabsf\(z\), ([\d.]+)f, 1.0f", text), re.search(r"z \* z, (-[\d.]+)f, p", text)
    z = np.concatenate([np.linspace(-5.6, 5.6, 400001), np.linspace(-0.2, 0.2, 200001), np.linspace(-38, 38, 20001)]).astype(f32)
    t = off_by((1.0 / np.float64(fma(np.abs(z), f32(third[1]), f32(1)))).astype(f32), rcp)
    p = np.full_like(z, f32(coeffs[0]))
    for c in coeffs[1:]:
        p = fma(p, t, f32(c))
    q = t * off_by(np.exp2(np.float64(fma(z * z, f32(gauss[1]), p))).astype(f32), exp)
    want = ndtr(-np.abs(np.float64(z)))
    near = np.abs(z) < 5.6
    assert (np.abs(q - want)[near] <= 2e-6 * want[near]).all()
    assert (np.abs(np.where(z < 0, q, f32(1) - q) - ndtr(np.float64(z))) <= 3.5e-7).all()
