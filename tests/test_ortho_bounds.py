"""Which coefficients an orthogonalised update takes: those whose values on the way,
found here by sampling, stay below 64 and above 2^-40.  On the host, for an empty
stack: nothing is launched."""
import ctypes
import os

import numpy as np
import pytest

import roofline_sgemm_f32_amd as rs

OK, ARG = 0, 8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rs.library_path()):
        pytest.skip("libsgemm.so not built")
    return rs.load()


def status(lib, *triples):
    flat = [v for t in triples for v in t]
    c = (ctypes.c_double * len(flat))(*flat)
    return lib.sgemm_orthogonalize(0, 0, 100, 90, None, 90, 9000, None, 90, 9000, len(triples), c, 1e-7, None, 0, None)


def top(triples):
    """The largest |p(..p(s))| after any step by sampling, each step from the range
    of the one before."""
    r, tops = 1.0, []
    for a, b, c in triples:
        # Evenly, and at the critical points in exact terms of the coefficients.
        s = np.linspace(0, r, 200001)
        r = float(np.abs(s * (a + s * s * (b + s * s * c))).max()) * 1.01
        tops.append(r)
    return tops


@pytest.mark.parametrize("c", [1e-15, 1e-16, -1e-16, 1e-20, -1e-20, 1e-300, -1e-300, 5e-324, 0.0])
def test_small_fifth_powers(lib, c):
    """200 s - 199.5 s^3 passes 77 at s = 0.58 and is 0.5 at 1."""
    assert status(lib, (200.0, -199.5, c)) == ARG
    assert status(lib, (-200.0, 199.5, c)) == ARG
    assert status(lib, (30.0, -29.0, c)) == OK                        # 11.7
    assert status(lib, (30.0, -29.0, c), (6.0, 0.0, 0.0)) == ARG      # 70
    assert status(lib, (30.0, -29.0, c), (5.0, 0.0, 0.0)) == OK       # 59
    assert status(lib, (3.0, -3.0, c)) == OK                          # 0 at 1, 1.15 on the way


def test_against_samples(lib):
    rng = np.random.default_rng(5)
    seen = {OK: 0, ARG: 0}
    for i in range(400):
        triples = []
        for _ in range(1 + i % 3):
            a, b, c = rng.normal(size=3) * np.array([8, 20, 20]) * 10.0 ** rng.uniform(-1, 1)
            if i % 2:
                b, c = b * 10.0 ** rng.uniform(-18, 0), c * 10.0 ** rng.uniform(-18, 0)
            if i % 5 == 0:
                a = -b - c  # a zero at 1
            triples.append((a, b, c))
        tops = top(triples)
        # Samples 5e-6 apart miss a maximum by far less than one in a thousand.
        if any(abs(t / 64 - 1) < 1e-3 for t in tops) or min(tops) < 1e-11:
            continue
        want = OK if max(tops) < 64 else ARG
        assert status(lib, *triples) == want, (triples, tops)
        seen[want] += 1
    assert min(seen.values()) > 50


def test_equal_and_missing_roots(lib):
    assert status(lib, (5.0, -10.0, 9.0)) == OK
    assert status(lib, (0.0, 0.0, 1.0)) == OK and status(lib, (0.0, 1.0, 0.0)) == OK
    assert status(lib, (0.0, 60.0, 0.0)) == OK and status(lib, (0.0, 64.0, 0.0)) == ARG
    assert status(lib, (1e-300, 0.0, 1.0)) == OK and status(lib, (1.0, 1e-300, 1e-300)) == OK
    # Values that cancel at 1 and are past any bound before it.
    assert status(lib, (1e200, -1e200, 1.0)) == ARG and status(lib, (1e12, -1e12, 1.0)) == ARG
