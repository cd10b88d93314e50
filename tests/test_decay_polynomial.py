"""The polynomial of the scan's decays on the FMA pipe: its coefficients, as they stand in the source, hold the error that its
comment states (no GPU needed)."""

import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ssm_compressed_chunked_b200", "csrc",
                      "selective_scan.cu")


def coefficients():
    found = re.findall(r"\bkE([1-5]) = ([0-9.e-]+)f\b", open(SOURCE).read())
    assert [k for k, _ in found] == ["1", "2", "3", "4", "5"]
    return [np.float32(v) for _, v in found]


def stated():
    """The two errors of the comment: of the polynomial, and with its sums rounded."""
    m = re.search(r"relative error ([0-9.e-]+) with the coefficients rounded to fp32, ([0-9.e-]+) once the sums are rounded",
                  open(SOURCE).read())
    assert m, "the comment states both errors"
    return float(m.group(1)), float(m.group(2))


def test_polynomial_error():
    k = [float(c) for c in coefficients()]
    f = np.linspace(-0.5, 0.5, 2000001)
    p = np.ones_like(f)
    acc = np.zeros_like(f)
    for c in reversed(k):
        acc = acc * f + c
    err = np.abs((p + f * acc) / np.exp2(f) - 1.0).max()
    assert 0.9 * stated()[0] < err <= stated()[0], err


def test_polynomial_error_with_rounded_sums():
    """Each step an fma in fp32: a product and sum in fp64 (exact to 2^-53), rounded once to fp32."""
    f = np.linspace(-0.5, 0.5, 2000001).astype(np.float32)
    k = coefficients()
    q = np.full(f.shape, k[4], dtype=np.float32)
    for c in (k[3], k[2], k[1], k[0], np.float32(1.0)):
        q = (q.astype(np.float64) * f.astype(np.float64) + np.float64(c)).astype(np.float32)
    r = q.astype(np.float64) / np.exp2(f.astype(np.float64)) - 1.0
    assert 0.9 * stated()[1] < np.abs(r).max() <= stated()[1], np.abs(r).max()
    # near 0, where a decay is close to 1 and thousands of them multiply, the error has no bias of its own
    near = np.abs(f) < 2.0 ** -8
    assert abs(r[near].mean()) < 2.0 ** -26, r[near].mean()
