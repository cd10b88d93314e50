"""Inputs and error bounds of the SSM block's operators (test plumbing).

Error bounds, from the kernels' arithmetic (u = 2^-24, half a step of fp32):
* a stored output rounds by at most half a step of its type: finfo.eps / 2 of the value
  (bf16 2^-8, fp32 2^-24);
* ex2.approx is off by at most 2^-22 of the value, and by the rounding of its argument:
  |argument| u in the exponent;
* silu / sigmoid: that, an add and an approximate quotient (2 steps): 2^-20 + 2^-23 |z| of the value;
* softplus: 3e-6 of the value (its comment), plus 2^-22 and 2^-23 |z| through e^z;
* sums of n terms: n u of the sum of magnitudes.
The scan's bound follows the recurrence: an error in h decays with h and each token adds the errors of
its decay, its input and its rounding."""

import numpy as np
import torch

from helpers import f64
from oracle import block as OB
from oracle import ssm as OS

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# a bf16 cancellation to near zero still stores a value whose half step is tiny; the arithmetic terms cover it
TINY = 1e-30


def act_bound(name, v):
    """Relative error of act(v) computed in fp32."""
    return np.zeros_like(v) if name == "linear" else 2.0 ** -20 + 2.0 ** -23 * np.abs(v)


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def wide(rows, cols, dtype, gen, extra=0, scale=1.0):
    """[rows, cols] normal values; with ``extra`` a column window of a wider array (row stride cols + 2 extra)."""
    t = (torch.randn(rows, cols + 2 * extra, generator=gen) * scale).to(dtype)
    return t[:, extra:extra + cols]


def to_gpu(t):
    """A copy on the GPU with the same row stride (a window stays a window)."""
    if t is None:
        return None
    if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) != t.shape[1]:
        base = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype, device="cuda")
        off = t.storage_offset() % t.stride(0)
        base[:, off:off + t.shape[1]] = t.cuda()
        return base[:, off:off + t.shape[1]]
    return t.cuda()


def scan_inputs(T, D, N, dtype, seed, gate=True, skip=True, bias=True, extra=0):
    g = torch.Generator().manual_seed(seed)
    d = dict(x=wide(T, D, dtype, g, extra), dt=wide(T, D, dtype, g, extra), B=wide(T, N, dtype, g, extra),
             C=wide(T, N, dtype, g, extra), z=wide(T, D, dtype, g, extra) if gate else None,
             A=-torch.exp(torch.rand(D, N, generator=g) * np.log(16.0)),
             skip=torch.randn(D, generator=g) if skip else None, bias=None)
    if bias:
        d0 = torch.exp(torch.rand(D, generator=g) * np.log(100.0) + np.log(1e-3))
        d["bias"] = d0 + torch.log(-torch.expm1(-d0))
    return d


def scan_bound(d, cu, out_dtype, state=None, slots=None, cont=None):
    """Bounds (y [T, D], state) on the scan's error, from the oracle's own values."""
    x, dt, B, C, A = (f64(d[k]) for k in ("x", "dt", "B", "C", "A"))
    T, D = x.shape
    N = A.shape[1]
    bias = np.zeros(D) if d["bias"] is None else f64(d["bias"])
    zin = dt + bias
    delta = OS.softplus(zin)
    r_delta = 3e-6 + 2.0 ** -22 + 2.0 ** -23 * np.abs(zin)
    by = np.zeros((T, D))
    bst = None if state is None else np.zeros_like(f64(state))
    for s in range(len(cu) - 1):
        slot = -1 if state is None else (s if slots is None else int(slots[s]))
        h = np.zeros((D, N))
        if slot >= 0 and cont is not None and cont[s]:
            h = f64(state)[slot].T.copy()
        err = np.zeros((D, N))
        for t in range(cu[s], cu[s + 1]):
            e = np.abs(delta[t][:, None] * A)
            a = np.exp(-e)
            u = np.abs(delta[t] * x[t])[:, None] * np.abs(B[t])[None]
            err = a * err + a * np.abs(h) * (2.0 ** -22 + e * (r_delta[t][:, None] + 4 * U)) \
                + u * (r_delta[t][:, None] + 3 * U)
            h = np.exp(-e) * h + (delta[t] * x[t])[:, None] * B[t][None]
            err = err + 2 * U * np.abs(h) + U * u
            mag = np.abs(h) @ np.abs(C[t])
            sk = 0.0 if d["skip"] is None else np.abs(f64(d["skip"]) * x[t])
            v = h @ C[t] + (0.0 if d["skip"] is None else f64(d["skip"]) * x[t])
            b = err @ np.abs(C[t]) + (N + 6) * U * (mag + sk)
            if d["z"] is not None:
                z = f64(d["z"])[t]
                g = np.abs(OB.silu(z))
                b = b * g + np.abs(v) * g * (act_bound("silu", z) + U)
                v = v * OB.silu(z)
            by[t] = b + HALF[out_dtype] * (np.abs(v) + b) + TINY
        if slot >= 0:
            bst[slot] = err.T + TINY
    return by, bst


def assert_within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err - bound)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; at {k} got {got[k]!r}, ref {ref[k]!r}, "
                             f"err {err[k]:.3e} > bound {bound[k]:.3e}")
