"""The operators of a Mamba block around the selective SSM (oracle; test infrastructure only).

Sources
-------
* pith.science review, "Assumptions & free parameters": the SSM is a selective
  state-space model (Mamba, Section 3.2, Eq. 3).

Readings taken where the pages are silent
-----------------------------------------
* The block's short convolution is causal and depthwise: y[t, d] = act(bias[d] +
  sum_{k<K} w[d, k] x[t-(K-1)+k, d]); positions ahead of a sequence come from its
  carried window (its last K-1 inputs, oldest first) or are zero.
* The SSM block adds skip[d] x[t, d] to C . h and multiplies by silu(z).
* Packed sequences: cu[s] .. cu[s+1] are the tokens of sequence s; slots[s] its state
  row (-1: none), cont[s] whether it continues from it.
* norm(v, w) = v / sqrt(mean(v^2) + eps) * w (root mean square norm).

Plain float64 numpy, one token at a time; states are returned as new arrays.
"""

import numpy as np

from .ssm import selective_scan as _scan_one


def silu(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return v * np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


ACTS = {"linear": lambda v: np.asarray(v, dtype=np.float64), "silu": silu, "sigmoid": sigmoid}


def _slot(slots, s):
    return s if slots is None else int(slots[s])


def causal_conv(x, w, bias, cu, state=None, slots=None, cont=None, act="silu"):
    """x [T, D], w [D, K], bias [D] or None, state [n_slots, K-1, D] or None.

    Returns (y [T, D] with NaN in rows no sequence owns, state afterwards)."""
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(w, dtype=np.float64)
    T, D = x.shape
    K = w.shape[1]
    y = np.full((T, D), np.nan)
    st = None if state is None else np.array(state, dtype=np.float64)
    for s in range(len(cu) - 1):
        slot = _slot(slots, s) if st is not None else -1
        line = np.zeros((K - 1, D))
        if slot >= 0 and cont is not None and cont[s]:
            line = st[slot].copy()
        for t in range(cu[s], cu[s + 1]):
            taps = np.concatenate([line, x[t:t + 1]])
            acc = np.zeros(D) if bias is None else np.asarray(bias, dtype=np.float64).copy()
            for k in range(K):
                acc = acc + w[:, k] * taps[k]
            y[t] = ACTS[act](acc)
            line = taps[1:]
        if slot >= 0:
            st[slot] = line
    return y, st


def selective_scan(x, dt, bias, A, B, C, cu, skip=None, z=None, state=None, slots=None, cont=None):
    """x, dt, z [T, D], B, C [T, N], A [D, N], state [n_slots, N, D] or None.

    Returns (y [T, D] with NaN in rows no sequence owns, state afterwards)."""
    x = np.asarray(x, dtype=np.float64)
    T, D = x.shape
    N = np.asarray(A).shape[1]
    b = np.zeros(D) if bias is None else bias
    y = np.full((T, D), np.nan)
    st = None if state is None else np.array(state, dtype=np.float64)
    for s in range(len(cu) - 1):
        a, e = int(cu[s]), int(cu[s + 1])
        slot = _slot(slots, s) if st is not None else -1
        h = np.zeros((D, N))
        if slot >= 0 and cont is not None and cont[s]:
            h = st[slot].T.copy()
        if e > a:
            v, h = _scan_one(x[a:e], dt[a:e], b, A, B[a:e], C[a:e], np.zeros(e - a, dtype=bool), h)
            if skip is not None:
                v = v + np.asarray(skip, dtype=np.float64) * x[a:e]
            if z is not None:
                v = v * silu(z[a:e])
            y[a:e] = v
        if slot >= 0:
            st[slot] = h.T
    return y, st


def norm(v, w, eps):
    v = np.asarray(v, dtype=np.float64)
    return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def block_norm(y, res, w_post=None, w_pre=None, gate=None, act="silu", gate_first=False, scale=None, alpha=1.0,
               eps=1e-5):
    """Returns (r, h): the residual sum and, with w_pre, its norm (else None)."""
    if y is None:
        r = np.asarray(res, dtype=np.float64)
    else:
        v = np.asarray(y, dtype=np.float64)
        if gate is not None and gate_first:
            v = v * ACTS[act](gate)
        if w_post is not None:
            v = norm(v, w_post, eps)
        if gate is not None and not gate_first:
            v = v * ACTS[act](gate)
        if scale is not None:
            v = v * np.asarray(scale, dtype=np.float64)
        r = alpha * v + (0.0 if res is None else np.asarray(res, dtype=np.float64))
    return r, (None if w_pre is None else norm(r, w_pre, eps))
