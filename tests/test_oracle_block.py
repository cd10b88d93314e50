"""Pins of the block oracle (oracle.block): closed forms, library functions, and packing invariants."""

import numpy as np
import torch

from oracle import block as OB
from oracle import ssm as OS


def _rng(seed):
    return np.random.default_rng(seed)


def test_activations_match_torch():
    v = np.linspace(-120, 120, 481)
    t = torch.from_numpy(v)
    assert np.allclose(OB.silu(v), torch.nn.functional.silu(t).numpy(), rtol=1e-13, atol=1e-300)
    assert np.allclose(OB.sigmoid(v), torch.sigmoid(t).numpy(), rtol=1e-13, atol=1e-300)


def test_conv_matches_torch_conv1d():
    g = _rng(0)
    for K in (2, 3, 4):
        x, w, b = g.normal(size=(19, 8)), g.normal(size=(8, K)), g.normal(size=8)
        y, _ = OB.causal_conv(x, w, b, [0, 19], act="linear")
        ref = torch.nn.functional.conv1d(torch.from_numpy(np.concatenate([np.zeros((K - 1, 8)), x]).T[None]),
                                         torch.from_numpy(w[:, None]), torch.from_numpy(b), groups=8)[0].T.numpy()
        assert np.allclose(y, ref, rtol=1e-12, atol=1e-12)


def test_conv_and_scan_in_pieces_equal_the_whole():
    """A sequence in three calls, each continuing from the state the one before left, is the sequence in one."""
    g = _rng(1)
    T, D, N, K = 23, 8, 16, 4
    x, dt, z = g.normal(size=(T, D)), g.normal(size=(T, D)), g.normal(size=(T, D))
    B, C = g.normal(size=(T, N)), g.normal(size=(T, N))
    A, w = -np.exp(g.normal(size=(D, N))), g.normal(size=(D, K))
    whole, wst = OB.selective_scan(x, dt, None, A, B, C, [0, T], z=z, state=np.ones((2, N, D)), slots=[1])
    cwhole, cwst = OB.causal_conv(x, w, None, [0, T], state=np.ones((2, K - 1, D)), slots=[1])
    st, cst = np.ones((2, N, D)), np.ones((2, K - 1, D))
    for a, b, cont in ((0, 2, 0), (2, 3, 1), (3, T, 1)):
        sl = slice(a, b)
        y, st = OB.selective_scan(x[sl], dt[sl], None, A, B[sl], C[sl], [0, b - a], z=z[sl], state=st, slots=[1], cont=[cont])
        cy, cst = OB.causal_conv(x[sl], w, None, [0, b - a], state=cst, slots=[1], cont=[cont])
        assert np.allclose(y, whole[sl], rtol=1e-12) and np.allclose(cy, cwhole[sl], rtol=1e-12)
    assert np.allclose(st, wst) and np.allclose(cst, cwst) and np.all(st[0] == 1.0) and np.all(cst[0] == 1.0)


def test_packing_keeps_sequences_apart_and_the_tail_out():
    g = _rng(2)
    T, D, N = 12, 8, 16
    x, dt, B, C = g.normal(size=(T, D)), g.normal(size=(T, D)), g.normal(size=(T, N)), g.normal(size=(T, N))
    A = -np.exp(g.normal(size=(D, N)))
    cu = [0, 5, 5, 11]
    y, st = OB.selective_scan(x, dt, None, A, B, C, cu, state=np.full((3, N, D), 7.0), slots=[2, 0, -1])
    one, h = OS.selective_scan(x[:5], dt[:5], np.zeros(D), A, B[:5], C[:5], np.arange(5) == 0)
    assert np.allclose(y[:5], one) and np.isnan(y[11]).all()
    assert np.allclose(st[2], h.T)
    assert np.all(st[0] == 0.0) and np.all(st[1] == 7.0)      # an empty sequence that starts anew; an unused row


def test_norm_matches_torch_rms_norm_and_composes():
    g = _rng(3)
    v, w = g.normal(size=(5, 16)), g.normal(size=16)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(v), (16,), torch.from_numpy(w), 1e-5).numpy()
    assert np.allclose(OB.norm(v, w, 1e-5), ref, rtol=1e-12)
    gate, res = g.normal(size=(5, 16)), g.normal(size=(5, 16))
    r, h = OB.block_norm(v, res, w_post=w, w_pre=w, gate=gate, gate_first=True, scale=2 * w, alpha=0.5)
    assert np.allclose(r, res + 0.5 * 2 * w * OB.norm(v * OB.silu(gate), w, 1e-5)) and np.allclose(h, OB.norm(r, w, 1e-5))
    r, h = OB.block_norm(v, res, w_post=w, gate=gate, act="linear")
    assert np.allclose(r, res + OB.norm(v, w, 1e-5) * gate) and h is None
