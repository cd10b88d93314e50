"""The SSM block's operators run together, as a model runs them: layer.SsmMixer stage by stage against the oracle
(each stage fed the GPU's own inputs to it, so a stage wired to the wrong buffer fails), prompts in pieces and decoding
against the whole prompt, and layer.Block around both mixers."""

import math

import numpy as np
import pytest
import torch

from block_cases import HALF, TINY, U, assert_within, offsets, scan_bound
from helpers import Guarded, assert_bf16_close, assert_written, f64
from oracle import block as OB
from oracle import projection as OP
from ssm_compressed_chunked_b200 import attamba as A
from ssm_compressed_chunked_b200 import layer
from ssm_compressed_chunked_b200 import workloads as W
from test_gpu_ssm_block import conv_bound, i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def mixer_weights(D, Di, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, f=1.0: torch.randn(*s, generator=g) * f  # noqa: E731
    d0 = torch.exp(torch.rand(Di, generator=g) * np.log(100.0) + np.log(1e-3))
    return dict(W_in=n(2 * Di, D, f=D ** -0.5).to(BF), W_x=n(Di + 2 * N, Di, f=Di ** -0.5).to(BF),
                W_O=n(D, Di, f=Di ** -0.5).to(BF), conv_w=n(Di, K, f=K ** -0.5), conv_b=n(Di, f=0.1),
                A=-torch.exp(torch.rand(Di, N, generator=g) * np.log(16.0)), bias=d0 + torch.log(-torch.expm1(-d0)),
                skip=n(Di))


def gemm_check(Y, X, Wm, what):
    ref = OP.project(f64(X), f64(Wm))
    mag = np.abs(f64(X)) @ np.abs(f64(Wm)).T
    assert_within(f64(Y), ref, HALF[BF] * np.abs(ref) + X.shape[1] * U * mag + 1e-6, what)


def cuda(w):
    return {k: v.cuda() for k, v in w.items()}


@pytest.mark.parametrize("D,Di,N,K,lens,pad", [(128, 256, 16, 4, [70, 0, 200, 31], 0), (64, 128, 32, 3, [9], 0),
                                               (64, 192, 16, 2, [300, 150], 5)])
def test_mixer_stages_match_oracle(D, Di, N, K, lens, pad):
    w = mixer_weights(D, Di, N, K, seed=Di)
    T, S = sum(lens) + pad, len(lens)
    guard = Guarded()
    mix = layer.SsmMixer(D, Di, N, K, cuda(w), T + 10, alloc=guard)
    cu, slots = offsets(lens), list(range(S, 0, -1))
    cont = [s % 2 for s in range(S)]
    win, ssm = mix.new_state(S + 1)
    g = torch.Generator().manual_seed(1)
    win.copy_(torch.randn(win.shape, generator=g))
    ssm.copy_(torch.randn(ssm.shape, generator=g))
    win0, ssm0 = win.cpu().clone(), ssm.cpu().clone()
    h = torch.randn(T, D, generator=g).to(BF)
    y = mix.forward(h.cuda(), A.Seqs(i32(cu), T, slots=i32(slots), cont=i32(cont)), state=(win, ssm))
    torch.cuda.synchronize()
    guard.check()
    assert mix.status.item() == 0
    n = sum(lens)
    b = {k: v[:n].cpu() for k, v in mix.buf.items()}
    gemm_check(b["x"], h[:n], w["W_in"][:Di], "x")
    gemm_check(b["z"], h[:n], w["W_in"][Di:], "z")
    args = (f64(b["x"]), f64(w["conv_w"]), f64(w["conv_b"]), cu, f64(win0), slots, cont)
    pre, _ = OB.causal_conv(*args, act="linear")
    ref, ref_win = OB.causal_conv(*args)
    assert_within(f64(b["u"]), ref, conv_bound(b["x"], w["conv_w"], w["conv_b"], pre, ref, cu, BF, "silu", win0, slots, cont), "u")
    assert np.array_equal(f64(win), ref_win)
    for name, rows in (("dt", slice(0, Di)), ("B", slice(Di, Di + N)), ("C", slice(Di + N, Di + 2 * N))):
        gemm_check(b[name], b["u"], w["W_x"][rows], name)
    d = dict(x=b["u"], dt=b["dt"], B=b["B"], C=b["C"], z=b["z"], A=w["A"], bias=w["bias"], skip=w["skip"])
    ref, ref_ssm = OB.selective_scan(f64(b["u"]), f64(b["dt"]), f64(w["bias"]), f64(w["A"]), f64(b["B"]), f64(b["C"]), cu,
                                     f64(w["skip"]), f64(b["z"]), f64(ssm0), slots, cont)
    by, bst = scan_bound(d, cu, BF, ssm0, slots, cont)
    assert_within(f64(b["s"]), ref, by, "s")
    assert_within(f64(ssm)[slots], ref_ssm[slots], bst[slots], "ssm state")
    gemm_check(y[:n].cpu(), b["s"], w["W_O"], "y")


def test_mixer_in_pieces_and_token_by_token():
    """A batch of prompts in one call; the same prompts in two calls; and their last tokens decoded one at a time from
    the carried states, in a batch padded with a row of no sequence: the same rows out.  The bound: bf16's half
    step of every stage on the way, through the stages behind it (2^-8 of values of order 1, some of them summed)."""
    D, Di, N, K = 128, 256, 16, 4
    w = cuda(mixer_weights(D, Di, N, K, seed=9))
    lens = [90, 41, 130]
    T, S = sum(lens), len(lens)
    g = torch.Generator().manual_seed(3)
    h = torch.randn(T, D, generator=g).to(BF).cuda()
    mix = layer.SsmMixer(D, Di, N, K, w, T)
    whole_state = mix.new_state(S)
    whole = mix.forward(h, A.Seqs(i32(offsets(lens)), T), state=whole_state).clone()
    cu, keep = offsets(lens), 6
    first = [n - keep for n in lens]
    rows = lambda a, b: torch.cat([h[cu[s] + a[s]:cu[s] + b[s]] for s in range(S)])  # noqa: E731
    half = [n // 2 for n in first]
    state = mix.new_state(S)
    out = {s: [] for s in range(S)}
    for a, b, cont in (([0] * S, half, 0), (half, first, 1)):
        part = [b[s] - a[s] for s in range(S)]
        x = rows(a, b)
        y = mix.forward(x, A.Seqs(i32(offsets(part)), len(x), cont=i32([cont] * S)), state=state)
        for s in range(S):
            o = offsets(part)
            out[s].append(y[o[s]:o[s + 1]].clone())
    slots = i32([2, -1, 0, 1])
    for k in range(keep):
        x = torch.zeros(4, D, dtype=BF, device="cuda")
        for row, s in ((0, 2), (2, 0), (3, 1)):
            x[row] = h[cu[s] + first[s] + k]
        y = mix.decode_step(state, x, slots=slots)
        for row, s in ((0, 2), (2, 0), (3, 1)):
            out[s].append(y[row:row + 1].clone())
    assert mix.status.item() == 0
    for s in range(S):
        assert_bf16_close(f64(torch.cat(out[s])), f64(whole[cu[s]:cu[s + 1]]), f"sequence {s}", rel=2.0 ** -6)
    assert torch.allclose(state[1], whole_state[1], rtol=2e-2, atol=2e-2)
    assert torch.allclose(state[0].float(), whole_state[0].float(), rtol=2e-2, atol=2e-2)


@pytest.mark.parametrize("res", [torch.float32, BF])
def test_blocks_around_the_layer_and_the_mixer(res):
    """A block around the Attamba layer, then one around the SSM mixer, the norms joined; against the operators called one
    by one and the oracle's norms of the GPU's own values; a second pass with the norms apart gives the same rows."""
    B, n, H, N, dh = 2, 96, 2, 16, 64
    D = H * dh
    cfg = W.shrink(W.BF16_TEST_P8_L64, B=B, n=n, D=D, H=H)
    inp = W.make_layer(cfg)
    g = torch.Generator().manual_seed(5)
    shapes = {"W_Q": (D, D), "W_dtK": (D, D), "W_dtV": (D, D), "W_BK": (N, D), "W_CK": (N, D), "W_BV": (N, D),
              "W_CV": (N, D), "W_O": (D, D)}
    lw = {k: (torch.randn(*s, generator=g) / math.sqrt(D)).to(BF).cuda() for k, s in shapes.items()}
    lw.update({k: inp[k].cuda() for k in ("bias_k", "bias_v", "A_k", "A_v")})
    lay = layer.Layer(B, n, D, H, dh, N, lw, cfg.P, cfg.offset, cfg.L, A.MASK_TEST, inp["scale"])
    mix = layer.SsmMixer(D, 2 * D, N, 4, cuda(mixer_weights(D, 2 * D, N, 4, 6)), B * n)
    n1, n2, n3, post, scale = (torch.rand(D, generator=g).cuda() + 0.5 for _ in range(5))
    one = layer.Block(lay, n1, w_post=post, alpha=0.5)
    two = layer.Block(mix, n2, scale=scale)
    seqs = A.Seqs(i32([0, n, 2 * n]), 2 * n)
    r0 = torch.randn(B * n, D, generator=g).to(res).cuda()
    r = r0.clone()
    r, h = one.forward(r, next_norm=n2)
    r1, h2 = r.clone(), h.clone()
    r, h = two.forward(r, seqs, h=h, next_norm=n3)
    r2, h3 = r.clone(), h.clone()
    # the same apart: every norm on its own
    q = r0.clone()
    q, none = one.forward(q)
    assert none is None and torch.equal(q, r1)
    ya = lay.y.clone()
    q, none = two.forward(q, seqs)
    hx = torch.empty(B * n, D, dtype=BF, device="cuda")
    A.block_norm(None, r0, h=hx, w_pre=n1)
    y1 = lay.forward(hx).clone()
    assert torch.equal(y1, ya)
    # a norm apart reads the stream as stored, joined it reads the sum before that rounding
    ref, _ = OB.block_norm(f64(y1), f64(r0), w_post=f64(post), alpha=0.5)
    bound = HALF[res] * np.abs(ref) + 60 * U * (np.abs(ref) + np.abs(f64(r0))) + TINY
    assert_within(f64(r1), ref, bound, "r after the layer")
    assert_within(f64(h2), OB.norm(ref, f64(n2), 1e-5), (HALF[BF] + 100 * U) * np.abs(OB.norm(ref, f64(n2), 1e-5)) + 60 * U, "h")
    y2 = mix.forward(h2, seqs).clone()
    ref, _ = OB.block_norm(f64(y2), f64(r1), scale=f64(scale))
    bound = HALF[res] * np.abs(ref) + 60 * U * (np.abs(ref) + np.abs(f64(r1))) + TINY
    assert_within(f64(r2), ref, bound, "r after the mixer")
    assert_written(h3, "h")
    # decoding a token per sequence through both blocks runs and leaves a finite stream
    cache, state = lay.new_cache(32), mix.new_state(B)
    rt = torch.randn(B, D, generator=g).to(res).cuda()
    for _ in range(3):
        rt, ht = one.decode_step(cache, rt, next_norm=n2)
        rt, ht = two.decode_step(state, rt, h=ht, next_norm=n3)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(rt.float()).all()) and lay.status.item() == 0 and mix.status.item() == 0


def test_mixer_refuses_wrong_weights_and_too_many_tokens():
    w = cuda(mixer_weights(64, 128, 16, 4, 1))
    for name in w:
        bad = dict(w, **{name: w[name][:-1]})
        with pytest.raises(A.AttambaError, match=name):
            layer.SsmMixer(64, 128, 16, 4, bad, 8)
    with pytest.raises(A.AttambaError, match="A must"):
        layer.SsmMixer(64, 128, 16, 4, {k: v for k, v in w.items() if k != "A"}, 8)
    mix = layer.SsmMixer(64, 128, 16, 4, {k: v for k, v in w.items() if k not in ("conv_b", "bias", "skip")}, 8)
    h = torch.zeros(9, 64, dtype=BF, device="cuda")
    with pytest.raises(A.AttambaError, match="holds 1 to 8"):
        mix.forward(h, A.Seqs(i32([0, 9]), 9))
    assert mix.forward(h[:8], A.Seqs(i32([0, 8]), 8)).abs().max().item() == 0.0


def test_decode_step_in_a_captured_graph():
    """Two blocks' decode step captured once and replayed, new tokens copied into its input, against eager steps: the same
    streams and states, bit for bit."""
    D, Di, N, K, B = 128, 256, 16, 4, 5
    mixers = [layer.SsmMixer(D, Di, N, K, cuda(mixer_weights(D, Di, N, K, 20 + k)), B) for k in range(2)]
    g = torch.Generator().manual_seed(2)
    norms = [torch.rand(D, generator=g).cuda() + 0.5 for _ in range(4)]
    blocks = [layer.Block(m, norms[k], w_post=norms[2 + k], alpha=0.7) for k, m in enumerate(mixers)]
    slots = i32([3, 0, -1, 5, 1])
    tokens = torch.randn(4, B, D, generator=g).cuda()

    def step(states, r):
        h = None
        for k, b in enumerate(blocks):
            r, h = b.decode_step(states[k], r, h=h, slots=slots, next_norm=norms[1] if k == 0 else None)
        return r

    eager_states = [m.new_state(6) for m in mixers]
    eager = [step(eager_states, t.clone()).clone() for t in tokens]
    states, r = [m.new_state(6) for m in mixers], tokens[0].clone()
    step(states, r)                      # warm-up ahead of the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(states, r)
    for win, ssm in states:
        win.zero_()
        ssm.zero_()
    live = [0, 1, 3, 4]                  # row 2 fills the batch up: its mixer output is what the buffer held
    for t, want in zip(tokens, eager):
        r.copy_(t)
        graph.replay()
        assert torch.equal(r[live], want[live])
    for (win, ssm), (ewin, essm) in zip(states, eager_states):
        assert torch.equal(win, ewin) and torch.equal(ssm, essm)
    assert all(m.status.item() == 0 for m in mixers)
